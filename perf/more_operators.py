"""The key/value cache operators as they are measured: cases, inputs, their plain
forms in torch and the calls a user makes.

Cache.  K [pages, Hkv, page, d] and V [pages, Hkv, page, dv], bf16, or e4m3 with one
fp32 scale for each row of d (dv) values.  tables[b] lists the pages of sequence b:
its position p is row p % page of page tables[b][p / page].
Write.  Token t < counts[b] of sequence b goes to position starts[b] + t:
    a = max(|x|) (2^-60 at least), code = e4m3(x * (448 / a)), scale = a * (1 / 448)
Read back.  bf16(code * scale) of positions 0 .. lengths[b] - 1, zeros after them.
Attention.  Row t (of Tq) of sequence b stands at its position p = lengths[b] - Tq + t,
behind P tokens of a prefix that a group of sequences shares (P = 0 without one); it
sees the P prefix keys and its own keys j <= p.  With key positions counted from the
prefix's start, x = scale * q . k, then
    x = c * tanh(x / c)                     with a soft cap c
    x = x - slope_h * (P + p - position)    with distance slopes
    visible: P + p - position < window      with a window
    O = softmax(x) V over what is visible, L = logsumexp of it
(p < 0: a padding row, which sees nothing: O = 0, L = -inf).
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
LEAST = 2.0 ** -60


def _write(name, B, Hkv, T, d, dv=0, quant=True, page=64, lo=0, start=0, packed=False):
    return {"name": name, "op": "write", "B": B, "Hkv": Hkv, "T": T, "d": d, "dv": dv or d, "quant": quant, "page": page,
            "lo": lo or T, "start": start, "packed": packed}


def _read(name, B, Hkv, T, d, dv=0, quant=True, page=64, lo=0):
    return {"name": name, "op": "read", "B": B, "Hkv": Hkv, "T": T, "d": d, "dv": dv or d, "quant": quant, "page": page,
            "lo": lo or T}


def _attn(name, B, Hq, Hkv, Tq, lo, hi, d, dv=0, quant=True, page=64, window=0, softcap=0.0, slopes=False, groups=0,
          prefix=0):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "Tq": Tq, "lo": lo, "hi": hi, "d": d,
            "dv": dv or d, "quant": quant, "page": page, "window": window, "softcap": softcap, "slopes": slopes,
            "groups": groups, "prefix": prefix}


def listed():
    return [
        # one new token of each of 32 requests, far into its context: a decoding step's write
        _write("write_B32_T1", 32, 8, 1, 128, start=5000),
        # two prompts as they come out of the projection, quantised
        _write("write_B2_T8192", 2, 8, 8192, 128, packed=True),
        # padded prompts of odd lengths behind a cached part, heads of 64, kept in bf16
        _write("write_B3_T4099_d64_bf16", 3, 16, 4099, 64, quant=False, page=16, lo=1000, start=37),
        # a quantised context back as the forward takes it (the next chunk of a long prompt)
        _read("read_B2_T8192", 2, 8, 8192, 128),
        # the same of small odd sequences, values wider than keys
        _read("read_B5_T777_d64_dv128", 5, 2, 777, 64, dv=128, page=32, lo=1),
        # the smallest call: one short sequence, where latency is all there is
        _attn("decode_B1_T200_d64_bf16", 1, 8, 2, 1, 200, 200, 64, quant=False, page=16),
        # a decoding step of 32 requests, quantised cache
        _attn("decode_B32_T8192", 32, 32, 8, 1, 8192, 8192, 128),
        # a few very long contexts in bf16
        _attn("decode_B4_T65536_bf16", 4, 32, 8, 1, 50000, 65536, 128, quant=False, page=128),
        # four drafted tokens of each of 48 requests of mixed lengths, capped scores, a window
        _attn("drafts_B48_Tq4_capped", 48, 16, 4, 4, 3, 7000, 128, window=4096, softcap=50.0),
        # 64 answers to one prompt, each a few hundred tokens long
        _attn("shared_B64_P8192", 64, 32, 8, 1, 16, 1000, 128, groups=1, prefix=8192),
        # sampling for training: 16 answers to each of 8 prompts, bf16 heads of 64, distance slopes
        _attn("shared_B128_P2001_groups_d64_bf16", 128, 16, 8, 1, 1, 700, 64, quant=False, page=32, slopes=True, groups=8,
              prefix=2001),
        # the largest: many answers to one long document
        _attn("shared_B256_P32768_bf16", 256, 32, 8, 1, 100, 600, 128, quant=False, groups=1, prefix=32768),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d, dv = rng.choice(((64, 64), (128, 128), (128, 128), (64, 128), (128, 64)))
    quant, page, Hkv = rng.random() < 0.6, rng.choice((16, 32, 64, 128, 256)), rng.choice((1, 2, 4, 8))
    op = rng.choice(("write", "read", "attention", "attention", "shared", "shared"))
    if op in ("write", "read"):
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(2, min(8192, 2 * 8 * 8192 // (B * Hkv))))
        lo = rng.choice((T, rng.randrange(1, T + 1)))
        c = _write("", B, Hkv, T, d, dv, quant, page, lo, rng.choice((0, rng.randrange(3000))), rng.random() < 0.5) \
            if op == "write" else _read("", B, Hkv, T, d, dv, quant, page, lo)
        del c["name"]
        return c
    G, Tq = rng.choice((1, 2, 4, 8)), rng.choice((1, 1, 1, 2, 3, 5, 8))
    groups = prefix = 0
    B = _log_int(rng, 1, 128)
    if op == "shared":
        groups = rng.choice((1, 1, 2, 5))
        B = groups * _log_int(rng, 2, 128 // groups)
        # flops: rows times keys of the largest listed case at most
        prefix = _log_int(rng, 50, min(32768, 256 * 32 * 32768 // (B * G * Hkv * Tq)))
    hi = _log_int(rng, Tq, max(Tq + 1, min(65536 if not prefix else 2000, 200_000 * 8 // (B * Hkv))))
    lo = rng.choice((hi, rng.randrange(1, hi + 1)))
    c = _attn("", B, G * Hkv, Hkv, Tq, lo, hi, d, dv, quant, page,
              _log_int(rng, 1, prefix + hi) if rng.random() < 0.2 else 0, rng.choice((0.0, 0.0, 20.0, 50.0)),
              rng.random() < 0.25, groups, prefix)
    del c["name"]
    return c


def _spread(lo, hi, B):
    """B lengths between lo and hi, the longest among them, in no order."""
    at = np.arange(B) * 0.6180339887498949 % 1.0
    n = lo + np.floor((hi - lo + 1) * at).astype(np.int64)
    n[B // 2] = hi
    return np.minimum(n, hi)


def _seen(case):
    """(visible pairs of one query head, keys that any row sees), over the batch."""
    B, Tq, P, W = case["B"], case["Tq"], case["prefix"], case["window"] or 1 << 40
    lens = _spread(case["lo"], case["hi"], B)
    pos = lens[:, None] - Tq + np.arange(Tq)
    live = pos >= 0
    mine, total = np.where(live, np.minimum(pos + 1, W), 0), np.where(live, np.minimum(P + pos + 1, W), 0)
    first = np.where(live, P + pos - W + 1, 1 << 40).min(1)  # per sequence, counted from the prefix's start
    keys = np.where(live.any(1), lens - np.clip(first - P, 0, None), 0).sum()
    if P:
        keys += np.clip(P - np.clip(first.reshape(case["groups"], -1).min(1), 0, None), 0, None).sum()
    assert (mine <= total).all()
    return int(total.sum()), int(keys)


def work(case):
    Hkv, dd = case["Hkv"], case["d"] + case["dv"]
    held = (dd + 8) if case["quant"] else 2 * dd  # bytes of a key and its value in the cache
    if case["op"] != "attention":
        rows = int(_spread(case["lo"], case["T"], case["B"]).sum()) * Hkv
        whole = case["B"] * case["T"] * Hkv if case["op"] == "read" else rows
        return {"bytes": rows * held + whole * 2 * dd, "flops": rows * dd * (2 if case["quant"] else 0)}
    pairs, keys = _seen(case)
    rows = case["B"] * case["Hq"] * case["Tq"]
    return {"bytes": keys * Hkv * held + rows * (2 * dd + 4), "flops": 2 * dd * pairs * case["Hq"]}


# ---------------------------------------------------------------- inputs
def _quantise(x):
    a = x.float().abs().amax(-1, keepdim=True).clamp_min(LEAST)
    f = torch.full_like(a, E4M3_MAX) / a  # (a number divided by a tensor would be its product with a reciprocal)
    return (x.float() * f).to(torch.float8_e4m3fn), (a * (1.0 / E4M3_MAX)).squeeze(-1)


def _tables(g, dev, rows, n, first):
    """Pages first, first + 1, ... dealt to `rows` tables of n in no order."""
    return (torch.randperm(rows * n, generator=g, device=dev) + first).view(rows, n).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hkv, d, dv, page, quant = (case[k] for k in ("B", "Hkv", "d", "dv", "page", "quant"))

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    s = {"case": case}
    T = {"write": lambda: case["start"] + case["T"], "read": lambda: case["T"], "attention": lambda: case["hi"]}[case["op"]]()
    n = -(-T // page)
    lens = torch.from_numpy(_spread(case["lo"], case["hi"] if case["op"] == "attention" else case["T"], B)).to(dev, torch.int32)
    s["lengths"], s["tables"], pages = lens, _tables(g, dev, B, n, 0), B * n
    if case["op"] == "attention" and case["prefix"]:
        S, m = case["groups"], -(-case["prefix"] // page)
        s["prefix_tables"], pages = _tables(g, dev, S, m, pages), pages + S * m
        s["prefix_lengths"] = torch.full((S,), case["prefix"], dtype=torch.int32, device=dev)
        s["prefix_starts"] = torch.arange(S + 1, dtype=torch.int32, device=dev) * (B // S)
    if case["op"] == "write":
        kind = torch.float8_e4m3fn if quant else torch.bfloat16
        s["K"], s["V"] = (torch.zeros(pages, Hkv, page, w, dtype=torch.bfloat16, device=dev).to(kind) for w in (d, dv))
        s["k_scale"], s["v_scale"] = (torch.zeros(pages, Hkv, page, device=dev) if quant else None for _ in range(2))
        s["starts"] = torch.full((B,), case["start"], dtype=torch.int32, device=dev)
        # values differ in size from token to token, as they do in a model
        size = torch.exp(torch.randn(B, case["T"], 1, 1, generator=g, device=dev))
        if case["packed"] and d == dv:  # views of the packed projection [B, T, (K heads, V heads) d]
            kv = (normal(B, case["T"], 2 * Hkv, d) * size).to(torch.bfloat16)
            s["new_K"], s["new_V"] = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
        else:
            s["new_K"], s["new_V"] = ((normal(B, case["T"], Hkv, w) * size).to(torch.bfloat16).transpose(1, 2).contiguous()
                                      for w in (d, dv))
        return s
    # (filled page by page: the fp32 values of a large pool at once would be many times its size)
    step = max(1, (1 << 26) // (Hkv * page * max(d, dv)))
    for what, w in (("K", d), ("V", dv)):
        parts = [normal(min(step, pages - i), Hkv, page, w) for i in range(0, pages, step)]
        if quant:
            parts = [_quantise(x) for x in parts]
            s["k_scale" if what == "K" else "v_scale"] = torch.cat([p[1] for p in parts])
            s[what] = torch.cat([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn)
        else:
            s["k_scale" if what == "K" else "v_scale"] = None
            s[what] = torch.cat(parts)
    if case["op"] == "attention":
        H = case["Hq"]
        s["Q"] = normal(B, H, case["Tq"], d, std=1.5)
        s["slopes"] = None
        if case["slopes"]:
            s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H)).float().to(dev)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _gather(pages, scale, tables, T):
    """Positions 0 .. T - 1 of every table: fp32 [tables, Hkv, T, w]."""
    at = tables.long()
    x = pages.view(torch.uint8)[at].view(pages.dtype).float()  # [tables, n, Hkv, page, w]
    if scale is not None:
        x = x * scale[at].unsqueeze(-1)
    return x.transpose(1, 2).flatten(2, 3)[:, :, :T]


def _plain_write(s):
    case = s["case"]
    page = case["page"]
    b, t = torch.where(torch.arange(case["T"], device=s["tables"].device) < s["lengths"][:, None])
    p = s["starts"].long()[b] + t
    to, off = s["tables"].long()[b, p // page], p % page
    for new, pages, scale in ((s["new_K"], s["K"], s["k_scale"]), (s["new_V"], s["V"], s["v_scale"])):
        rows = new[b, :, t]  # [tokens, Hkv, w]
        if scale is None:
            pages[to, :, off] = rows
        else:
            codes, a = _quantise(rows)
            pages.view(torch.uint8)[to, :, off] = codes.view(torch.uint8)
            scale[to, :, off] = a
    return _cache_of(s)


def _cache_of(s):
    out = {"K": s["K"], "V": s["V"]}
    if s["k_scale"] is not None:
        out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
    return out


def _plain_read(s):
    T = s["case"]["T"]
    past = (torch.arange(T, device=s["tables"].device) >= s["lengths"][:, None])[:, None, :, None]
    return tuple(_gather(s[x], s[f], s["tables"], T).masked_fill_(past, 0.0).to(torch.bfloat16)
                 for x, f in (("K", "k_scale"), ("V", "v_scale")))


def _plain_attention(s):
    case = s["case"]
    B, Hq, Hkv, Tq, d, dv, P, S = (case[k] for k in ("B", "Hq", "Hkv", "Tq", "d", "dv", "prefix", "groups"))
    G, T, dev = Hq // Hkv, case["hi"], s["Q"].device
    Q = s["Q"].float().view(B, Hkv, G * Tq, d)
    x = torch.matmul(Q, _gather(s["K"], s["k_scale"], s["tables"], T).transpose(-1, -2)).view(B, Hkv, G, Tq, T)
    key = torch.arange(T, device=dev) + P
    if P:  # the rows of a group side by side against its prefix
        rows = Q.view(S, B // S, Hkv, G * Tq, d).transpose(1, 2).reshape(S, Hkv, -1, d)
        xp = torch.matmul(rows, _gather(s["K"], s["k_scale"], s["prefix_tables"], P).transpose(-1, -2))
        xp = xp.view(S, Hkv, B // S, G, Tq, P).transpose(1, 2).reshape(B, Hkv, G, Tq, P)
        x = torch.cat((xp, x), -1)
        key = torch.cat((torch.arange(P, device=dev), key))
        del xp
    x.mul_(1.0 / math.sqrt(d))
    if case["softcap"]:
        x.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    at = s["lengths"].long()[:, None] - Tq + torch.arange(Tq, device=dev) + P  # [B, Tq]
    far = at[:, :, None] - key
    if s["slopes"] is not None:
        x.sub_(s["slopes"].view(1, Hkv, G, 1, 1) * far.float()[:, None, None])
    hidden = (far < 0) | (at < P)[:, :, None]
    if case["window"]:
        hidden |= far >= case["window"]
    x.masked_fill_(hidden[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    L = (m + l.log()).view(B, Hq, Tq)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l)))
    O = torch.matmul(p[..., P:].reshape(B, Hkv, G * Tq, T), _gather(s["V"], s["v_scale"], s["tables"], T))
    if P:
        rows = p[..., :P].reshape(S, B // S, Hkv, G * Tq, P).transpose(1, 2).reshape(S, Hkv, -1, P)
        o = torch.matmul(rows, _gather(s["V"], s["v_scale"], s["prefix_tables"], P))
        O = O + o.view(S, Hkv, B // S, G * Tq, dv).transpose(1, 2).reshape(B, Hkv, G * Tq, dv)
    return O.view(B, Hq, Tq, dv).to(torch.bfloat16), L


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    case = s["case"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attention": _plain_attention}[case["op"]](s)
    import tiled_attention_05_gb300 as fa

    if "cache" not in s:  # the handle of the pools, which a program keeps as long as those
        s["cache"] = fa.KVCache(s["K"], s["V"], s["k_scale"], s["v_scale"])
    if case["op"] == "write":
        fa.fa_cache_write(s["cache"], s["new_K"], s["new_V"], s["tables"], s["starts"], counts=s["lengths"])
        return _cache_of(s)
    if case["op"] == "read":
        return fa.fa_cache_read(s["cache"], s["tables"], s["lengths"], case["T"])
    prefix = (s["prefix_tables"], s["prefix_lengths"], s["prefix_starts"]) if case["prefix"] else None
    return fa.fa_cache_attention(s["Q"], s["cache"], s["tables"], s["lengths"], window=case["window"],
                                 softcap=case["softcap"], slopes=s["slopes"], prefix=prefix)


# ---------------------------------------------------------------- from the definition, in 64 bits
def _nearest_e4m3(x):
    """The e4m3 value next to each x (ties to the even code): steps of 2^(e - 3) from 2^e on, of 2^-9 below 2^-6."""
    e = torch.frexp(x.abs().clamp_min(2.0 ** -6))[1] - 1
    step = torch.exp2((e - 3).double())
    return torch.round(x / step) * step


def _sequence(s, table, n):
    """fp64 K, V [Hkv, n, w] of the first n positions of one table."""
    page = s["case"]["page"]
    p = torch.arange(n, device=table.device)
    to, off = table.long()[p // page], p % page
    out = []
    for x, f in (("K", "k_scale"), ("V", "v_scale")):
        rows = s[x].view(torch.uint8 if s["case"]["quant"] else torch.int16)[to, :, off].view(s[x].dtype).double()
        out.append((rows if s[f] is None else rows * s[f][to, :, off].double()[..., None]).transpose(0, 1))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    lens = s["lengths"].tolist()
    if case["op"] == "write":
        page = case["page"]
        out = {k: v.double() for k, v in _cache_of(s).items()}
        for b, n in enumerate(lens):
            p = torch.arange(n, device=s["tables"].device) + case["start"]
            to, off = s["tables"][b].long()[p // page], p % page
            for new, x, f in ((s["new_K"], "K", "k_scale"), (s["new_V"], "V", "v_scale")):
                rows = new[b, :, :n].double().transpose(0, 1)
                if f in out:
                    top = rows.abs().amax(-1).clamp_min(LEAST)
                    out[f][to, :, off] = top / E4M3_MAX
                    rows = _nearest_e4m3(rows * (E4M3_MAX / top[..., None]))
                out[x][to, :, off] = rows
        return out
    if case["op"] == "read":
        K, V = (torch.zeros(case["B"], case["Hkv"], case["T"], w, dtype=torch.float64, device=s["tables"].device)
                for w in (case["d"], case["dv"]))
        for b, n in enumerate(lens):
            K[b, :, :n], V[b, :, :n] = _sequence(s, s["tables"][b], n)
        return K, V
    Hkv, G, Tq, P, W = case["Hkv"], case["Hq"] // case["Hkv"], case["Tq"], case["prefix"], case["window"]
    O, L, at_group = [], [], None
    for b, n in enumerate(lens):
        K, V = _sequence(s, s["tables"][b], n)
        if P:
            group = b // (case["B"] // case["groups"])
            if group != at_group:
                pk, pv = _sequence(s, s["prefix_tables"][group], P)
                at_group = group
            K, V = torch.cat((pk, K), 1), torch.cat((pv, V), 1)
        x = torch.einsum("hgtd,hjd->hgtj", s["Q"][b].double().unflatten(0, (Hkv, G)), K) / case["d"] ** 0.5
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        i = torch.arange(Tq, device=x.device).view(-1, 1) + P + n - Tq
        j = torch.arange(P + n, device=x.device).view(1, -1)
        if s["slopes"] is not None:
            x = x - s["slopes"].double().view(Hkv, G, 1, 1) * (i - j)
        sees = (j <= i) & (i >= P)
        if W:
            sees = sees & (i - j < W)
        x = torch.where(sees, x, -math.inf)
        L.append(torch.logsumexp(x, -1).flatten(0, 1))
        weight = torch.where(sees.any(-1, keepdim=True), torch.softmax(x, -1), 0.0)
        O.append(torch.einsum("hgtj,hjd->hgtd", weight, V).flatten(0, 1))
    return torch.stack(O), torch.stack(L)
