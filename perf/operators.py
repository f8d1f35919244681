"""The score-modified attention and rotary operators as they are measured: cases,
inputs, their plain forms in torch and the calls a user makes.

Attention.  For query row i (of Tq) and key j (of Tk), off = Tk - Tq:
    x_ij = scale * q_i . k_j
    x_ij = c * tanh(x_ij / c)                       with a soft cap c
    x_ij = x_ij - slope_h * |i + off - j|           with distance slopes
    visible: j <= i + off (causal) or j < prefix;  j > i + off - window;
             doc(i) == doc(j) >= 0
    P = softmax over the visible keys, O = P V, L = logsumexp of the visible x
    (a row that sees nothing: O = 0, L = -inf, no gradient)
    dP = dO V^T, dx = P (dP - rowsum(P dP)), through the cap: dx (1 - tanh^2)
    dQ = scale dx K, dK = scale dx^T Q, dV = P^T dO
Rotary.  Frequency f of section a turns its pair of channels by
positions[a, b, t] * inv_freq[f]; the gradient turns back.
"""
import math

import numpy as np
import torch

own = False

FREQ_BASE = 1e6


def _attn(name, B, Hq, Hkv, Tq, Tk, d, dv=0, causal=True, window=0, softcap=0.0, slopes=False, docs="", prefix="",
          grad=False):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "Tq": Tq, "Tk": Tk, "d": d, "dv": dv or d,
            "causal": causal, "window": window, "softcap": softcap, "slopes": slopes, "docs": docs, "prefix": prefix,
            "grad": grad}


def _rotary(name, B, Hq, Hkv, T, d, rot, sections, interleaved=False, first=0, grad=False):
    return {"name": name, "op": "rotary", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "d": d, "rot": rot,
            "sections": sections, "interleaved": interleaved, "first": first, "grad": grad}


def listed():
    return [
        # the smallest call: one head of two tiles, where launch and set-up are all there is
        _attn("capped_T256_d64", 1, 1, 1, 256, 256, 64, causal=False, softcap=30.0),
        # a capped layer of a long-context model in training (the headline shape of the benchmark), forward alone
        _attn("capped_T8192_d128", 2, 32, 8, 8192, 8192, 128, softcap=50.0),
        # a distance-biased layer, many short heads of 64
        _attn("distance_T2048_d64", 4, 16, 16, 2048, 2048, 64, slopes=True),
        # one packed row of documents of very different lengths, its end padded
        _attn("documents_T8192_d128", 1, 32, 8, 8192, 8192, 128,
              docs="1900,37,411,1024,129,2600,5,700,888,301"),
        # a question of 32 tokens over a long context, capped and distance-biased
        _attn("appended_Tq32_Tk8032", 1, 32, 8, 32, 8032, 128, softcap=50.0, slopes=True),
        # a training step of a prefix-LM batch: each row sees its own prompt both ways (ragged length)
        _attn("prefix_step_T2001_d128", 2, 16, 4, 2001, 2001, 128, prefix="700,45", grad=True),
        # a training step of a capped layer over packed documents
        _attn("capped_documents_step_T8192_d128", 1, 32, 8, 8192, 8192, 128, softcap=50.0,
              docs="3001,1095,2048,650,1398", grad=True),
        # a training step of a distance-biased layer, heads of 64
        _attn("distance_step_T2048_d64", 4, 16, 16, 2048, 2048, 64, slopes=True, grad=True),
        # a small training step with everything on: ragged, a window, padded documents, values wider than keys
        _attn("all_step_T777_d64_dv128", 2, 6, 2, 777, 777, 64, dv=128, window=200, softcap=20.0, slopes=True,
              docs="300,2,200,250|511,266", grad=True),
        # one new token of each of 32 requests, far into its context
        _rotary("rotary_B32_T1", 32, 32, 8, 1, 128, 128, "16,24,24", first=100000),
        # the prompt of a video model: three axes, from the packed projection
        _rotary("rotary_B2_T8192", 2, 32, 8, 8192, 128, 128, "16,24,24"),
        # the gradient of a partly rotated layer with odd lengths, pairs of neighbours
        _rotary("rotary_grad_B3_T4099", 3, 16, 16, 4099, 64, 32, "8,8", interleaved=True, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut(rng, T):
    """Lengths of documents that fill most of T."""
    left, lens = T - (rng.randrange(T // 8 + 1) if rng.random() < 0.5 else 0), []
    while left > 0:
        n = min(left, _log_int(rng, 1, max(2, T // 2)))
        lens.append(n if len(lens) < 60 else left)
        left -= lens[-1]
    return ",".join(map(str, lens))


def draw(rng):
    if rng.random() < 0.3:
        d = rng.choice((64, 128))
        rot = rng.choice((d, d, d // 2))
        G, Hkv = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8))
        B = rng.choice((1, 2, 3, 8, 32))
        T = _log_int(rng, 1, max(2, min(8192, 2 * 40 * 8192 * 128 // (B * Hkv * (G + 1) * d))))
        half = rot // 2
        a = rng.randrange(1, half - 1)
        sections = rng.choice((str(half), "%d,%d" % (a, half - a),
                               "%d,%d,%d" % (half // 4, half // 4 + half // 8, half - half // 2 - half // 8)))
        c = _rotary("", B, G * Hkv, Hkv, T, d, rot, sections, rng.random() < 0.4, rng.choice((0, 5, 100000)),
                    rng.random() < 0.5)
        del c["name"]
        return c
    d, dv = rng.choice(((64, 64), (128, 128), (128, 128), (64, 128), (128, 64)))
    G, Hkv, B = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8)), rng.choice((1, 1, 2, 3))
    grad = rng.random() < 0.5
    room = 2 * 32 * 8192 * 8192 / (B * G * Hkv * (5.0 if grad else 1.0))  # scores of the largest listed case
    # training sequences start at some dozens of tokens (the gradient of a row that sees one key is zero), calls at one
    T = _log_int(rng, 64 if grad else 1, min(8192, int(room ** 0.5)))
    kind = rng.choice(("plain", "plain", "docs", "prefix", "cross"))
    causal = kind == "prefix" or rng.random() < 0.7
    Tq = T if kind != "cross" else _log_int(rng, min(T, 64) if grad else 1, T)
    docs = "|".join(_cut(rng, T) for _ in range(B)) if kind == "docs" else ""
    prefix = ",".join(str(rng.randrange(T + 1)) for _ in range(B)) if kind == "prefix" else ""
    softcap = rng.choice((0.0, 15.0, 30.0, 50.0))
    slopes = rng.random() < 0.4
    if not (softcap or slopes or docs or prefix):
        softcap = 40.0
    window = rng.randrange(1, T + 1) if causal and not prefix and rng.random() < 0.25 else 0
    c = _attn("", B, G * Hkv, Hkv, Tq, T, d, dv, causal, window, softcap, slopes, docs, prefix, grad)
    del c["name"]
    return c


def _doc_ids(case):
    """[B, T] document of each token, -1 past the last one."""
    rows = case["docs"].split("|")
    ids = np.full((case["B"], case["Tk"]), -1, np.int32)
    for b in range(case["B"]):
        at = 0
        for n, length in enumerate(int(x) for x in rows[b % len(rows)].split(",")):
            ids[b, at:at + length] = n
            at += length
    return ids


def _prefix(case):
    p = [int(x) for x in case["prefix"].split(",")]
    return np.array([p[b % len(p)] for b in range(case["B"])], np.int32)


def _slopes(H):
    return 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H)


def _pairs(case):
    """Visible (query, key) pairs of one head, all batch rows."""
    B, Tq, Tk = case["B"], case["Tq"], case["Tk"]
    at = np.arange(Tq) + Tk - Tq
    total = 0
    ids = _doc_ids(case) if case["docs"] else None
    prefix = _prefix(case) if case["prefix"] else None
    for b in range(B):
        hi = np.full(Tq, Tk)
        if case["causal"]:
            hi = np.minimum(np.maximum(at + 1, prefix[b] if prefix is not None else 0), Tk)
        lo = np.maximum(at - case["window"] + 1, 0) if case["window"] else np.zeros(Tq, np.int64)
        if ids is not None:
            first = np.searchsorted(np.where(ids[b] < 0, 1 << 30, ids[b]), ids[b], "left")
            last = np.searchsorted(np.where(ids[b] < 0, 1 << 30, ids[b]), ids[b], "right")
            lo = np.maximum(lo, first)
            hi = np.where(ids[b] < 0, 0, np.minimum(hi, last))
        total += int(np.maximum(hi - lo, 0).sum())
    return total


def work(case):
    if case["op"] == "rotary":
        n = case["B"] * (case["Hq"] + case["Hkv"]) * case["T"] * case["d"]
        turned = n * case["rot"] / case["d"]
        axes = len(case["sections"].split(","))
        return {"bytes": 4 * n + 4 * axes * case["B"] * case["T"] + 2 * case["rot"], "flops": 3 * turned}
    B, Hq, Hkv, Tq, Tk, d, dv = (case[k] for k in ("B", "Hq", "Hkv", "Tq", "Tk", "d", "dv"))
    pairs = _pairs(case) * Hq
    q, kv, rows = 2 * B * Hq * Tq * d, 2 * B * Hkv * Tk * (d + dv), B * Hq * Tq
    bytes_, flops = q + kv + 2 * rows * dv + 4 * rows, 2 * pairs * (d + dv)
    if case["grad"]:
        bytes_ += q + kv + 2 * rows * dv
        flops += 2 * pairs * (3 * d + 2 * dv)
    return {"bytes": bytes_ + (8 * B * Tk if case["docs"] else 0), "flops": flops}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    if case["op"] == "rotary":
        B, Hq, Hkv, T, d, rot = (case[k] for k in ("B", "Hq", "Hkv", "T", "d", "rot"))
        sections = [int(x) for x in case["sections"].split(",")]
        axes = len(sections)
        inv_freq = FREQ_BASE ** (-torch.arange(rot // 2, device=dev, dtype=torch.float64) * 2 / rot)
        t = torch.arange(T, device=dev, dtype=torch.int32) + case["first"]
        start = torch.randint(0, 1000, (axes, B, 1), generator=g, device=dev, dtype=torch.int32)
        # time, height, width of a 24-wide frame of patches; one axis: the token's place
        walk = torch.stack([t // 384, t // 24 % 16, t % 24, t][:axes] if axes > 1 else [t])
        s = {"case": case, "positions": (start + walk[:, None, :]).contiguous(), "inv_freq": inv_freq.float(),
             "sections": sections,
             "axis": torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=dev)}
        if case["grad"]:  # the attention's gradients, [B, H, T, d]
            s["Q"], s["K"] = normal(B, Hq, T, d), normal(B, Hkv, T, d)
        else:  # views of the packed projection [B, T, (Hq + 2 Hkv) d]
            qkv = normal(B, T, Hq + 2 * Hkv, d)
            s["Q"], s["K"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        return s
    B, Hq, Hkv, Tq, Tk, d, dv = (case[k] for k in ("B", "Hq", "Hkv", "Tq", "Tk", "d", "dv"))
    s = {"case": case, "Q": normal(B, Hq, Tq, d, std=1.5), "K": normal(B, Hkv, Tk, d),
         "V": normal(B, Hkv, Tk, dv), "slopes": None, "docs": None, "prefix": None}
    if case["grad"]:
        s["dO"] = normal(B, Hq, Tq, dv)
    if case["slopes"]:
        s["slopes"] = _slopes(Hq).float().to(dev)
    if case["docs"]:
        s["docs"] = torch.from_numpy(_doc_ids(case)).to(dev)
    if case["prefix"]:
        s["prefix"] = torch.from_numpy(_prefix(case)).to(dev)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _plain_rotary(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = s["positions"].double()[s["axis"]].permute(1, 2, 0) * s["inv_freq"].double()  # [B, T, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["grad"]:
        sin = -sin

    def turn(x):
        y = x.float().clone(memory_format=torch.contiguous_format)
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        a, b = x[..., first].float(), x[..., second].float()
        y[..., first] = a * cos - b * sin
        y[..., second] = b * cos + a * sin
        return y.to(x.dtype)

    return turn(s["Q"]), turn(s["K"])


def _visible(s, dev):
    """[B or 1, Tq, Tk] truth values."""
    case = s["case"]
    at = torch.arange(case["Tq"], device=dev)[:, None] + case["Tk"] - case["Tq"]
    j = torch.arange(case["Tk"], device=dev)[None, :]
    vis = torch.ones(1, case["Tq"], case["Tk"], dtype=torch.bool, device=dev)
    if case["causal"]:
        vis = vis & (j <= at)
    if s["prefix"] is not None:
        vis = vis | (j < s["prefix"][:, None, None])
    if case["window"]:
        vis = vis & (j > at - case["window"])
    if s["docs"] is not None:
        ids = s["docs"]
        vis = vis & (ids[:, :, None] == ids[:, None, :]) & (ids >= 0)[:, :, None]
    return vis


def _plain_attention(s):
    case = s["case"]
    B, Hq, Hkv, Tq, Tk, d, dv = (case[k] for k in ("B", "Hq", "Hkv", "Tq", "Tk", "d", "dv"))
    G, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    Q = s["Q"].float().view(B, Hkv, G * Tq, d)
    K, V = s["K"].float(), s["V"].float()
    x = torch.matmul(Q, K.transpose(-1, -2)).mul_(scale)
    t = None
    if case["softcap"]:
        t = x.div_(case["softcap"]).tanh_()
        x = t * case["softcap"]
        if not case["grad"]:
            t = None
    x = x.view(B, Hkv, G, Tq, Tk)
    if s["slopes"] is not None:
        at = torch.arange(Tq, device=x.device, dtype=torch.float32)[:, None] + (Tk - Tq)
        far = (at - torch.arange(Tk, device=x.device, dtype=torch.float32)).abs()
        x.sub_(s["slopes"].view(1, Hkv, G, 1, 1) * far)
    x.masked_fill_(~_visible(s, x.device)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    L = (m + l.log()).view(B, Hq, Tq)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l))).view(B, Hkv, G * Tq, Tk)
    O = torch.matmul(p, V)
    out = {"O": O.view(B, Hq, Tq, dv).to(torch.bfloat16), "L": L}
    if case["grad"]:
        dO = s["dO"].float().view(B, Hkv, G * Tq, dv)
        out["dV"] = torch.matmul(p.transpose(-1, -2), dO).to(torch.bfloat16)
        dx = torch.matmul(dO, V.transpose(-1, -2))
        dx = dx.sub_((O * dO).sum(-1, keepdim=True)).mul_(p)
        if t is not None:
            dx.mul_(1 - t.square_())
        out["dQ"] = torch.matmul(dx, K).mul_(scale).view(B, Hq, Tq, d).to(torch.bfloat16)
        out["dK"] = torch.matmul(dx.transpose(-1, -2), Q).mul_(scale).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    s = state
    case = s["case"]
    if not own:
        if case["op"] == "rotary":
            return _plain_rotary(s)
        return _plain_attention(s)
    import tiled_attention_05_gb300 as fa

    if case["op"] == "rotary":
        call = fa.fa_rotary_backward if case["grad"] else fa.fa_rotary
        return call(s["Q"], s["K"], s["positions"], s["inv_freq"], sections=s["sections"],
                    interleaved=case["interleaved"])
    mask = None
    if s["docs"] is not None or s["prefix"] is not None:
        mask = fa.fa_mask_plan(case["B"], case["Tq"], case["Tk"], case["causal"], window=case["window"],
                               doc_q=s["docs"], doc_k=s["docs"], prefix=s["prefix"])
    mods = dict(window=case["window"], softcap=case["softcap"], slopes=s["slopes"], mask=mask)
    O, L = fa.fa_forward(s["Q"], s["K"], s["V"], case["causal"], **mods)
    out = {"O": O, "L": L}
    if case["grad"]:
        out["dQ"], out["dK"], out["dV"] = fa.fa_backward(s["Q"], s["K"], s["V"], O, s["dO"], L, case["causal"], **mods)
    return out


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        out = []
        owner = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
        theta = torch.stack([s["positions"][a].double() * f for a, f in zip(owner, s["inv_freq"].double())], -1)
        spin = torch.polar(torch.ones_like(theta), -theta if case["grad"] else theta).unsqueeze(1)
        n = len(owner)
        for x in (s["Q"].double(), s["K"].double()):
            pairs = x[..., :2 * n].unflatten(-1, (n, 2) if case["interleaved"] else (2, n))
            re, im = pairs.unbind(-1 if case["interleaved"] else -2)
            z = torch.complex(re, im) * spin
            y = torch.stack((z.real, z.imag), -1 if case["interleaved"] else -2).flatten(-2)
            out.append(torch.cat((y, x[..., 2 * n:]), -1))
        return tuple(out)
    B, Hq, Hkv, Tq, Tk = (case[k] for k in ("B", "Hq", "Hkv", "Tq", "Tk"))
    got = {k: [] for k in (("O", "L", "dQ", "dK", "dV") if case["grad"] else ("O", "L"))}
    dev = s["Q"].device
    i = torch.arange(Tq, device=dev).view(-1, 1) + (Tk - Tq)
    j = torch.arange(Tk, device=dev).view(1, -1)
    for b in range(B):
        hidden = torch.zeros(Tq, Tk, dtype=torch.bool, device=dev)
        if case["causal"]:
            hidden |= j > i
        if s["prefix"] is not None:
            hidden &= j >= int(s["prefix"][b])
        if case["window"]:
            hidden |= i - j >= case["window"]
        if s["docs"] is not None:
            hidden |= s["docs"][b].view(-1, 1) != s["docs"][b].view(1, -1)
            hidden |= (s["docs"][b] < 0).view(1, -1)
        none = hidden.all(1)
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            q, k, v = (x.double().requires_grad_(case["grad"]) for x in (s["Q"][b, h], s["K"][b, kv], s["V"][b, kv]))
            score = q @ k.t() / case["d"] ** 0.5
            if case["softcap"]:
                score = case["softcap"] * torch.tanh(score / case["softcap"])
            if s["slopes"] is not None:
                score = score - float(s["slopes"][h]) * (i - j).abs()
            score = torch.where(hidden & ~none.view(-1, 1), -math.inf, score)
            weight = torch.softmax(score, -1) * (~none).view(-1, 1)
            o = weight @ v
            got["O"].append(o.detach())
            got["L"].append(torch.where(none, -math.inf, torch.logsumexp(score.detach(), -1)))
            if case["grad"]:
                for name, x in zip(("dQ", "dK", "dV"), torch.autograd.grad(o, (q, k, v), s["dO"][b, h].double())):
                    got[name].append(x)
    out = {k: torch.stack(v).unflatten(0, (B, Hq)) for k, v in got.items()}
    for k in ("dK", "dV"):
        if k in out:
            out[k] = out[k].unflatten(1, (Hkv, Hq // Hkv)).sum(2)
    return out
