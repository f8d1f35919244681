// Score-modified forward instances (fa_fwd_kernel.cuh) with Q and K heads of 128, packed and split.
#include "fa_fwd_kernel.cuh"

namespace {

template <int HDV>
fa::FwdLauncher launcher(int bits) {
  constexpr int F = fa::kFew;
  switch (bits) {
    case 0:
      return launch_fwd_t<128, HDV, false, false, F>;
    case fa::kCap:
      return launch_fwd_t<128, HDV, false, false, F | fa::kCap>;
    case fa::kCap | fa::kBounded:
      return launch_fwd_t<128, HDV, false, false, F | fa::kCap | fa::kBounded>;
    case fa::kSlopes:
      return launch_fwd_t<128, HDV, false, false, F | fa::kSlopes>;
    case fa::kCap | fa::kSlopes:
      return launch_fwd_t<128, HDV, false, false, F | fa::kCap | fa::kSlopes>;
  }
  return launch_fwd_t<128, HDV, false, false, F | fa::kCap | fa::kSlopes | fa::kBounded>;
}

}  // namespace

fa::FwdLauncher fa::fwd_scored_few_128(const Problem& p, const ScoreMods& m) {
  return p.dv == 64 ? launcher<64>(m.fwd_bits(p.Tk)) : launcher<128>(m.fwd_bits(p.Tk));
}
