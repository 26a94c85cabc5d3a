// The tile kernel with the exponentials' epilogue (archead_cross_entropy).
#include "tile32.h"

namespace archead {

namespace {

template <int GC, int TT>
hipError_t launch_exp_g(const FwdArgs& a, const T32Exp& ex, hipStream_t s) {
  const T32Grid G = t32_grid(a, TT);
  const size_t codes = (size_t)kT32CB * 32 * t32_code_stride(a.ng);
  hipLaunchKernelGGL((tile32_exp_kernel<GC, TT>), dim3((unsigned)(G.ttiles * ex.vtiles)), dim3(kT32Threads), (uint32_t)codes, s, a, ex);
  return hipGetLastError();
}

template <int TT>
hipError_t launch_exp(const FwdArgs& a, const T32Exp& ex, hipStream_t s) {
  if (a.g == 32) return launch_exp_g<2, TT>(a, ex, s);
  if (a.g == 64) return launch_exp_g<1, TT>(a, ex, s);
  return launch_exp_g<0, TT>(a, ex, s);
}

}  // namespace

hipError_t launch_tile_exp(const FwdArgs& a, const T32Exp& ex, int tt, hipStream_t s) {
  switch (tt) {
    case 2: return launch_exp<2>(a, ex, s);
    case 4: return launch_exp<4>(a, ex, s);
    case 6: return launch_exp<6>(a, ex, s);
    default: return launch_exp<8>(a, ex, s);
  }
}

}  // namespace archead
