// Launches of the units of many query rows over a cache of 8-bit codes (rope_attend_tc.cuh).
#include "rope_attend_tc.cuh"
#include "serving.h"

namespace rope {
namespace attend {
namespace {

template <typename T, int DP>
cudaError_t launch(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c, cudaStream_t stream) {
  auto kernel = attend_tc_kernel<T, DP, Code>;
  constexpr size_t smem = sizeof(TcShared<DP, true>);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  const cudaError_t e = opt_in_shared(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped_smem(kernel, (unsigned)c.grid, TcShape<DP, true>::kThreads, smem, stream,
                                static_cast<const T*>(p.query), static_cast<const Code*>(p.k_cache),
                                static_cast<const Code*>(p.v_cache), static_cast<T*>(p.out), p.lse, g, a, c);
}

template <typename T>
cudaError_t launch_typed(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c,
                         cudaStream_t stream) {
  if (p.D <= 64) return launch<T, 64>(p, g, a, c, stream);
  if (p.D <= 128) return launch<T, 128>(p, g, a, c, stream);
  return launch<T, 256>(p, g, a, c, stream);
}

}  // namespace

cudaError_t launch_codes_tall(const AttendProblem& p, const Pointers& g, const AttendArgs& a, const Cut& c,
                              cudaStream_t stream) {
  return p.dtype == kF16 ? launch_typed<__half>(p, g, a, c, stream) : launch_typed<__nv_bfloat16>(p, g, a, c, stream);
}

}  // namespace attend
}  // namespace rope
