// Causal attention of new tokens over a paged KV cache of 8-bit codes with a shared prefix: the formulas of
// rope_attend.cu with k and v being code * scale.
#include <algorithm>

#include "rope_attend_join.cuh"

namespace rope {
namespace {

using namespace attend;

template <typename T>
cudaError_t launch_typed(const AttendProblem& p, cudaStream_t stream) {
  AttendArgs a;
  Pointers g;
  const cudaError_t er = arguments_of(p, sizeof(T), 1, a, g);
  if (er != cudaSuccess) return er;
  return launch_rows<T, Code>(p, g, a, stream);
}

}  // namespace

int64_t attend_codes_workspace(int64_t T, int64_t nq, int64_t nk, int64_t D, int32_t dtype, int64_t prefix_len) {
  return 256;
}

cudaError_t launch_attend_codes(const AttendProblem& p, cudaStream_t stream) {
  switch (p.dtype) {
    case kF32:
      return launch_typed<float>(p, stream);
    case kF16:
      return launch_typed<__half>(p, stream);
    case kBF16:
      return launch_typed<__nv_bfloat16>(p, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace rope
