// Launches of the decode kernel with modified scores (decode_kernel.cuh, MOD):
// capped by a tanh, biased by distance, visible from a first token on, and
// with rotary positions applied to the query and the new key. A kernel of its
// own so that the plain decode carries none of it.
#include "decode_kernel.cuh"

namespace pa {
namespace {

template <int D, int P, int KVT>
cudaError_t launch_t(const ScoredArgs &a, cudaStream_t stream) {
  return launch_cfg<Config<D, P, KVT, KVT != PA_KV_BF16 ? PA_DECODE_STAGES_U8 : PA_DECODE_STAGES_BF16,
                           true>>(a, stream);
}

}  // namespace

cudaError_t launch_decode_scored(int D, int P, int kv_dtype, const ScoredArgs &a,
                                 cudaStream_t stream) {
#define PA_L(D_, P_, K_) \
  if (D == D_ && P == P_ && kv_dtype == K_) return launch_t<D_, P_, K_>(a, stream)
  PA_L(128, 16, 0); PA_L(128, 32, 0); PA_L(64, 16, 0); PA_L(64, 32, 0);
  PA_L(128, 16, 1); PA_L(128, 32, 1); PA_L(64, 16, 1); PA_L(64, 32, 1);
  PA_L(128, 16, 2); PA_L(128, 32, 2); PA_L(64, 16, 2); PA_L(64, 32, 2);
  PA_L(128, 16, 3); PA_L(128, 32, 3); PA_L(64, 16, 3); PA_L(64, 32, 3);
#undef PA_L
  return cudaErrorInvalidValue;
}

}  // namespace pa
