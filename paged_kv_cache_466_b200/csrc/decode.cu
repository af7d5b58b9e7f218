// Launches of the plain decode kernel (decode_kernel.cuh).
#include "decode_kernel.cuh"

namespace pa {
namespace {

template <int D, int P, int KVT>
cudaError_t launch_t(const DecodeArgs &a, cudaStream_t stream) {
  // A ragged batch launched longest unit first over several waves of CTAs
  // (ordered == 2) runs one CTA per (sequence, KV head), each streaming its
  // whole unit: there deeper rings (two CTAs per SM instead of three) pay.
  // Measured on the Llama-3-8B-shaped step: bf16 with three blocks per warp
  // instead of two 2-6 % faster (and 5 % slower on one wave of equal units,
  // the Llama-3-70B step, which keeps two); INT8 and FP8 with three pairs
  // instead of two 0.7-2.7 % faster on two B200s, 0.5 % slower on a third.
  // INT4 keeps its ring (four CTAs per SM fit only with it).
  if constexpr (KVT == PA_KV_BF16)
    if (a.ordered == 2) return launch_cfg<Config<D, P, KVT, PA_DECODE_STAGES_BF16_LPT>>(a, stream);
  if constexpr (KVT == PA_KV_U8_PER_TOKEN || KVT == PA_KV_FP8_PER_TOKEN)
    if (a.ordered == 2) return launch_cfg<Config<D, P, KVT, PA_DECODE_STAGES_U8_LPT>>(a, stream);
  return launch_cfg<Config<D, P, KVT>>(a, stream);
}

template <int D, int P, int KVT>
int ctas_per_sm_t() {
  using C = Config<D, P, KVT>;
  const size_t smem = C::SM::bytes(256);
  if (ensure_smem_attr<C>() != cudaSuccess) return 1;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, C::fn(), C::W * 32, smem) != cudaSuccess)
    return 1;
  return n > 0 ? n : 1;
}

}  // namespace

#define PA_DISPATCH(D_, P_, K_, CALL)                                  \
  if (D == D_ && P == P_ && kv_dtype == K_) return CALL<D_, P_, K_>

cudaError_t launch_decode(int D, int P, int kv_dtype, const DecodeArgs &a, cudaStream_t stream) {
#define PA_L(D_, P_, K_) PA_DISPATCH(D_, P_, K_, launch_t)(a, stream)
  PA_L(128, 16, 0); PA_L(128, 32, 0); PA_L(64, 16, 0); PA_L(64, 32, 0);
  PA_L(128, 16, 1); PA_L(128, 32, 1); PA_L(64, 16, 1); PA_L(64, 32, 1);
  PA_L(128, 16, 2); PA_L(128, 32, 2); PA_L(64, 16, 2); PA_L(64, 32, 2);
  PA_L(128, 16, 3); PA_L(128, 32, 3); PA_L(64, 16, 3); PA_L(64, 32, 3);
#undef PA_L
  return cudaErrorInvalidValue;
}

int decode_ctas_per_sm(int D, int P, int kv_dtype) {
#define PA_O(D_, P_, K_) PA_DISPATCH(D_, P_, K_, ctas_per_sm_t)()
  PA_O(128, 16, 0); PA_O(128, 32, 0); PA_O(64, 16, 0); PA_O(64, 32, 0);
  PA_O(128, 16, 1); PA_O(128, 32, 1); PA_O(64, 16, 1); PA_O(64, 32, 1);
  PA_O(128, 16, 2); PA_O(128, 32, 2); PA_O(64, 16, 2); PA_O(64, 32, 2);
  PA_O(128, 16, 3); PA_O(128, 32, 3); PA_O(64, 16, 3); PA_O(64, 32, 3);
#undef PA_O
  return 1;
}

}  // namespace pa
