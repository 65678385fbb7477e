// pa_fused.cu -- pa_decode_fused: the workspace of the persistent decode and its dispatch
// (the kernel is in pa_fused_kernel.cuh).
#include "pa_fused_kernel.cuh"

namespace pa {

size_t fused_workspace_bytes(int num_seqs, int num_kv_heads, int head_dim, int num_sms) {
  const size_t warps = static_cast<size_t>(num_sms) * kFusedMaxCtasPerSm * kFusedWarps;
  return fused_counter_bytes(num_seqs, num_kv_heads) +
         2 * warps * fused_record_floats(head_dim) * sizeof(float);
}

namespace {

template <typename QT, int KIND>
cudaError_t fused_shape(const FusedArgs& a, int D, int BS, size_t ws, cudaStream_t s) {
#define PA_CASE(DD, BB) \
  if (D == DD && BS == BB) return launch_fused_t<QT, KIND, DD, BB, false>(a, ws, s);
  PA_CASE(128, 16)
  PA_CASE(128, 8)
  PA_CASE(128, 32)
  PA_CASE(64, 16)
  PA_CASE(64, 8)
  PA_CASE(64, 32)
#undef PA_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_fused(const FusedArgs& a, int q_dtype, int cache_dtype, int head_dim,
                         int block_size, size_t workspace_bytes, cudaStream_t s) {
  const bool qh = q_dtype == PA_F16;
  switch (cache_dtype) {
    case PA_F16: return fused_shape<__half, kKind16>(a, head_dim, block_size, workspace_bytes, s);
    case PA_BF16:
      return fused_shape<__nv_bfloat16, kKind16>(a, head_dim, block_size, workspace_bytes, s);
    case PA_INT8:
      return qh ? fused_shape<__half, kKindI8>(a, head_dim, block_size, workspace_bytes, s)
                : fused_shape<__nv_bfloat16, kKindI8>(a, head_dim, block_size, workspace_bytes, s);
    case PA_FP8E4M3:
      return qh ? fused_shape<__half, kKindE4M3>(a, head_dim, block_size, workspace_bytes, s)
                : fused_shape<__nv_bfloat16, kKindE4M3>(a, head_dim, block_size, workspace_bytes,
                                                        s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
