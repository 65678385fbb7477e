// pa_prefill_masked.cu -- launches of pa_prefill_masked's tcgen05 form (the kernel is in
// pa_prefill_kernel.cuh).
#include "pa_prefill_kernel.cuh"

namespace pa {
namespace {

template <int BS>
cudaError_t kv_maps(CUtensorMap* mk, CUtensorMap* mv, const PrefillArgs& a) {
  cudaError_t e = make_cache_map<kKind16, kD, BS>(mk, a.k_cache, a.num_kv_heads, a.num_blocks);
  if (e != cudaSuccess) return e;
  return make_cache_map<kKind16, kD, BS>(mv, a.v_cache, a.num_kv_heads, a.num_blocks);
}

template <typename QT, int MOD>
cudaError_t launch_mod(const PrefillArgs& a, int max_query_len, cudaStream_t stream) {
  const int G = a.num_heads / a.num_kv_heads;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_q_map(&mq, a.q, a.total_q, a.num_heads, G);
  if (e != cudaSuccess) return e;
  switch (a.block_size) {
    case 8: e = kv_maps<8>(&mk, &mv, a); break;
    case 16: e = kv_maps<16>(&mk, &mv, a); break;
    default: e = kv_maps<32>(&mk, &mv, a); break;
  }
  if (e != cudaSuccess) return e;
  auto kern = prefill_kernel<QT, 0, MOD>;
  static int configured[64] = {0};
  e = opt_in_smem(reinterpret_cast<const void*>(kern), kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  const int rows_per_cta = kQTiles * (kRows / G);
  const int tiles = (max_query_len + rows_per_cta - 1) / rows_per_cta;
  const int ng = tiles < kTileGroup ? tiles : kTileGroup;
  const dim3 grid(ng * a.num_kv_heads, a.num_seqs, (tiles + ng - 1) / ng);
  return launch_kernel(kern, grid, dim3(prefill_threads<MOD>()), kSmemBytes, stream, pdl_mode() != 0, mq, mk, mv,
                       a);
}

template <typename QT>
cudaError_t launch_q(const PrefillArgs& a, int max_query_len, cudaStream_t s) {
  switch ((a.cap_in != 0.f ? 1 : 0) | (a.slopes ? 2 : 0)) {
    case 0: return launch_mod<QT, 0>(a, max_query_len, s);
    case 1: return launch_mod<QT, 1>(a, max_query_len, s);
    case 2: return launch_mod<QT, 2>(a, max_query_len, s);
  }
  return launch_mod<QT, 3>(a, max_query_len, s);
}

}  // namespace

cudaError_t launch_prefill_masked_tc(const PrefillArgs& a, int q_dtype, int max_query_len,
                                     cudaStream_t s) {
  return q_dtype == PA_BF16 ? launch_q<__nv_bfloat16>(a, max_query_len, s)
                            : launch_q<__half>(a, max_query_len, s);
}

}  // namespace pa
