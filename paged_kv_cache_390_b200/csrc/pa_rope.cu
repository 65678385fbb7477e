// pa_rope.cu -- rotary positions with several axes, fused with the paged cache
// write (pa_rope_and_cache) for sm_100a.
//
// Pair i of a row's first rotary_dim elements turns by
//   angle = positions[axis(i)][token] * inv_freq[i]:  (a, b) -> (a cos - b sin, a sin + b cos)
// with its own position axis (time, height, width), so text (all axes equal) and
// images (a grid) take the same kernel.  Query rows go to `out`; key rows go, turned,
// and value rows, as they are, to the token's slot of the paged cache, quantised there
// as pa_write.cuh describes (from the fp32 turned value: one rounding).
//
// The angle is taken in 64 bits and its whole turns dropped there (at position 2^20 a
// 32-bit angle is off by up to 0.06); sine and cosine of the rest are 32-bit.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tile.cuh"
#include "pa_write.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;

template <typename ST>
__device__ __forceinline__ ST from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Bound: the rows' bytes, each read and written once.  8191 tokens x 80 rows x 128 bf16
// (336 MB): 59.2 us, 5.7 TB/s, with ten CTAs an SM (48 registers; nine without the bound 61.4,
// twelve at 40 registers 61.6; fp32 rows 3.6 us without, 4.0 with it).  Two or three rows' loads in flight per lane, or the first
// ones before the sine and cosine, were slower (63 to 83 us: fewer CTAs fit an SM).
// One CTA per (token, slice of its rows).  A row of D elements is D / (2 VE) lanes'
// work; lane j of a row holds pairs [j VE, (j + 1) VE): its two 16-byte vectors are the
// halves' vectors j (halves form) or the row's vectors 2j and 2j + 1 (side by side).
template <typename ST, int MODE, int D>
__global__ void __launch_bounds__(kThreads, sizeof(ST) == 2 && MODE == kWriteCopy ? 10 : 1)
    rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int VE = 16 / static_cast<int>(sizeof(ST));
  constexpr int LPR = D / (2 * VE);            // lanes per row: 4 (16-bit, D 64) .. 16 (fp32, D 128)
  constexpr int RPP = kThreads / LPR;          // rows per pass
  struct alignas(16) Vec {
    ST v[VE];
  };
  __shared__ float2 turn[D / 2];               // (cos, sin) of the token's pairs

  griddep_launch_dependents();
  griddep_wait();
  const int token = blockIdx.x;
  const int half = a.rotary_dim / 2;
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const int ax = a.pair_axis[i];
    float2 cs = make_float2(1.f, 0.f);         // an axis outside the positions: no turn
    if (ax >= 0 && ax < a.num_axes) {
      const double x = static_cast<double>(a.positions[static_cast<size_t>(ax) * a.num_tokens + token]) *
                       a.inv_freq[i];
      const double u = x * 0.15915494309189535;                  // turns: x / (2 pi)
      sincospif(static_cast<float>(2.0 * (u - rint(u))), &cs.y, &cs.x);
    }
    turn[i] = cs;
  }
  __syncthreads();

  const int j = threadIdx.x % LPR;
  const bool rot = j * VE < half;
  int e0, e1;                                  // first elements of the lane's two vectors
  if (a.interleaved || !rot) {
    e0 = 2 * j * VE;
    e1 = e0 + VE;
  } else {
    e0 = j * VE;
    e1 = e0 + half;
  }
  float2 cs[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) cs[e] = rot ? turn[j * VE + e] : make_float2(1.f, 0.f);

  const int H = a.num_heads, Hkv = a.num_kv_heads;
  const int nrows = H + 2 * Hkv;
  const int per = (nrows + gridDim.y - 1) / gridDim.y;
  const int row_end = min(nrows, static_cast<int>(blockIdx.y + 1) * per);
  const int64_t slot = a.slots[token];
  const int64_t pool = static_cast<int64_t>(a.num_blocks) * a.block_size;
  const bool write = slot >= 0 && slot < pool;
  if (slot >= pool && threadIdx.x == 0 && blockIdx.y == 0 && a.err_flag)
    report_error(a.err_flag, kErrSlot);

  // the lanes of one row leave the loop together (a row's lanes are consecutive and
  // LPR divides 32), so the shuffles below run over whole rows
  for (int row = blockIdx.y * per + threadIdx.x / LPR; row < row_end; row += RPP) {
    const bool is_q = row < H, is_v = row >= H + Hkv;
    if (!is_q && !write) continue;
    const int head = is_q ? row : (is_v ? row - H - Hkv : row - H);
    const ST* src = static_cast<const ST*>(is_q ? a.q : (is_v ? a.v : a.k)) +
                    static_cast<size_t>(token) * (is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride)) +
                    static_cast<size_t>(head) * D;
    Vec w0 = *reinterpret_cast<const Vec*>(src + e0);
    Vec w1 = *reinterpret_cast<const Vec*>(src + e1);
    float x[2 * VE];                           // the lane's values, w0's then w1's
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      x[e] = to_f32<ST>(w0.v[e]);
      x[VE + e] = to_f32<ST>(w1.v[e]);
    }
    if (rot && !is_v) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float p = x[2 * e], q = x[2 * e + 1];
          x[2 * e] = p * cs[e].x - q * cs[e].y;
          x[2 * e + 1] = p * cs[e].y + q * cs[e].x;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float p = x[e], q = x[VE + e];
          x[e] = p * cs[e].x - q * cs[e].y;
          x[VE + e] = p * cs[e].y + q * cs[e].x;
        }
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        w0.v[e] = from_f32<ST>(x[e]);
        w1.v[e] = from_f32<ST>(x[VE + e]);
      }
    }
    if (is_q || MODE == kWriteCopy) {
      ST* dst = is_q ? static_cast<ST*>(a.out) + (static_cast<size_t>(token) * H + head) * D
                     : static_cast<ST*>(is_v ? a.v_cache : a.k_cache) +
                           (static_cast<size_t>(slot) * Hkv + head) * D;
      *reinterpret_cast<Vec*>(dst + e0) = w0;
      *reinterpret_cast<Vec*>(dst + e1) = w1;
      continue;
    }
    if constexpr (MODE != kWriteCopy) {
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * VE; ++e) amax = fmaxf(amax, fabsf(x[e]));
      const uint32_t lanes = (LPR == 32 ? ~0u : ((1u << LPR) - 1u)) << ((threadIdx.x & 31) / LPR * LPR);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
      const float s = __fdiv_rn(amax, MODE == kWriteInt8 ? 127.0f : 448.0f);
      uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                     (static_cast<size_t>(slot) * Hkv + head) * D;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        struct alignas(VE) Codes {
          uint8_t b[VE];
        } codes;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          codes.b[e] = s != 0.f ? static_cast<uint8_t>(quant_code<MODE>(x[w * VE + e], s)) : 0;
        *reinterpret_cast<Codes*>(dst + (w ? e1 : e0)) = codes;
      }
      if (j == 0)
        (is_v ? a.v_scale : a.k_scale)[(static_cast<size_t>(slot / a.block_size) * Hkv + head) *
                                           a.block_size + slot % a.block_size] = s;
    }
  }
}

template <typename ST, int MODE, int D>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t s) {
  // few tokens: a token's rows over several CTAs, until every SM has one (32 tokens of
  // 80 rows: 2.4 us against 3.8 with a CTA each)
  constexpr int kRowsPerPass = kThreads / (D / (32 / static_cast<int>(sizeof(ST))));
  const long long passes = (a.num_heads + 2LL * a.num_kv_heads + kRowsPerPass - 1) / kRowsPerPass;
  int sms = 0;
  const cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  long long slices = (sms + a.num_tokens - 1) / a.num_tokens;
  if (slices > passes) slices = passes;
  return launch_kernel(rope_kernel<ST, MODE, D>, dim3(a.num_tokens, static_cast<unsigned>(slices)),
                       dim3(kThreads), 0, s, pdl_mode() != 0, a);
}

template <typename ST>
cudaError_t launch_src(const RopeArgs& a, int cache_dtype, int D, cudaStream_t s) {
  const bool wide = D == 128;
  if (cache_dtype == PA_INT8)
    return wide ? launch_t<ST, kWriteInt8, 128>(a, s) : launch_t<ST, kWriteInt8, 64>(a, s);
  if (cache_dtype == PA_FP8E4M3)
    return wide ? launch_t<ST, kWriteFp8, 128>(a, s) : launch_t<ST, kWriteFp8, 64>(a, s);
  return wide ? launch_t<ST, kWriteCopy, 128>(a, s) : launch_t<ST, kWriteCopy, 64>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int src_dtype, int cache_dtype, int head_dim,
                        cudaStream_t s) {
  switch (src_dtype) {
    case PA_F32: return launch_src<float>(a, cache_dtype, head_dim, s);
    case PA_F16: return launch_src<__half>(a, cache_dtype, head_dim, s);
    case PA_BF16: return launch_src<__nv_bfloat16>(a, cache_dtype, head_dim, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
