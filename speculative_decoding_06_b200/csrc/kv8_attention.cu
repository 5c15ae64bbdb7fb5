// Attention over the 8-bit paged cache: the plain kernel, one warp per (row,
// query head), a key at a time with the online softmax in 32 bits.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8.h"

namespace spec {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float4 codes4(const uint8_t* p, float s) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  const __nv_fp8_e4m3* h = reinterpret_cast<const __nv_fp8_e4m3*>(&w);
  return make_float4((float)h[0] * s, (float)h[1] * s, (float)h[2] * s, (float)h[3] * s);
}
template <typename T>
__device__ __forceinline__ float4 rows4(const T* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const T* h = reinterpret_cast<const T*>(&w);
  return make_float4(to_f32<T>(h[0]), to_f32<T>(h[1]), to_f32<T>(h[2]), to_f32<T>(h[3]));
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) kv8_attention_plain_kernel(Kv8View c, spec_kv8_attention_args a) {
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= a.rows * a.n_q_heads) return;
  const int row = unit / a.n_q_heads, qh = unit - row * a.n_q_heads;
  const int kvh = qh / (a.n_q_heads / c.hkv);
  int b = -1;
  for (int i = 0; i < a.batch; ++i)
    if (a.offsets[i] <= row && row < a.offsets[i + 1]) b = i;
  if (b < 0) return;
  const int first = a.offsets[b], n = a.offsets[b + 1] - first;
  const int seq = a.seq_ids ? a.seq_ids[b] : b;
  if (first < 0 || n > a.max_nodes || first + n > a.rows || seq < 0 || seq >= a.n_seqs) return;
  const int P = a.lengths[seq];
  if (P < 0 || P > a.max_prefix) return;
  const float4 q = rows4(reinterpret_cast<const T*>(a.q) + a.q_row_stride * row + a.q_head_stride * qh + 4 * lane);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto see = [&](float4 k, float4 v) {
    const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * a.scale;
    const float m2 = fmaxf(m, s);
    const float keep = m2 == m ? 1.f : expf(m - m2), p = expf(s - m2);
    m = m2;
    l = l * keep + p;
    o = make_float4(o.x * keep + p * v.x, o.y * keep + p * v.y, o.z * keep + p * v.z, o.w * keep + p * v.w);
  };
  for (int j = 0; j < P; ++j) {
    const int pg = a.tables[(size_t)seq * a.max_blocks + (j >> c.page_log2)];
    if (pg < 0 || pg >= c.n_pages) {
      see(make_float4(NAN, NAN, NAN, NAN), make_float4(NAN, NAN, NAN, NAN));
      continue;
    }
    const size_t ph = (size_t)pg * c.hkv + kvh;
    const size_t at = ((ph << c.page_log2) + (j & (c.page - 1))) * kKv8Hd + 4 * lane;
    see(codes4(c.codes[0] + at, exp2f((float)c.exps[0][ph] - 127.f)),
        codes4(c.codes[1] + at, exp2f((float)c.exps[1][ph] - 127.f)));
  }
  for (int j = row - first; a.k_new && j >= 0;) {
    see(rows4(reinterpret_cast<const T*>(a.k_new) + a.k_row_stride * (first + j) + a.k_head_stride * kvh + 4 * lane),
        rows4(reinterpret_cast<const T*>(a.v_new) + a.v_row_stride * (first + j) + a.v_head_stride * kvh + 4 * lane));
    const int up = a.parents ? a.parents[first + j] : j - 1;
    j = up < j ? up : -1;
  }
  const bool any = l > 0.f || isnan(l);
  const float inv = any ? 1.f / l : 0.f;
  T* out = reinterpret_cast<T*>(a.out) + a.out_row_stride * row + qh * kKv8Hd + 4 * lane;
  out[0] = from_f32<T>(o.x * inv);
  out[1] = from_f32<T>(o.y * inv);
  out[2] = from_f32<T>(o.z * inv);
  out[3] = from_f32<T>(o.w * inv);
  if (a.lse && lane == 0) a.lse[(size_t)row * a.n_q_heads + qh] = any ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8View& c, const spec_kv8_attention_args& a, int sm_count, cudaStream_t s) {
  (void)sm_count;
  const int grid = (a.rows * a.n_q_heads + kWarps - 1) / kWarps;
  if (a.dtype == SPEC_DTYPE_BF16) kv8_attention_plain_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, s>>>(c, a);
  else kv8_attention_plain_kernel<__half><<<grid, 32 * kWarps, 0, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace spec
