// Quantising store of the 8-bit paged cache.
//
// A run is a stretch of rows whose slots follow each other inside one page.  For
// each run, kv head and plane: a = max |x| over the run's finite values, and
// e = the least whole number of [-60, 120] with a <= 448 * 2^e (448 is e4m3's
// largest value).  A run that starts at place o > 0 keeps at least the page's
// exponent; if it grows, the o tokens before the run are multiplied by
// 2^(e_old - e) and rounded again (exact unless they become subnormal).  The
// run's values are stored as e4m3(x * 2^-e), rounded to nearest even, infinities
// saturated to 448: half a step of e4m3, at most 2^-4 of a value.  A NaN makes its
// page's exponent byte 255, which reads as NaN and stays until the page is opened
// anew (place 0): the codes themselves need no NaN, and their readers no test.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8.h"

namespace spec {

namespace {

constexpr int kThreads = 128;         // 64 for K, 64 for V
constexpr int kLanes = 16;            // threads of a row: 8 values each
constexpr int kRowsAtOnce = 64 / kLanes;

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]

// the least e of the cache's range with a <= 448 * 2^e; a finite, not negative
__device__ __forceinline__ int exponent_of(float a) {
  const int bits = __float_as_int(a);
  // a = m * 2^x with m in [0.5, 1); 448 = 0.875 * 2^9
  const int x = (bits >> 23) - 126;
  const int e = x - 9 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(kKv8ExpMax, max(kKv8ExpMin, e));
}

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(h[i]);
}

// eight values times `s` as e4m3, round to nearest even, saturating
__device__ __forceinline__ uint2 encode8(const float* v, float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * s, v[2 * i + 1] * s), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(Kv8View c, spec_kv8_append_args a, int rows_per_cta) {
  __shared__ int run_len;
  __shared__ float part[4];
  const int tid = threadIdx.x, plane = tid >> 6, t = tid & 63;
  const int head = blockIdx.y;
  const int sub = t / kLanes, col = (t % kLanes) * 8;
  const T* src = reinterpret_cast<const T*>(plane ? a.v : a.k) + (plane ? a.v_head_stride : a.k_head_stride) * head + col;
  const int64_t row_stride = plane ? a.v_row_stride : a.k_row_stride;
  const int limit = c.n_pages << c.page_log2;
  // a row's slot, -1 where it stores nothing
  auto slot_of = [&](int i) {
    const int s = a.slots[i];
    const int r = a.src_rows ? a.src_rows[i] : i;
    return (s >= 0 && s < limit && r >= 0 && r < a.n_src) ? s : -1;
  };
  const int r0 = blockIdx.x * rows_per_cta;
  const int r1 = min(a.rows, r0 + rows_per_cta);
  int i = r0;
  while (i < r1) {
    // (uniform over the CTA)
    const int slot = slot_of(i);
    const int place = slot & (c.page - 1);
    if (slot < 0 || (i > 0 && place > 0 && slot_of(i - 1) == slot - 1)) {
      ++i;
      continue;
    }
    // the run's length
    if (tid == 0) run_len = c.page - place;
    __syncthreads();
    if (place + tid < c.page && (i + tid >= a.rows || slot_of(i + tid) != slot + tid)) atomicMin(&run_len, tid);
    __syncthreads();
    const int n = run_len;
    const int pg = slot >> c.page_log2;
    float amax = 0.f;
    bool nan = false;
    for (int r = sub; r < n; r += kRowsAtOnce) {
      float v[8];
      load8(src + row_stride * (a.src_rows ? a.src_rows[i + r] : i + r), v);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float m = fabsf(v[q]);
        amax = fmaxf(amax, m < INFINITY ? m : 0.f);
        nan |= m != m;
      }
    }
    amax = __any_sync(0xffffffffu, nan) ? NAN : warp_max(amax);
    if ((tid & 31) == 0) part[tid >> 5] = amax;
    __syncthreads();
    nan = isnan(part[2 * plane]) || isnan(part[2 * plane + 1]);
    amax = fmaxf(part[2 * plane], part[2 * plane + 1]);
    if (!(amax >= 0.f)) amax = 0.f;  // both NaN
    uint8_t* ep = c.exps[plane] + (size_t)pg * c.hkv + head;
    uint8_t* base = c.codes[plane] + (((size_t)pg * c.hkv + head) << c.page_log2) * kKv8Hd + col;
    int e = exponent_of(amax);
    if (place > 0) {
      const int old = (int)*ep - 127;
      nan |= old == 128;
      e = nan ? e : max(e, old);
      if (!nan && e > old) {
        const float f = pow2f(max(old - e, -126));
        for (int r = sub; r < place; r += kRowsAtOnce) {
          uint2* p = reinterpret_cast<uint2*>(base + (size_t)r * kKv8Hd);
          const uint2 was = *p;
          const __nv_fp8_e4m3* h = reinterpret_cast<const __nv_fp8_e4m3*>(&was);
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = (float)h[q];
          *p = encode8(v, f);
        }
      }
    }
    const float f = pow2f(-e);
    for (int r = sub; r < n; r += kRowsAtOnce) {
      float v[8];
      load8(src + row_stride * (a.src_rows ? a.src_rows[i + r] : i + r), v);
      *reinterpret_cast<uint2*>(base + (size_t)(place + r) * kKv8Hd) = encode8(v, f);
    }
    __syncthreads();  // every thread has read the exponent, `part` and `run_len`
    if (t == 0) *ep = (uint8_t)(nan ? 255 : e + 127);
    i += n;
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8View& c, const spec_kv8_append_args& a, int sm_count, cudaStream_t s) {
  int per = (int)((long long)a.rows * c.hkv / (16 * sm_count));
  per = per < 1 ? 1 : per > c.page ? c.page : per;
  const dim3 grid((a.rows + per - 1) / per, c.hkv);
  if (a.dtype == SPEC_DTYPE_F32) kv8_append_kernel<float><<<grid, kThreads, 0, s>>>(c, a, per);
  else if (a.dtype == SPEC_DTYPE_BF16) kv8_append_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(c, a, per);
  else kv8_append_kernel<__half><<<grid, kThreads, 0, s>>>(c, a, per);
  return cudaGetLastError();
}

}  // namespace spec
