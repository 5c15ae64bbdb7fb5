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
//
// Prompts in pages of up to 64 tokens read and write each byte once: 195 MB of bf16 rows and their codes take 40 us,
// 4.9 TB/s, three quarters of the measured copy rate.  A page's rows wait in registers for its largest value, so that the reads in flight are what four
// CTAs of 256 threads per SM hold (three: 63 us before the instructions were cut; shared memory in place of registers,
// six CTAs: 43 where registers took 42); issue slots are busy two thirds of the time, for the magnitudes, the products
// and the conversions.  Runs of more rows than the registers hold are read a second time, mostly from L2: 64 rows here, so
// all of a page of 128 (31.7k whole pages of bf16: 41.8 us, 36.6 in pages of 64; fp32 67.0 and 59.7), 16 rows in the CTAs
// of decoding steps.  Pages of 16 make CTAs of 16 rows, whose loads do not fill an SM (88.5 us, fp32 150).  Tried without gain: heads of a row side by side in the grid, prefetch into L2 while the slots
// are read, loads that bypass L1, CTAs of 512 threads (51 us).  Steps of a few rows are bound by the chain of loads:
// slots, rows and the page's exponent (64 rows: 3.4 us; 317 gathered rows of 64 sequences in fp32: 6.3 us); where a page's
// scale grows, the codes before the run too (64 rows, all of whose pages grow: 8.0 us, 3.1 where none does).
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8.h"

namespace spec {

namespace {

constexpr int kLanes = 16;  // threads of a row: 8 values each

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]

// the least e of the cache's range with a <= 448 * 2^e; a finite, not negative
__device__ __forceinline__ int exponent_of(float a) {
  const int bits = __float_as_int(a);
  // a = m * 2^x with m in [0.5, 1); 448 = 0.875 * 2^9
  const int x = (bits >> 23) - 126;
  const int e = x - 9 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(kKv8ExpMax, max(kKv8ExpMin, e));
}

// eight values as they lie in memory
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const T* h = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(h[i]);
  }
};

// The largest magnitude of the values seen, as the bits of T without the sign (which are in the order of the
// magnitudes, infinity and NaN above all others).
template <typename T>
struct Top {
  uint32_t m = 0;  // a pair of 16-bit values
  __device__ __forceinline__ void see(const Eight<T>& x) {
    const uint4& w = x.w[0];
    m = max2(max2(m, w.x), max2(w.y, max2(w.z, w.w)));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    using T2 = std::conditional_t<__is_same(T, __half), __half2, __nv_bfloat162>;
    const T2 c = __hmax2_nan(__habs2(reinterpret_cast<const T2&>(a)), __habs2(reinterpret_cast<const T2&>(b)));
    return reinterpret_cast<const uint32_t&>(c);
  }
  __device__ __forceinline__ uint32_t bits() const { return max(m & 0x7fffu, m >> 16 & 0x7fffu); }
  static __device__ __forceinline__ bool finite(uint32_t b) { return b < (__is_same(T, __half) ? 0x7c00u : 0x7f80u); }
  static __device__ __forceinline__ float value(uint32_t b) {
    const uint16_t h = (uint16_t)b;
    return to_f32<T>(reinterpret_cast<const T&>(h));
  }
};
template <>
struct Top<float> {
  uint32_t m = 0;
  __device__ __forceinline__ void see(const Eight<float>& x) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
  }
  __device__ __forceinline__ uint32_t bits() const { return m; }
  static __device__ __forceinline__ bool finite(uint32_t b) { return b < 0x7f800000u; }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b); }
};

// four values as e4m3, round to nearest even, saturating
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}
// eight values times s, a power of two of 2^-120 .. 2^60, as e4m3
template <typename T>
__device__ __forceinline__ uint2 encode8(const Eight<T>& x, float s) {
  float v[8];
  if constexpr (__is_same(T, __nv_bfloat16)) {
    // (both factors are bf16, the product is rounded once, to 32 bits: one instruction instead of two)
    const uint16_t h = (uint16_t)(__float_as_uint(s) >> 16);
    const uint32_t w[4] = {x.w[0].x, x.w[0].y, x.w[0].z, x.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(v[2 * i]) : "h"((uint16_t)w[i]), "h"(h), "f"(-0.f));
      asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(v[2 * i + 1]) : "h"((uint16_t)(w[i] >> 16)), "h"(h), "f"(-0.f));
    }
  } else {
    x.get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f2_unpack(f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), f2_pack(s, s)), v[2 * i], v[2 * i + 1]);
  }
  return make_uint2(encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7]));
}

// THREADS: half of them for K, half for V.  HELD rows per thread stay in registers, so that runs of
// HELD * THREADS / 32 rows are read once.  CTAS: on an SM at a time.
template <typename T, int THREADS, int HELD, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) kv8_append_kernel(Kv8View c, spec_kv8_append_args a, int rows_per_cta) {
  constexpr int kPlane = THREADS / 2, kRowsAtOnce = kPlane / kLanes, kWarps = kPlane / 32;
  __shared__ uint32_t s_break[9];  // rows r0 .. r0 + 255: does a run end before this row?
  __shared__ int s_slot[256], s_src[256];
  __shared__ float part[2 * kWarps];
  __shared__ int part_nan[2 * kWarps];
  const int tid = threadIdx.x, plane = tid / kPlane, t = tid % kPlane;
  const int tile = blockIdx.x, head = blockIdx.y;
  const int sub = t / kLanes, col = (t % kLanes) * 8;
  const T* src = reinterpret_cast<const T*>(plane ? a.v : a.k) + (plane ? a.v_head_stride : a.k_head_stride) * head + col;
  const int64_t row_stride = plane ? a.v_row_stride : a.k_row_stride;
  const int limit = c.n_pages << c.page_log2;
  const int r0 = tile * rows_per_cta;
  // The runs that start in rows r0 .. r0 + rows_per_cta - 1 (at most a page) are this CTA's; the last of them ends
  // within a page from there.  A row that stores nothing has slot -1.
  auto slot_of = [&](int j, int& r) {
    const int s = a.slots[j];
    r = a.src_rows ? a.src_rows[j] : j;
    return (s >= 0 && s < limit && r >= 0 && r < a.n_src) ? s : -1;
  };
  // CTAs of a few rows mostly have no run that starts in theirs
  if (THREADS == 128) {
    bool starts = false;
    const int i = r0 + tid;
    if (tid < rows_per_cta && i < a.rows) {
      int none;
      const int slot = slot_of(i, none);
      starts = slot >= 0 && ((slot & (c.page - 1)) == 0 || i == 0 || slot_of(i - 1, none) != slot - 1);
    }
    if (!__syncthreads_or(starts)) return;
  }
  for (int w = tid; w < ((rows_per_cta + c.page + 31) & ~31); w += THREADS) {
    const int i = r0 + w;
    int slot = -1, row = 0, before = -1, none;
    if (i < a.rows) slot = slot_of(i, row);
    if (i > 0 && i <= a.rows) before = slot_of(i - 1, none);
    s_slot[w] = slot;
    s_src[w] = row;
    const bool brk = slot < 0 || before < 0 || slot != before + 1 || (slot & (c.page - 1)) == 0;
    const uint32_t m = __ballot_sync(0xffffffffu, brk);
    if ((tid & 31) == 0) s_break[w >> 5] = m;
  }
  if (tid == 0) s_break[(rows_per_cta + c.page + 31) >> 5] = 1u;
  __syncthreads();
  for (int i = 0; i < rows_per_cta;) {
    // (uniform over the CTA) the next break, from i on
    const uint32_t w = s_break[i >> 5] >> (i & 31);
    if (w == 0) {
      i = (i | 31) + 1;
      continue;
    }
    i += __ffs(w) - 1;
    if (i >= rows_per_cta) break;
    const int slot = s_slot[i];
    if (slot < 0) {
      ++i;
      continue;
    }
    int end = i + 1;
    while (!(s_break[end >> 5] >> (end & 31))) end = (end | 31) + 1;
    end += __ffs(s_break[end >> 5] >> (end & 31)) - 1;
    const int n = end - i, place = slot & (c.page - 1), pg = slot >> c.page_log2;
    uint8_t* const ep = c.exps[plane] + (size_t)pg * c.hkv + head;
    uint8_t* const base = c.codes[plane] + (((size_t)pg * c.hkv + head) << c.page_log2) * kKv8Hd + col;
    const int old_byte = place > 0 ? (int)*ep : 0;
    Eight<T> held[HELD];
    auto load = [&](int r0) {  // rows r0 .. of the run, HELD per thread in flight
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (r0 + sub + k * kRowsAtOnce < n) held[k].load(src + row_stride * s_src[i + r0 + sub + k * kRowsAtOnce]);
    };
    float amax = 0.f;
    bool nan = false;
    auto look = [&](const Eight<T>& x) {
      float v[8];
      x.get(v);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float m = fabsf(v[q]);
        amax = fmaxf(amax, m < INFINITY ? m : 0.f);
        nan |= m != m;
      }
    };
    constexpr int kBatch = HELD * kRowsAtOnce;
    for (int r = 0; r < n; r += kBatch) {
      load(r);
      Top<T> top;
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (r + sub + k * kRowsAtOnce < n) top.see(held[k]);
      const uint32_t bits = top.bits();
      if (Top<T>::finite(bits)) {
        amax = fmaxf(amax, Top<T>::value(bits));
      } else {  // (rare) value by value
#pragma unroll
        for (int k = 0; k < HELD; ++k)
          if (r + sub + k * kRowsAtOnce < n) look(held[k]);
      }
    }
    amax = warp_max(amax);
    nan = __any_sync(0xffffffffu, nan);
    if ((tid & 31) == 0) part[tid >> 5] = amax, part_nan[tid >> 5] = nan;
    __syncthreads();  // (also: every thread has read the page's exponent)
    amax = 0.f;
    nan = false;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      amax = fmaxf(amax, part[kWarps * plane + w]);
      nan |= part_nan[kWarps * plane + w] != 0;
    }
    int e = exponent_of(amax);
    if (place > 0) {
      const int old = old_byte - 127;
      nan |= old_byte == 255;
      e = nan ? e : max(e, old);
      if (!nan && e > old) {
        const float f = pow2f(max(old - e, -126));
        for (int r = sub; r < place; r += kRowsAtOnce) {
          uint2* p = reinterpret_cast<uint2*>(base + (size_t)r * kKv8Hd);
          const uint2 was = *p;
          const __nv_fp8_e4m3* h = reinterpret_cast<const __nv_fp8_e4m3*>(&was);
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = (float)h[q] * f;
          *p = make_uint2(encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7]));
        }
      }
    }
    const float f = pow2f(-e);
    uint8_t* const to = base + (size_t)place * kKv8Hd;
    auto put = [&](int r, const Eight<T>& x) { *reinterpret_cast<uint2*>(to + r * kKv8Hd) = encode8(x, f); };
    for (int r = 0; r < n; r += kBatch) {
      if (n > kBatch) load(r);  // (a run of one batch is still there)
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (r + sub + k * kRowsAtOnce < n) put(r + sub + k * kRowsAtOnce, held[k]);
    }
    if (t == 0) *ep = (uint8_t)(nan ? 255 : e + 127);
    i = end;
    __syncthreads();  // `part` may be written again
  }
}

template <typename T>
void launch_append(const Kv8View& c, const spec_kv8_append_args& a, int per, cudaStream_t s) {
  const dim3 grid((a.rows + per - 1) / per, c.hkv);
  if (per <= 4) kv8_append_kernel<T, 128, 4, 1><<<grid, 128, 0, s>>>(c, a, per);
  else kv8_append_kernel<T, 256, 8, sizeof(T) == 2 ? 4 : 2><<<grid, 256, 0, s>>>(c, a, per);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8View& c, const spec_kv8_append_args& a, int sm_count, cudaStream_t s) {
  // A sixteenth of an SM's share of the rows per CTA, at most a page: a CTA's runs are stored one after the other.
  // Up to four rows (decoding steps, accepted rows) CTAs have 128 threads (64 rows of bf16 and 8 heads: 3.3 us; 5.3
  // with 256 threads), for prompts 256 (31.7k such rows, 195 MB: 40 us, 4.9 TB/s; 84 with 128).
  int per = (int)((long long)a.rows * c.hkv / (16 * sm_count));
  per = per < 1 ? 1 : per > c.page ? c.page : per;
  if (a.dtype == SPEC_DTYPE_F32) launch_append<float>(c, a, per, s);
  else if (a.dtype == SPEC_DTYPE_BF16) launch_append<__nv_bfloat16>(c, a, per, s);
  else launch_append<__half>(c, a, per, s);
  return cudaGetLastError();
}

}  // namespace spec
