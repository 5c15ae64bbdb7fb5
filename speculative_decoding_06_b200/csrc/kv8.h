// The 8-bit paged K/V cache: what its entry points and kernels share.  Not part
// of the public C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/spec.h"

namespace spec {

constexpr int kKv8Hd = 128;      // head dimension
constexpr int kKv8ExpMin = -60;  // exponents of the page scales (bias 127 in the byte)
constexpr int kKv8ExpMax = 120;
constexpr int kKv8MaxBatch = 8192;
constexpr int kKv8MaxSeqs = 65536;
constexpr int kKv8MaxGroup = 64;  // query heads per kv head
constexpr int kKv8MaxNodes = 128;
constexpr int kKv8MaxRows = 1 << 30;    // of an append, of a plan: numbered in 32 bits, a grid's stride beyond the last one
constexpr int kKv8MaxGroups = 1 << 30;  // row tiles of an attention call of few rows, numbered likewise
constexpr int kKv8TcMaxChunks = 8;     // CTAs of a cluster that share a sequence's prefix (tree kernel)
constexpr int kKv8TcMaxKeys = 49152;   // keys of one of them

// One layer's planes of the cache.
struct Kv8View {
  uint8_t* codes[2];  // K, V: [page id][kv head][token][128]
  uint8_t* exps[2];   // K, V: [page id][kv head]
  int n_pages, page, page_log2, hkv;
  int row0[2];        // first row (of 128 codes) of each plane in the whole cache
};

cudaError_t kv8_plan_configure();
cudaError_t launch_kv8_plan(const spec_kv8_plan_args& a, int page_log2, int n_pages, cudaStream_t s);
cudaError_t launch_kv8_append(const Kv8View& c, const spec_kv8_append_args& a, int sm_count, cudaStream_t s);
cudaError_t kv8_attention_configure(int sm_count, int* clusters);
// workspace bytes that a call of these bounds needs (0: more than kKv8MaxGroups row tiles); that every call up to these
// bounds needs
size_t kv8_attention_need(const Kv8View& c, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix);
size_t kv8_attention_workspace(const Kv8View& c, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix);
cudaError_t launch_kv8_attention(const Kv8View& c, const CUtensorMap& map, const spec_kv8_attention_args& a, const int* clusters, cudaStream_t s);

// rows > 16 per kv head: the tensor-core kernel (prefixes up to kKv8TcMaxChunks * kKv8TcMaxKeys; no workspace)
// clusters[n]: how many clusters of n CTAs run at once, n = 1 .. kKv8TcMaxChunks
cudaError_t kv8_tree_configure(int sm_count, int* clusters);
cudaError_t launch_kv8_tree(const Kv8View& c, const spec_kv8_attention_args& a, const int* clusters, cudaStream_t s);

#ifdef __CUDACC__
// m + log2 l for a normal l > 0: l's exponent is added to m, which is of its size and the other sign, so that what rounds
// is of the result's size
__device__ __forceinline__ float kv8_log2_sum(float m, float l) {
  const int bits = __float_as_int(l);
  const float mantissa = __int_as_float((bits & 0x7fffff) | 0x3f800000);
  return l < INFINITY ? (m + (float)((bits >> 23) - 127)) + log2f(mantissa) : m + l;
}
// Heads head0 .. head0 + G - 1 of rows lo .. hi - 1 of out and lse (either may be null): NaN, or those of rows that see
// nothing.  (Kept out of the kernels: what they seldom run shall not lie among what they always run.)
inline __device__ __noinline__ void kv8_fill(uint16_t* out, int64_t row_stride, float* lse, int n_q_heads, int head0, int G,
                                             int lo, int hi, bool nan) {
  const uint32_t w = nan ? 0x7fff7fffu : 0u;  // (NaN in bf16 and in fp16)
  for (int64_t row = (int64_t)lo + (threadIdx.x >> 4); row < hi; row += blockDim.x >> 4)  // 16 threads each
    for (int head = head0; head < head0 + G; ++head) {
      const int at = threadIdx.x & 15;
      if (out) *reinterpret_cast<uint4*>(out + row_stride * row + (int64_t)head * kKv8Hd + 8 * at) = make_uint4(w, w, w, w);
      if (lse && at == 0) lse[row * n_q_heads + head] = __int_as_float(nan ? 0x7fffffff : 0xff800000);
    }
}
// What `fill` asks for of rows that no row tile writes, by all threads of one CTA per entry and kv head: the entry's own
// ones, as NaN, where it is out of range; the rows before the first entry and behind the last one as if they saw nothing.
__device__ __forceinline__ void kv8_fill_rows(const spec_kv8_attention_args& a, int b, int kvh, int G) {
  const int first = a.offsets[b], end = a.offsets[b + 1], n = end - first, seq = a.seq_ids ? a.seq_ids[b] : b;
  const int P = seq >= 0 && seq < a.n_seqs ? a.lengths[seq] : -1;
  const bool bad = P < 0 || P > a.max_prefix || first < 0 || n < 1 || n > a.max_nodes || n > a.rows - first;
  if (!bad && b > 0 && b < a.batch - 1) return;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {  // before the first entry, the entry, behind the last
    const int lo = part == 0 ? 0 : part == 1 ? first : end, hi = part == 0 ? first : part == 1 ? end : a.rows;
    if (part == 0 ? b == 0 : part == 1 ? bad : b == a.batch - 1)
      kv8_fill(a.fill & SPEC_KV8_FILL_OUT ? static_cast<uint16_t*>(a.out) : nullptr, a.out_row_stride,
               a.fill & SPEC_KV8_FILL_LSE ? a.lse : nullptr, a.n_q_heads, kvh * G, G, max(0, lo), min(a.rows, hi), part == 1);
  }
}
#endif

}  // namespace spec
