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
// workspace bytes that a call of these bounds needs; that every call up to these bounds needs
size_t kv8_attention_need(const Kv8View& c, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix);
size_t kv8_attention_workspace(const Kv8View& c, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix);
cudaError_t launch_kv8_attention(const Kv8View& c, const CUtensorMap& map, const spec_kv8_attention_args& a, const int* clusters, cudaStream_t s);

// rows > 16 per kv head: the tensor-core kernel (prefixes up to kKv8TcMaxChunks * kKv8TcMaxKeys; no workspace)
// clusters[n]: how many clusters of n CTAs run at once, n = 1 .. kKv8TcMaxChunks
cudaError_t kv8_tree_configure(int sm_count, int* clusters);
cudaError_t launch_kv8_tree(const Kv8View& c, const spec_kv8_attention_args& a, const int* clusters, cudaStream_t s);

}  // namespace spec
