// Page plan of the 8-bit paged cache: from every entry's length and change, the
// pages that it takes or gives back, the slots of its new rows and the new
// lengths.
//
// With T tokens per page, an entry that goes from P to N tokens has
// rows = max(0, N - P) new rows, takes max(0, ceil(N/T) - ceil(P/T)) pages and
// gives back max(0, ceil(P/T) - ceil(N/T)).  Exclusive prefix sums of the three
// over the batch give the first row, the first page of the ring and the first
// place behind its tail of every entry, so pages are handed out in entry order
// and no two threads meet: no atomics, the same result every time.  New row i of
// entry b (found by binary search in the row sums) sits at token P_b + i - off_b.
//
// One CTA plans the batch (the sums need every entry).  Few new rows are
// numbered by the same CTA; for many a second launch spreads them over the GPU,
// each CTA taking the sums of pages anew from what the first one wrote.  It is
// bound by latency: a chain of four dependent loads (ids, lengths, ring or
// table, and the arguments), a scan and the launch.
#include "common.cuh"
#include "kv8.h"

namespace spec {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
// new rows that the planning CTA numbers itself
constexpr int kPlanOwnRows = 4 * kPlanThreads;

struct PlanSmem {
  int* off;   // [batch + 1] new rows before each entry
  int* need;  // [batch] pages taken before each entry
  int* back;  // [batch + 1] pages given back before each entry
  int* cur;   // [batch] length before the step
};

__device__ __forceinline__ int blocks_of(int n, int lg) { return (int)(((unsigned)n + (1u << lg) - 1u) >> lg); }

// inclusive sums over the block of three values; `part` holds one triple per warp
__device__ __forceinline__ void block_scan3(long long v[3], long long (*part)[3], long long carry[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const long long u = __shfl_up_sync(0xffffffffu, v[q], o);
      if (lane >= o) v[q] += u;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int q = 0; q < 3; ++q) part[warp][q] = v[q];
  }
  __syncthreads();
  long long total[3] = {carry[0], carry[1], carry[2]};
  for (int w = 0; w < n_warps; ++w) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (w < warp) v[q] += part[w][q];
      total[q] += part[w][q];
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    v[q] += carry[q];
    carry[q] = total[q];
  }
  __syncthreads();
}

// the entry b with s[b] <= i < s[b + 1] (s ascending from 0, i < s[n])
__device__ __forceinline__ int entry_of(const int* s, int n, int i) {
  int lo = 0, hi = n;  // s[lo] <= i < s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// slots of rows first, first + step, ...; the row that opens a page writes its table entry
__device__ void fill_slots(const spec_kv8_plan_args& a, const PlanSmem& sm, int lg, int n_pages, int head, int total,
                           int first, int step) {
  for (int i = first; i < a.max_rows; i += step) {
    int slot = -1;
    if (i < total) {
      const int b = entry_of(sm.off, a.batch, i);
      const int pos = sm.cur[b] + (i - sm.off[b]);
      const int block = pos >> lg;
      const int k = block - blocks_of(sm.cur[b], lg);
      int* entry = a.tables + (size_t)(a.seq_ids ? a.seq_ids[b] : b) * a.max_blocks + block;
      const int place = pos & ((1 << lg) - 1);
      int pg;
      if (k >= 0) {
        int at = head + sm.need[b] + k;  // < 2 n_pages
        if (at >= n_pages) at -= n_pages;
        pg = a.ring[at];
        if (place == 0) *entry = pg;
      } else {
        pg = *entry;
      }
      slot = (int)(((unsigned)pg << lg) + (unsigned)place);
    }
    a.slots[i] = slot;
  }
}

__global__ void __launch_bounds__(kPlanThreads) kv8_plan_kernel(spec_kv8_plan_args a, int lg, int n_pages) {
  extern __shared__ int sm_raw[];
  __shared__ long long part[kPlanThreads / 32][3];
  const int n = a.batch, tid = threadIdx.x;
  PlanSmem sm;
  sm.off = sm_raw;
  sm.back = sm.off + n + 1;
  sm.need = sm.back + n + 1;
  sm.cur = sm.need + n;
  unsigned* seen = reinterpret_cast<unsigned*>(sm.cur + n);
  const int words = a.seq_ids ? (a.n_seqs + 31) >> 5 : 0;
  for (int i = tid; i < words; i += kPlanThreads) seen[i] = 0u;
  const int head = a.state[0], count = a.state[1];
  __syncthreads();
  int bad = 0;
  if (head < 0 || head >= n_pages || count < 0 || count > n_pages) bad |= SPEC_KV8_INDEX;
  const long long cap = (long long)a.max_blocks << lg;
  long long carry[3] = {0, 0, 0};
  for (int b0 = 0; b0 < n; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long v[3] = {0, 0, 0};
    int cur = 0;
    if (b < n) {
      const int id = a.seq_ids ? a.seq_ids[b] : b;
      bool ok = id >= 0 && id < a.n_seqs;
      if (ok && a.seq_ids) ok = !(atomicOr(&seen[id >> 5], 1u << (id & 31)) >> (id & 31) & 1u);
      if (ok) {
        cur = a.lengths[id];
        ok = cur >= 0 && cur <= cap;
      }
      if (!ok) {
        bad |= SPEC_KV8_INDEX;
        cur = 0;
      } else {
        const long long next = max(0ll, (long long)cur + a.add[b]);
        if (next > cap) bad |= SPEC_KV8_TABLE;
        const long long nb0 = blocks_of(cur, lg), nb1 = (next + (1 << lg) - 1) >> lg;
        v[0] = max(0ll, next - cur);
        v[1] = max(0ll, nb1 - nb0);
        v[2] = max(0ll, nb0 - nb1);
      }
    }
    const long long own[3] = {v[0], v[1], v[2]};
    block_scan3(v, part, carry);
    if (b < n) {
      sm.off[b] = (int)(v[0] - own[0]);
      sm.need[b] = (int)(v[1] - own[1]);
      sm.back[b] = (int)(v[2] - own[2]);
      sm.cur[b] = cur;
    }
  }
  if (carry[0] > a.max_rows) bad |= SPEC_KV8_ROWS;
  if (carry[1] > count) bad |= SPEC_KV8_PAGES;
  if (carry[2] + count > n_pages) bad |= SPEC_KV8_INDEX;  // more pages than the pool has
  int status = 0;
#pragma unroll
  for (int bit = 1; bit <= SPEC_KV8_INDEX; bit <<= 1)
    if (__syncthreads_or(bad & bit)) status |= bit;
  const int total = status ? 0 : (int)carry[0];
  if (tid == 0) {
    sm.off[n] = (int)carry[0];
    sm.back[n] = (int)carry[2];
  }
  __syncthreads();
  // the new lengths (every input length is read before any is written: they may be one array)
  for (int s0 = 0; s0 < a.n_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    if (s < a.n_seqs && a.lengths_out != a.lengths) a.lengths_out[s] = a.lengths[s];
  }
  __syncthreads();
  for (int b = tid; b < n; b += kPlanThreads) {
    a.offsets[b] = status ? 0 : sm.off[b];
    if (!status) {
      const int id = a.seq_ids ? a.seq_ids[b] : b;
      a.lengths_out[id] = (int)max(0ll, (long long)sm.cur[b] + a.add[b]);
    }
  }
  if (tid == 0) {
    int h2 = head, c2 = count;
    if (!status) {
      h2 = (int)((head + carry[1]) % n_pages);
      c2 = (int)(count - carry[1] + carry[2]);
    }
    a.offsets[n] = total;
    a.state_out[0] = h2;
    a.state_out[1] = c2;
    a.status[0] = status;
  }
  if (!status) {
    const int given = sm.back[n];
    for (int j = tid; j < given; j += kPlanThreads) {
      const int b = entry_of(sm.back, n, j);
      const int id = a.seq_ids ? a.seq_ids[b] : b;
      const long long next = max(0ll, (long long)sm.cur[b] + a.add[b]);
      const int block = blocks_of((int)next, lg) + (j - sm.back[b]);
      a.ring[((long long)head + count + j) % n_pages] = a.tables[(size_t)id * a.max_blocks + block];
    }
  }
  if (a.max_rows <= kPlanOwnRows)
    fill_slots(a, sm, lg, n_pages, head, total, tid, kPlanThreads);
}

// The slots of many new rows, from what kv8_plan_kernel wrote.
__global__ void __launch_bounds__(kFillThreads) kv8_fill_kernel(spec_kv8_plan_args a, int lg, int n_pages) {
  extern __shared__ int sm_raw[];
  __shared__ long long part[kFillThreads / 32][3];
  const int n = a.batch, tid = threadIdx.x;
  PlanSmem sm;
  sm.off = sm_raw;
  sm.back = nullptr;
  sm.need = sm.off + n + 1;
  sm.cur = sm.need + n;
  pdl_wait();
  const int total = a.offsets[n];
  long long carry[3] = {0, 0, 0};
  if (total > 0) {
    for (int b0 = 0; b0 < n; b0 += kFillThreads) {
      const int b = b0 + tid;
      long long v[3] = {0, 0, 0};
      int off = 0, cur = 0;
      if (b < n) {
        off = a.offsets[b];
        const int rows = a.offsets[b + 1] - off;
        const int next = a.lengths_out[a.seq_ids ? a.seq_ids[b] : b];
        cur = next - rows;
        if (rows > 0) v[1] = blocks_of(next, lg) - blocks_of(cur, lg);
      }
      const long long own = v[1];
      block_scan3(v, part, carry);
      if (b < n) {
        sm.off[b] = off;
        sm.need[b] = (int)(v[1] - own);
        sm.cur[b] = cur;
      }
    }
    if (tid == 0) sm.off[n] = total;
    __syncthreads();
  }
  int head = a.state_out[0] - (int)carry[1];
  if (head < 0) head += n_pages;
  fill_slots(a, sm, lg, n_pages, head, total, blockIdx.x * kFillThreads + tid, gridDim.x * kFillThreads);
}

size_t plan_smem(int batch, int n_seqs, bool ids) {
  return 4 * (4 * (size_t)batch + 2) + (ids ? 4 * (size_t)((n_seqs + 31) / 32) : 0);
}

}  // namespace

cudaError_t kv8_plan_configure() {
  cudaError_t e = cudaFuncSetAttribute(kv8_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)plan_smem(kKv8MaxBatch, kKv8MaxSeqs, true));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv8_fill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * (3 * kKv8MaxBatch + 1));
  return e;
}

cudaError_t launch_kv8_plan(const spec_kv8_plan_args& a, int page_log2, int n_pages, cudaStream_t s) {
  kv8_plan_kernel<<<1, kPlanThreads, plan_smem(a.batch, a.n_seqs, a.seq_ids != nullptr), s>>>(a, page_log2, n_pages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.max_rows <= kPlanOwnRows) return e;
  cudaLaunchConfig_t cfg = {};
  const int ctas = (a.max_rows + kFillThreads - 1) / kFillThreads;
  cfg.gridDim = dim3(ctas < 592 ? ctas : 592);
  cfg.blockDim = dim3(kFillThreads);
  cfg.dynamicSmemBytes = 4 * (3 * (size_t)a.batch + 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_fill_kernel, a, page_log2, n_pages);
}

}  // namespace spec
