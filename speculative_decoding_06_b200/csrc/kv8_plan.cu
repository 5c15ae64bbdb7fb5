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
// table, and the arguments), a scan and the launch: 3.6 us for a step of 4
// sequences, 7.9 us for 256, 9.4 us for prompts of 128 with the second launch (6.4, 10.3
// and 11.5 with a scan of one level and without ids and sums in shared memory).
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
  int* id;    // [batch] sequence
};

__device__ __forceinline__ int blocks_of(int n, int lg) { return (int)(((unsigned)n + (1u << lg) - 1u) >> lg); }

// Inclusive sums over the block of three values, on top of `carry`, which becomes the block's total; `part` holds one
// triple per warp and one more.
__device__ __forceinline__ void warp_scan3(long long v[3], int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const long long u = __shfl_up_sync(0xffffffffu, v[q], o);
      if (lane >= o) v[q] += u;
    }
  }
}
__device__ __forceinline__ void block_scan3(long long v[3], long long (*part)[3], long long carry[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  warp_scan3(v, lane);
  if (lane == 31) {
#pragma unroll
    for (int q = 0; q < 3; ++q) part[warp][q] = v[q];
  }
  __syncthreads();
  if (warp == 0) {
    long long w[3] = {0, 0, 0};
    if (lane < n_warps) {
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q] = part[lane][q];
    }
    warp_scan3(w, lane);
    if (lane < n_warps) {
#pragma unroll
      for (int q = 0; q < 3; ++q) part[lane][q] = w[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    v[q] += carry[q] + (warp ? part[warp - 1][q] : 0);
    carry[q] += part[n_warps - 1][q];
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
      int* entry = a.tables + (size_t)sm.id[b] * a.max_blocks + block;
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
  __shared__ int s_bad;
  const int n = a.batch, tid = threadIdx.x;
  PlanSmem sm;
  sm.off = sm_raw;
  sm.back = sm.off + n + 1;
  sm.need = sm.back + n + 1;
  sm.cur = sm.need + n;
  sm.id = sm.cur + n;
  unsigned* seen = reinterpret_cast<unsigned*>(sm.id + n);
  const int words = a.seq_ids ? (a.n_seqs + 31) >> 5 : 0;
  const int threads = blockDim.x;
  for (int i = tid; i < words; i += threads) seen[i] = 0u;
  if (tid == 0) s_bad = 0;
  const int head = a.state[0], count = a.state[1];
  __syncthreads();
  int bad = 0;
  if (head < 0 || head >= n_pages || count < 0 || count > n_pages) bad |= SPEC_KV8_INDEX;
  const long long cap = (long long)a.max_blocks << lg;
  long long carry[3] = {0, 0, 0};
  for (int b0 = 0; b0 < n; b0 += threads) {
    const int b = b0 + tid;
    long long v[3] = {0, 0, 0};
    int cur = 0, id = 0;
    if (b < n) {
      id = a.seq_ids ? a.seq_ids[b] : b;
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
      sm.id[b] = id;
    }
  }
  if (carry[0] > a.max_rows) bad |= SPEC_KV8_ROWS;
  if (carry[1] > count) bad |= SPEC_KV8_PAGES;
  if (carry[2] + count > n_pages) bad |= SPEC_KV8_INDEX;  // more pages than the pool has
  bad = __reduce_or_sync(0xffffffffu, bad);
  if ((tid & 31) == 0 && bad) atomicOr(&s_bad, bad);
  if (tid == 0) {
    sm.off[n] = (int)carry[0];
    sm.back[n] = (int)carry[2];
  }
  // (every input length is read by here: the output may be the same array)
  if (a.lengths_out != a.lengths)
    for (int i = tid; i < a.n_seqs; i += threads) a.lengths_out[i] = a.lengths[i];
  __syncthreads();
  const int status = s_bad;
  const int total = status ? 0 : (int)carry[0];
  for (int b = tid; b < n; b += threads) {
    a.offsets[b] = status ? 0 : sm.off[b];
    if (!status) a.lengths_out[sm.id[b]] = (int)max(0ll, (long long)sm.cur[b] + a.add[b]);
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
    for (int j = tid; j < given; j += threads) {
      const int b = entry_of(sm.back, n, j);
      const int kept = blocks_of(sm.cur[b], lg) - (sm.back[b + 1] - sm.back[b]);
      int at = head + count + j;  // < 3 n_pages
      at -= at >= 2 * n_pages ? 2 * n_pages : at >= n_pages ? n_pages : 0;
      a.ring[at] = a.tables[(size_t)sm.id[b] * a.max_blocks + kept + (j - sm.back[b])];
    }
  }
  if (a.max_rows <= kPlanOwnRows)
    fill_slots(a, sm, lg, n_pages, head, total, tid, threads);
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
  sm.id = sm.cur + n;
  pdl_wait();
  const int total = a.offsets[n];
  long long carry[3] = {0, 0, 0};
  if (total > 0) {
    for (int b0 = 0; b0 < n; b0 += kFillThreads) {
      const int b = b0 + tid;
      long long v[3] = {0, 0, 0};
      int off = 0, cur = 0, id = 0;
      if (b < n) {
        off = a.offsets[b];
        const int rows = a.offsets[b + 1] - off;
        id = a.seq_ids ? a.seq_ids[b] : b;
        const int next = a.lengths_out[id];
        cur = next - rows;
        if (rows > 0) v[1] = blocks_of(next, lg) - blocks_of(cur, lg);
      }
      const long long own = v[1];
      block_scan3(v, part, carry);
      if (b < n) {
        sm.off[b] = off;
        sm.need[b] = (int)(v[1] - own);
        sm.cur[b] = cur;
        sm.id[b] = id;
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
  return 4 * (5 * (size_t)batch + 2) + (ids ? 4 * (size_t)((n_seqs + 31) / 32) : 0);
}

}  // namespace

cudaError_t kv8_plan_configure() {
  cudaError_t e = cudaFuncSetAttribute(kv8_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)plan_smem(kKv8MaxBatch, kKv8MaxSeqs, true));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv8_fill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * (4 * kKv8MaxBatch + 1));
  return e;
}

cudaError_t launch_kv8_plan(const spec_kv8_plan_args& a, int page_log2, int n_pages, cudaStream_t s) {
  // a small step is bound by the latency of its barriers: fewer warps
  const int threads = a.batch <= 32 && a.max_rows <= 1024 ? 256 : kPlanThreads;
  kv8_plan_kernel<<<1, threads, plan_smem(a.batch, a.n_seqs, a.seq_ids != nullptr), s>>>(a, page_log2, n_pages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.max_rows <= kPlanOwnRows) return e;
  cudaLaunchConfig_t cfg = {};
  const int ctas = (a.max_rows + kFillThreads - 1) / kFillThreads;
  cfg.gridDim = dim3(ctas < 592 ? ctas : 592);
  cfg.blockDim = dim3(kFillThreads);
  cfg.dynamicSmemBytes = 4 * (4 * (size_t)a.batch + 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_fill_kernel, a, page_log2, n_pages);
}

}  // namespace spec
