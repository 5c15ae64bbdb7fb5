// Attention over the 8-bit paged cache for draft trees and prompt chunks, on the
// 5th-generation tensor cores.
//
// A CTA holds a tile of 128 query rows (row = node * G + g of one kv head,
// G = Hq / Hkv) and walks over keys in units of 64, first its share of the cached
// prefix, then the step's own rows that its rows can see.  Two softmax streams take
// the units in turn, each with its own running maximum, sum and output; they join
// at the end.
//
//   loader (1 thread)     bulk copies of the codes of a unit, three units deep, the first ones as soon as its warp
//       has looked up their pages.
//   helper (1 warp)       the tree's ancestor sets.
//   converters (4 warps for K, 4 for V)  turn codes into fp16 (exact) and write them as
//       the swizzled K and V operands.  K and V of the step's own rows become fp16
//       times a power of two that the largest value of 64 rows sets, or, where their sizes differ
//       by more than 2^kRowSpread, each row's own: a row must not suffer from one that it does not see.
//   issuers (1 thread per stream)  S = Q K^T (M 128, N 64) with q in TMEM, into one of three
//       TMEM buffers, and O += P V (P from TMEM, V MN-major); scores run a unit ahead of products.
//   softmax (4 warps per stream)  a thread per row: the online softmax in base 2, P as
//       fp16 over the S that it came from.
//
// What bounds it: a unit takes 0.59 us of a CTA, 1050 cycles, of which the MMAs need
// 512, the exponentials 512 of the special-function units, shared memory 770 (codes in and out, operands in and out)
// and the instructions of softmax and conversion some 700 of the issue slots; the rest is the latency of a unit's
// chain (codes to operand, tensor memory to registers and back, six barriers).  Start and end of a CTA take 9 us, with
// a cluster's join 10 - 14.  4 prompts of 6150 - 8192 tokens, 128 rows x 8 kv heads x 4: 92.5 us, 672 TFLOP/s (91.1 before
// the sums were made to hold for scales of any distance).
// Tried and slower: one issuer for both streams, which keeps them in step, so that both want the special-function
// units at once (0.95 us a unit); codes by cp.async of the converters (0.95 us); four threads per row, whose
// exchange of maxima costs what it saves (0.97 us); 128-key score tiles (0.97 us); q in shared memory, read again
// for every unit (0.03 us more).  Two row tiles that share a unit's conversion took 11 % less per row than one did
// then, but need twice the rows.  Tiles cut by their work, so that each SM has as many units, with parts joined by
// the last CTA to arrive: a second tile per CTA and the joining cost 19 us, more than the even load gave (the four
// prompts 104 us, 16 trees 89 us, when they took 94 and 79).  q by one bulk copy per row (128 copies of 256 bytes take
// 5 us), or read in half rows, a thread each (2000 cycles of the load pipe).
//
// Scales: the unit's K exponent (the largest of its pages'; codes of a page with a
// smaller one, by up to 2^kSpread, are multiplied by the difference as they are converted, which
// is exact; further apart, each key keeps its page's) multiplies the scores; its V exponent w goes
// into the exponential: p' = 2^(x + w - m) with m 7 below a running maximum of x + w,
// moved only when exceeded by more than 15 (p' <= 2^15, and fp16 has its full 11 bits
// down to 2^-21 of the largest p'), O sums p' times bare codes and the denominator
// p' 2^(12 - w).  The weights do not depend on V, so the denominator has to hold where p' does not: see kLift and kFar.
// p' is rounded to fp16 (2^-11 of itself) for the product; O is divided by the
// sum of the rounded p', so that a key's rounding cancels as far as its weight dominates, and
// the log-sum-exp is that of the unrounded ones.
//
// The CTAs of a cluster share a sequence's prefix evenly and merge their normalised
// outputs and log-sum-exps through distributed shared memory.
#include "common.cuh"
#include "kv8.h"

namespace spec {

namespace {

constexpr int kRowTile = 128;
constexpr int kKeys = 64;  // keys of a unit
constexpr int kConvWarps = 4;  // per plane
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kCodeStages = 3;
constexpr uint32_t kHalf = kKeys * 128;      // [64 keys][64 fp16]: 8 KB
constexpr uint32_t kUnit = 2 * kHalf;        // one unit's K or V
constexpr uint32_t kCodeTile = kKeys * kKv8Hd;  // one plane
constexpr int kMaxUnits = kKv8TcMaxKeys / kKeys;  // of a CTA's share: their pages are looked up up front

constexpr int kRowWarps = 8;  // two streams of four
constexpr int kIssueWarp = kRowWarps + 2 * kConvWarps;  // and the next one: one per stream
constexpr int kLoadWarp = kIssueWarp + 2;
constexpr int kHelpWarp = kLoadWarp + 1;  // ancestors
constexpr int kThreads = 32 * (kHelpWarp + 1);
constexpr int kStages = 4;    // most operand stages of K or V

constexpr int kByLength = 128;  // most sequences that are put in order
constexpr int kScores = 3;    // S buffers: unit u has buffer u % 3
// l is the sum of 2^(x - m + kLift).  With w in [-80, 120] and m 7 to 22 below the largest x + w, its largest term lies
// between 2^-101 and 2^107: the sum neither overflows nor loses terms above 2^-25 of the largest.
constexpr float kLift = 12.f;
// Units whose w is that far below the largest so far may have p' = 0 for weights that count in l: l then takes the weights
// themselves.  (A weight of 2^-43 of the largest has p' of 2^-126 or more at this distance.)
constexpr float kFar = 90.f;
// the smallest code is 2^-9 and fp16 ends at 2^-24
constexpr int kSpread = 15;
// (fp16 has its 11 bits down to 2^-21 of a tile's largest value: 2^-13 of the largest of a row that is 2^-8 as large)
constexpr int kRowSpread = 8;

// mbarriers: per operand stage; S, P and P V per stream, for its even and its odd units: no wait is for a phase that
// lies more than one behind what its waiter has seen, however far idle warps of a stream run ahead
enum { B_Q = 0, B_O = 1, B_TREF = 2, B_DRAIN = 4, B_ANC = 6, B_KFULL = 7, B_KEMPTY = B_KFULL + kStages, B_VFULL = B_KEMPTY + kStages,
       B_VEMPTY = B_VFULL + kStages, B_SFULL = B_VEMPTY + kStages, B_PFULL = B_SFULL + 4, B_PV = B_PFULL + 4,
       B_CFULL = B_PV + 4, B_CEMPTY = B_CFULL + 2 * kCodeStages, kNumBars = B_CEMPTY + 2 * kCodeStages };

constexpr uint32_t kJoin = kRowTile * (512 + 2 * 256);

constexpr uint32_t kQPitch = kKv8Hd * 2 + 16;  // a row of q: its pieces of 16 bytes meet in no bank

struct M {  // shared memory
  static constexpr int nk = 3;             // operand stages (units) of K
  static constexpr int nv = 4;             // and V
  static constexpr uint32_t q = 0;
  static constexpr uint32_t k = q + (kRowTile * kQPitch + 1023) / 1024 * 1024;
  static constexpr uint32_t v = k + nk * kUnit;
  static constexpr uint32_t codes = v + nv * kUnit;
  static constexpr uint32_t group = codes + 2 * kCodeStages * kCodeTile;  // int4 [kMaxUnits]: first rows / 16 of the groups of 16 keys
  static constexpr uint32_t kexp = group + 16 * kMaxUnits;                // uint32 [kMaxUnits]: exponent bytes of the four groups
  static constexpr uint32_t vexp = kexp + 4 * kMaxUnits;
  static constexpr uint32_t unit = vexp + 4 * kMaxUnits;  // float2 [kMaxUnits + 2]: factor of K (negative: each key has its own), exponent of V
  static constexpr uint32_t anc = unit + 8 * (kMaxUnits + 2);  // uint64 [2][128][2]
  static constexpr uint32_t jump = anc + 2 * 128 * 16;    // int [2][128]
  static constexpr uint32_t half = jump + 2 * 128 * 4;    // float [2][128]: largest values of the halves of q, at the end the streams' log-sum-exps
  static constexpr uint32_t row = half + 2 * 128 * 4;     // uint32 [2][2][64]: the largest values of halves of 64 own rows of K and V; at the end float [128]: the rows' log-sum-exps
  static constexpr uint32_t own = row + 2 * 128 * 4;      // uint8 [2][128]: exponent bytes of the own rows of K and V
  static constexpr uint32_t vbad = own + 256;             // uint32 [4]: own rows whose V holds an infinity or NaN
  static constexpr uint32_t bars = vbad + 16;
  static constexpr uint32_t misc = bars + 8 * kNumBars + 8;
  static constexpr uint32_t end = misc + 16;
  static constexpr uint32_t dyn = end + 1024;             // to a 1024-byte boundary
  // at the end, over the operands: the tile's O (128 rows of 512 B), then half a row of each stream for the other
  static constexpr uint32_t stage = 0;
};
static_assert(M::dyn <= 227 * 1024, "shared memory");
static_assert(M::codes - M::stage >= kJoin, "staging");

// TMEM columns: O of the streams, the S buffers (P lies over the first half of its S), q as the scores' A operand.
// (q in shared memory would be read again for every unit: 256 of the 1024 cycles that a unit then takes of the
// shared-memory pipe.)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256, kColQ = kColS + kScores * kKeys;
static_assert(kColQ + 64 <= kTmemCols, "tensor memory");
constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRowTile >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(kRowTile >> 4) << 24);

struct TcPlan {
  int chunks;          // CTAs of a cluster
  bool by_length;      // blocks of the longest prefixes first
  uint32_t by_chunks;  // ceil(2^32 / chunks): x / chunks = x * by_chunks >> 32 for x < 2^29
  uint32_t by_group;   // ceil(2^20 / G): x / G = x * by_group >> 20 for x <= 128 * 64
};

// `bytes` (a multiple of 16) from global to shared memory, counted on `bar`
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// the converters of one plane
__device__ __forceinline__ void sync_converters(int plane) {
  asm volatile("bar.sync %0, %1;" ::"r"(3 + plane), "n"(kConvThreads) : "memory");
}
__device__ __forceinline__ void sync_rows() { asm volatile("bar.sync 2, %0;" ::"n"(32 * kRowWarps) : "memory"); }
// four e4m3 codes as fp16
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& x, uint32_t& y) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(x), "=r"(y)
      : "r"(w));
}
// the factor that a page's exponent byte stands for (255: NaN)
__device__ __forceinline__ float scale_of(int byte) { return byte >= 255 ? NAN : __int_as_float(byte << 23); }
__device__ __forceinline__ float exp_of(int byte) { return byte >= 255 ? NAN : (float)(byte - 127); }
__device__ __forceinline__ int max4(uint32_t w) {
  return max(max((int)(w & 255), (int)(w >> 8 & 255)), max((int)(w >> 16 & 255), (int)(w >> 24)));
}
__device__ __forceinline__ int min4(uint32_t w) {
  return min(min((int)(w & 255), (int)(w >> 8 & 255)), min((int)(w >> 16 & 255), (int)(w >> 24)));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t v, __half2 f) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&v), f);
  return *reinterpret_cast<const uint32_t*>(&y);
}
// the exponent that brings values up to `amax` below 2^7 (0 where all are 0)
__device__ __forceinline__ int shift_of(float amax, int least = -120) {
  const int e = (__float_as_int(amax) >> 23) - 127 - 6;
  return amax > 0.f ? max(least, min(120, e)) : 0;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(e[i]);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8], float f) {
  return make_uint4(pack2(v[0] * f, v[1] * f), pack2(v[2] * f, v[3] * f), pack2(v[4] * f, v[5] * f),
                    pack2(v[6] * f, v[7] * f));
}

// largest magnitude of two 16-bit values' bits (sign cleared), pairwise
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
template <typename T> __device__ __forceinline__ constexpr uint32_t inf_bits() { return __is_same(T, __half) ? 0x7c00u : 0x7f80u; }
// the same by the type's own maximum, NaN above all others
template <typename T>
__device__ __forceinline__ uint32_t max_abs_nan(uint32_t m, uint32_t w) {
  using T2 = std::conditional_t<__is_same(T, __half), __half2, __nv_bfloat162>;
  const T2 y = __hmax2_nan(reinterpret_cast<const T2&>(m), __habs2(reinterpret_cast<const T2&>(w)));
  return reinterpret_cast<const uint32_t&>(y);
}
// sets infinities and NaN among eight 16-bit values to 0; whether there were any
template <typename T>
__device__ __forceinline__ bool finite_only(uint4& r) {
  bool any = false;
  auto one = [&](uint32_t& w) {
    const bool lo = (w & 0x7fffu) >= inf_bits<T>(), hi = (w >> 16 & 0x7fffu) >= inf_bits<T>();
    any |= lo | hi;
    w &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
  };
  one(r.x), one(r.y), one(r.z), one(r.w);
  return any;
}

// Each thread of the warp reads 4, writes 2 consecutive 32-bit columns of its own lane.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st2_async(uint32_t taddr, uint32_t a, uint32_t b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}

// a + c, a in 16 bits
__device__ __forceinline__ float add_half(float c, uint16_t a) {
  float d;
  asm("add.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(a), "f"(c));
  return d;
}

// A unit whose keys have exponents of their own, or whose weights p' may not hold, in tensor memory at `ts` (rare, and so
// kept out of the loop that calls it).  P false: the largest x + w.  P true: writes p' over the scores and returns the sum
// of the weights 2^(x - m + kLift), taken as squares: these end at 2^-149 where one exponential ends at 2^-126.
// bytes: K's exponent bytes, V's behind them; null: f is K's whole factor and ve V's exponent.
template <bool P>
__device__ __noinline__ float unit_apart(uint32_t ts, uint64_t see, const uint8_t* bytes, bool pages, float f, float ve,
                                         float m) {
  float r = P ? 0.f : -INFINITY;
#pragma unroll 1
  for (int j = 0; j < kKeys / 4; ++j) {
    float x[4], w[4];
    tmem_ld4(ts + 4 * j, x);
    const uint32_t sees = (uint32_t)(see >> (4 * j));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[k] = ve;
      float kf = f;
      if (bytes) {
        const uint8_t* at = bytes + (pages ? j >> 2 : 4 * j + k);
        kf *= scale_of(*at);
        w[k] = exp_of(at[pages ? M::vexp - M::kexp : 128]);
      }
      x[k] = sees >> k & 1u ? x[k] * kf : -INFINITY;
      if (P) {
        const float h = fast_exp2(0.5f * (x[k] - m + kLift));
        r = fmaf(h, h, r);
        x[k] = fast_exp2(x[k] + (w[k] - m));
      } else {
        r = fmaxf(r, x[k] + w[k]);
      }
    }
    if (P) tmem_st2_async(ts + 2 * j, pack2(x[0], x[1]), pack2(x[2], x[3]));  // over scores that have been read
  }
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) kv8_tree_kernel(Kv8View c, spec_kv8_attention_args a, TcPlan pl) {
  extern __shared__ uint8_t smem_raw[];
  // (to a 1024-byte boundary by an offset, so that the compiler still knows what it points to as shared memory)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + M::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + M::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + M::misc + 4);
  int4* s_group = reinterpret_cast<int4*>(smem + M::group);
  uint32_t* s_vbad = reinterpret_cast<uint32_t*>(smem + M::vbad);
  float2* s_unit = reinterpret_cast<float2*>(smem + M::unit);
  float* s_row = reinterpret_cast<float*>(smem + M::row);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kLoadWarp && lane == 0) {
    mbar_init(&bar[B_Q], kRowWarps);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar[B_KFULL + s], kConvWarps);
      mbar_init(&bar[B_KEMPTY + s], 1);
      mbar_init(&bar[B_VFULL + s], kConvWarps);
      mbar_init(&bar[B_VEMPTY + s], 1);
    }
    for (int s = 0; s < 2 * kCodeStages; ++s) {
      mbar_init(&bar[B_CFULL + s], 1);
      mbar_init(&bar[B_CEMPTY + s], kConvWarps);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bar[B_SFULL + s], 1);
      mbar_init(&bar[B_PFULL + s], 4);
      mbar_init(&bar[B_PV + s], 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&bar[B_TREF + s], 2 * kConvWarps);
    mbar_init(&bar[B_O], 2);
    mbar_init(&bar[B_DRAIN], 1);
    mbar_init(&bar[B_DRAIN + 1], 1);
    mbar_init(&bar[B_ANC], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  const int G = a.n_q_heads / c.hkv;
  auto by_g = [&](int x) { return (int)((uint32_t)x * pl.by_group >> 20); };
  // grid: x = row tiles * chunks (a cluster is the chunks of a row tile), y = kv heads, z = batch.  The CTAs of a
  // cluster differ in `share` only: they return together or not at all
  const int share = pl.chunks > 1 ? (int)cluster_rank() : 0;
  const int row0 = (pl.chunks > 1 ? (int)cluster_id_x() : (int)blockIdx.x) * kRowTile;
  const int kvh = blockIdx.y;
  int b = blockIdx.z;
  if (pl.by_length) {  // blocks start in order: the longest prefixes first
    int* len = reinterpret_cast<int*>(s_row);
    if (tid < a.batch) {
      const int s = a.seq_ids ? a.seq_ids[tid] : tid;
      len[tid] = s < 0 || s >= a.n_seqs ? -1 : a.lengths[s];
    }
    __syncthreads();
    if (tid < a.batch) {
      const int own = len[tid];
      int rank = 0;
      for (int i = 0; i < a.batch; ++i) rank += len[i] > own || (len[i] == own && i < tid);
      if (rank == b) len[kByLength] = tid;
    }
    __syncthreads();
    b = len[kByLength];
  }
  const int first = a.offsets[b], n = a.offsets[b + 1] - first;
  const int seq = a.seq_ids ? a.seq_ids[b] : b;
  if (a.fill && row0 == 0 && share == 0) kv8_fill_rows(a, b, kvh, G);
  if (seq < 0 || seq >= a.n_seqs || first < 0 || n < 1 || n > a.max_nodes || n > a.rows - first) return;
  const int P = a.lengths[seq];
  const int rows = n * G;
  if (P < 0 || P > a.max_prefix || row0 >= rows) return;
  // this CTA's share of the prefix, whole units; the last one also has the step's own rows, which take as long as two
  const int even = (int)__umulhi((uint32_t)(P + (a.k_new ? 2 * kKeys : 0) + pl.chunks - 1), pl.by_chunks);
  const int per = pl.chunks == 1 ? P : min((even + kKeys - 1) / kKeys * kKeys, kKv8TcMaxKeys);
  const int c0 = min(P, share * per), c1 = min(P, c0 + per);
  const int top = min(n - 1, by_g(row0 + kRowTile - 1));  // last node that a row here can see
  const int np = (c1 - c0 + kKeys - 1) / kKeys;                   // units of the prefix
  const int nt = (a.k_new && share == pl.chunks - 1) ? top / kKeys + 1 : 0;  // of the step's own rows: they come last
  const int nu = np + nt;

  // the copies of the first units start before the CTA's other threads are ready for them
  const uint32_t ring = smem_u32(smem + M::codes);
  auto load_unit = [&](int u, int st, int p) {
    const int4 at = s_group[u];
    uint64_t* full = &bar[B_CFULL + p * kCodeStages + st];
    mbar_arrive_expect_tx(full, kCodeTile);
    const uint32_t dst = ring + (p * kCodeStages + st) * kCodeTile;
    const uint8_t* src = c.codes[p];
    if (at.y == at.x + 1 && at.z == at.x + 2 && at.w == at.x + 3) {  // one stretch of memory
      bulk_load(dst, src + (size_t)at.x * (16 * kKv8Hd), kCodeTile, full);
    } else {
      bulk_load(dst, src + (size_t)at.x * (16 * kKv8Hd), kCodeTile / 4, full);
      bulk_load(dst + kCodeTile / 4, src + (size_t)at.y * (16 * kKv8Hd), kCodeTile / 4, full);
      bulk_load(dst + kCodeTile / 2, src + (size_t)at.z * (16 * kKv8Hd), kCodeTile / 4, full);
      bulk_load(dst + kCodeTile / 4 * 3, src + (size_t)at.w * (16 * kKv8Hd), kCodeTile / 4, full);
    }
  };
  ulonglong2* const s_anc = reinterpret_cast<ulonglong2*>(smem + M::anc);
  int* const s_jump = reinterpret_cast<int*>(smem + M::jump);
  uint4 qraw[8];  // half a warp per row, 16 rows per row warp
  if (warp < kRowWarps) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int qr = row0 + 16 * warp + 2 * i + (lane >> 4), node = by_g(qr);
      qraw[i] = make_uint4(0, 0, 0, 0);
      if (qr < rows)
        qraw[i] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + a.q_row_stride * (first + node) +
                                                       a.q_head_stride * (kvh * G + (qr - node * G))) + (lane & 15));
    }
  } else if (warp == kHelpWarp) {
    if (nt > 0 && a.parents) {
      for (int node = lane; node < 128; node += 32) {
        const int up = node <= top ? a.parents[first + node] : -1;
        s_anc[node] = make_ulonglong2(node < 64 ? 1ull << node : 0ull, node < 64 ? 0ull : 1ull << (node - 64));
        s_jump[node] = up < node && up >= 0 ? up : -1;
      }
    }
  } else {
    // pages of the share's units: four groups of 16 keys, each inside one page; the loading warp has the first ones
    for (int i0 = warp == kLoadWarp ? 0 : 32 * (warp - kRowWarps + 1); i0 < np; i0 += 32 * (kHelpWarp - kRowWarps)) {
      const int i = i0 + lane;
      int pg[4], at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int key = c0 + kKeys * i + 16 * u;
        pg[u] = key < c1 ? a.tables[(size_t)seq * a.max_blocks + (key >> c.page_log2)] : -1;
      }
      uint32_t bad = 0;  // keys without a page
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool ok = pg[u] >= 0 && pg[u] < c.n_pages;
        if (!ok && c0 + kKeys * i + 16 * u < c1) bad |= 255u << (8 * u);
        at[u] = (ok ? pg[u] : 0) * c.hkv + kvh;
      }
      if (i < np) {
        int w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = ((at[u] << c.page_log2) + ((c0 + kKeys * i + 16 * u) & (c.page - 1))) >> 4;
        s_group[i] = make_int4(w[0], w[1], w[2], w[3]);
      }
      if (warp == kLoadWarp && i0 == 0) {
        __syncwarp();
        if (elect_one())
          for (int u = 0; u < min(np, kCodeStages); ++u)
            for (int p = 0; p < 2; ++p) load_unit(u, u, p);
        __syncwarp();
      }
      if (i < np) {
        uint32_t ke = bad, ve = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // (groups behind the end have the first one's)
          const int from = c0 + kKeys * i + 16 * u >= c1 ? at[0] : at[u];
          ke |= (uint32_t)c.exps[0][from] << (8 * u);
          ve |= (uint32_t)c.exps[1][from] << (8 * u);
        }
        reinterpret_cast<uint32_t*>(smem + M::kexp)[i] = ke;
        reinterpret_cast<uint32_t*>(smem + M::vexp)[i] = ve;
        const int k_top = max4(ke), v_top = max4(ve);
        const bool keyed = max(k_top - min4(ke), v_top - min4(ve)) > kSpread;
        s_unit[i] = make_float2(keyed ? -scale_of(k_top) : scale_of(k_top), exp_of(v_top));
      }
    }
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (tid < 4) s_vbad[tid] = 0u;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto held = [&](int which, uint32_t parity) { return mbar_wait(&bar[which], parity, nullptr, abort_flag); };

  if (warp == kHelpWarp) {
    // ------------------------------------------------------------ ancestors: each node's set doubles its reach per round
    if (nt > 0 && a.parents) {
      __syncwarp();
      int cur = 0;
      for (int reach = 1; reach <= top; reach *= 2) {
#pragma unroll
        for (int node = lane; node < 128; node += 32) {
          ulonglong2 set = s_anc[128 * cur + node];
          int up = s_jump[128 * cur + node];
          if (up >= 0) {
            const ulonglong2 more = s_anc[128 * cur + up];
            set.x |= more.x;
            set.y |= more.y;
            up = s_jump[128 * cur + up];
          }
          s_anc[128 * (cur ^ 1) + node] = set;
          s_jump[128 * (cur ^ 1) + node] = up;
        }
        cur ^= 1;
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&bar[B_ANC]);
    }
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    if (elect_one()) {
      bool ok = true;
      int u = min(np, kCodeStages);
      for (int st = 0, ph = 0; u < np && ok; ++u) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ok = ok && held(B_CEMPTY + p * kCodeStages + st, ph);
          if (ok) load_unit(u, st, p);
        }
        if (++st == kCodeStages) st = 0, ph ^= 1;
      }
      // copies land before the CTA's memory is released: the last into each stage may be under way (a phase that
      // had none is one that its waiters have seen complete, or never began: the wait then passes or runs out)
      for (int k = max(0, u - kCodeStages); k < u; ++k)
        for (int p = 0; p < 2; ++p)
          mbar_wait(&bar[B_CFULL + p * kCodeStages + k % kCodeStages], (k / kCodeStages) & 1, nullptr, nullptr);
    }
    __syncwarp();
  } else if (warp >= kIssueWarp) {
    // ------------------------------------------------------------ MMA issue, stream t
    const int t = warp - kIssueWarp;
    if (elect_one()) {
      const uint64_t dk = sw128_kmajor_desc(smem_u32(smem + M::k));
      const uint64_t dv = sw128_mnmajor_desc(smem_u32(smem + M::v), kHalf);
      const int n_own = (nu - t + 1) >> 1;  // units t, t + 2, ...
      int ks_ = t, kp = 0, vs = t, vp = 0;  // operand stages of K and V, and their phases
      int sb = t, pb = t;                   // S buffer of the next scores and of the next product
      bool ok = held(B_Q, 0);
      for (int i = 0; i <= n_own && ok; ++i) {
        if (i < n_own) {
          // the S buffer holds P of three units ago, unit j of the other stream, until that one's product is done
          const int j = i - 2 + t;
          ok = (j < 0 || held(B_PV + 2 * (t ^ 1) + (j & 1), (j >> 1) & 1)) && held(B_KFULL + ks_, kp);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)  // 16 dimensions per step: 8 columns of q (a descriptor's low bits count 16 bytes)
            tc_mma_ts(tmem + kColS + kKeys * sb, tmem + kColQ + 8 * ks,
                      dk + ((ks_ * kUnit + (ks >> 2) * kHalf + (ks & 3) * 32) >> 4), kIdescS, ks > 0 ? 1u : 0u);
          tc_commit(&bar[B_SFULL + 2 * t + (i & 1)]);
          tc_commit(&bar[B_KEMPTY + ks_]);
          if ((ks_ += 2) >= M::nk) ks_ -= M::nk, kp ^= 1;
          if ((sb += 2) >= kScores) sb -= kScores;
        }
        if (i > 0) {  // O += P V of the unit before
          ok = held(B_VFULL + vs, vp) && held(B_PFULL + 2 * t + ((i - 1) & 1), ((i - 1) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)  // 16 keys per step: 8 columns of P
            tc_mma_ts(tmem + 128 * t, tmem + kColS + kKeys * pb + kk * 8, dv + ((vs * kUnit + kk * 16 * 128) >> 4),
                      kIdescPV, (i > 1 || kk > 0) ? 1u : 0u);
          tc_commit(&bar[B_PV + 2 * t + ((i - 1) & 1)]);
          tc_commit(&bar[B_VEMPTY + vs]);
          if ((vs += 2) >= M::nv) vs -= M::nv, vp ^= 1;
          if ((pb += 2) >= kScores) pb -= kScores;
        }
      }
      if (ok) {
        if (nu > 0) tc_commit(&bar[B_O]);  // (without units nobody waits for it: it could land in released memory)
      } else {
        *abort_flag = 1;
        tc_commit(&bar[B_DRAIN + t]);  // issued MMAs finish before the CTA's memory is released
        mbar_wait(&bar[B_DRAIN + t], 0, nullptr, nullptr);
      }
    }
    __syncwarp();
  } else if (warp >= kRowWarps) {
    // ------------------------------------------------------------ converters
    const int p = (warp - kRowWarps) / kConvWarps;  // 0: K, 1: V
    const int x = tid - 32 * kRowWarps - p * kConvThreads;
    // 16 dimensions (piece ch) of keys kr, + 16, + 32, + 48 of a unit: eight lanes have eight keys and eight pieces,
    // which meet in no bank, neither where the codes lie in rows of 128 bytes nor in the swizzled operands
    const int wv = x >> 5, kr = (wv >> 1) * 8 + (lane & 7), ch = ((lane >> 3) + 4 * (wv & 1) + lane) & 7;
    uint8_t* const op0 = smem + (p ? M::v : M::k) + (ch >> 2) * kHalf + kr * 128;
    const uint32_t col0 = ((2 * (ch & 3)) ^ (kr & 7)) << 4, col1 = ((2 * (ch & 3) + 1) ^ (kr & 7)) << 4;
    bool ok = true;
    // operand stages in turn; one is free once the MMAs that read its last unit are done
    const int n_stages = p ? M::nv : M::nk;
    int st = 0, ph = 1;
    auto enter = [&]() {
      if (ok) ok = held((p ? B_VEMPTY : B_KEMPTY) + st, ph);  // (the first round's waits pass at once)
      ok = __all_sync(0xffffffffu, ok);
      return op0 + st * kUnit;
    };
    auto arrive = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[(p ? B_VFULL : B_KFULL) + st]);
      if (++st == n_stages) st = 0, ph ^= 1;
    };
    const uint32_t* const s_exp = reinterpret_cast<const uint32_t*>(smem + (p ? M::vexp : M::kexp));
    // the step's own rows, 64 nodes per tile: their largest finite values set the exponents.  They are looked at
    // last, while the prefix's last units wait for their turn
    const T* const own = reinterpret_cast<const T*>(p ? a.v_new : a.k_new) +
                         (p ? a.v_head_stride : a.k_head_stride) * kvh + 16 * ch;
    const int64_t own_stride = p ? a.v_row_stride : a.k_row_stride;
    auto own_row = [&](int tt, int u, uint4 (&raw)[2]) {
      const int node = kKeys * tt + 16 * u + kr;
      raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
      if (node <= top) {
        const uint4* at = reinterpret_cast<const uint4*>(own + own_stride * (first + node));
        raw[0] = __ldg(at);
        raw[1] = __ldg(at + 1);
      }
    };
    const uint8_t* const codes = smem + M::codes + p * (kCodeStages * kCodeTile) + kr * kKv8Hd + 16 * ch;
    int cs = 0, cp = 0;  // stage of the codes, its phase
    for (int j = 0; j < np; ++j) {
      if (ok) ok = held(B_CFULL + p * kCodeStages + cs, cp);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint4 w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = *reinterpret_cast<const uint4*>(codes + cs * kCodeTile + u * (16 * kKv8Hd));
      if (p && j == np - 1) {  // what lies behind the sequence's end may be anything; 0 * NaN would spread
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c0 + kKeys * j + 16 * u + kr >= c1) w[u] = make_uint4(0, 0, 0, 0);
      }
      const uint32_t e4 = s_exp[j];
      uint8_t* const op = enter();
      if (!ok) break;
      if (e4 == __byte_perm(e4, 0, 0) || s_unit[j].x < 0.f) {  // pages of one scale, or codes as they are
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 lo, hi;
          expand4(w[u].x, lo.x, lo.y);
          expand4(w[u].y, lo.z, lo.w);
          expand4(w[u].z, hi.x, hi.y);
          expand4(w[u].w, hi.z, hi.w);
          *reinterpret_cast<uint4*>(op + 2048 * u + col0) = lo;
          *reinterpret_cast<uint4*>(op + 2048 * u + col1) = hi;
        }
      } else {
        const int ref = max4(e4);
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          const int d = ref - (int)(e4 >> (8 * u) & 255);
          const __half2 f = __float2half2_rn(pow2i(-d));
          const uint4 y = u == 0 ? w[0] : u == 1 ? w[1] : u == 2 ? w[2] : w[3];
          uint4 lo, hi;
          expand4(y.x, lo.x, lo.y);
          expand4(y.y, lo.z, lo.w);
          expand4(y.z, hi.x, hi.y);
          expand4(y.w, hi.z, hi.w);
          *reinterpret_cast<uint4*>(op + 2048 * u + col0) =
              make_uint4(mul_h2(lo.x, f), mul_h2(lo.y, f), mul_h2(lo.z, f), mul_h2(lo.w, f));
          *reinterpret_cast<uint4*>(op + 2048 * u + col1) =
              make_uint4(mul_h2(hi.x, f), mul_h2(hi.y, f), mul_h2(hi.z, f), mul_h2(hi.w, f));
        }
      }
      arrive();
      if (lane == 0) mbar_arrive(&bar[B_CEMPTY + p * kCodeStages + cs]);  // (all lanes have read theirs: arrive() syncs)
      if (++cs == kCodeStages) cs = 0, cp ^= 1;
    }
    // (whatever `ok`: the plane's warps meet here)
    for (int tt = 0; tt < nt; ++tt) {
      uint4 raw[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) own_row(tt, u, raw[u]);
      uint32_t big[4];  // of the thread's half pieces of four rows, then of the warp's
      uint32_t wild = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint4 r = raw[u][hh];
          m = max_abs_nan<T>(max_abs_nan<T>(max_abs_nan<T>(max_abs_nan<T>(m, r.x), r.y), r.z), r.w);
        }
        big[u] = max(m & 0xffffu, m >> 16);
        wild |= big[u] >= inf_bits<T>() ? 1u << u : 0u;
      }
      if (wild) {  // (rare) infinities or NaN
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (!(wild >> u & 1u)) continue;
          uint32_t m = 0;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            finite_only<T>(raw[u][hh]);
            m = max_abs2(max_abs2(max_abs2(max_abs2(m, raw[u][hh].x), raw[u][hh].y), raw[u][hh].z), raw[u][hh].w);
          }
          big[u] = max(m & 0xffffu, m >> 16);
          const int node = kKeys * tt + 16 * u + kr;
          if (p) atomicOr(&s_vbad[node >> 5], 1u << (node & 31));
        }
      }
      // four lanes have pieces of a row in this warp, four more in its neighbour
      uint32_t* const red = reinterpret_cast<uint32_t*>(smem + M::row) + 128 * p;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        big[u] = max(big[u], __shfl_xor_sync(0xffffffffu, big[u], 8));
        big[u] = max(big[u], __shfl_xor_sync(0xffffffffu, big[u], 16));
        if (lane < 8) red[64 * (wv & 1) + 16 * u + kr] = big[u];
      }
      sync_converters(p);
      // (every warp alike) the rows' exponents; rows of zeros take the tile's
      int e[2], most = -1000, least = 1000;
      bool zero[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint16_t bits = (uint16_t)max(red[lane + 32 * k], red[64 + lane + 32 * k]);
        e[k] = shift_of(to_f32<T>(*reinterpret_cast<const T*>(&bits)), p ? -80 : -120);
        zero[k] = bits == 0;
        most = zero[k] ? most : max(most, e[k]);
        least = zero[k] ? least : min(least, e[k]);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      least = __reduce_min_sync(0xffffffffu, least);
      if (most == -1000) most = 0;
      const bool keyed = most - least > kRowSpread;
      if (wv == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          smem[M::own + 128 * p + kKeys * tt + lane + 32 * k] = (uint8_t)(127 + (keyed && !zero[k] ? e[k] : most));
        // (K's sign, V's 1024: the keys have exponents of their own)
        if (lane == 0) (&s_unit[np + tt].x)[p] = p ? (float)(keyed ? most + 1024 : most) : keyed ? -pow2i(most) : pow2i(most);
      }
      sync_converters(p);  // (also: everyone has read `red`)
      if (lane == 0) mbar_arrive(&bar[B_TREF + tt]);
    }
    for (int tt = 0; tt < nt && ok; ++tt) {
      uint8_t* const op = enter();
      if (!ok) break;
      // V's infinities and NaN become 0, because 0 * NaN would reach rows that do not see them; they are added at
      // the end
      const bool wild = p && (s_vbad[2 * tt] | s_vbad[2 * tt + 1]);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint4 raw[2];
        own_row(tt, u, raw);
        const float f = pow2i(127 - (int)smem[M::own + 128 * p + kKeys * tt + 16 * u + kr]);
        if (wild) {
          finite_only<T>(raw[0]);
          finite_only<T>(raw[1]);
        }
        float v[8];
        unpack8<T>(raw[0], v);
        *reinterpret_cast<uint4*>(op + 2048 * u + col0) = pack8(v, f);
        unpack8<T>(raw[1], v);
        *reinterpret_cast<uint4*>(op + 2048 * u + col1) = pack8(v, f);
      }
      arrive();
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ------------------------------------------------------------ softmax rows
    const int t = warp >> 2;                 // stream
    const int r = (warp & 3) * 32 + lane;    // TMEM lane
    const bool warp_on = __any_sync(0xffffffffu, row0 + r < rows);
    // what the row sees of the step's own rows, in the last of the rounds' buffers
    bool ok = true;
    auto seen = [&](uint64_t& lo, uint64_t& hi) {  // (after B_ANC, or a barrier with warps that waited for it)
      const int node = row0 + r < rows ? by_g(row0 + r) : 0;
      if (a.parents) {
        const ulonglong2 set = s_anc[128 * ((32 - __clz(top)) & 1) + node];
        lo = set.x, hi = set.y;
      } else {
        lo = node >= 63 ? ~0ull : (2ull << node) - 1;
        hi = node < 64 ? 0 : node >= 127 ? ~0ull : (2ull << (node - 64)) - 1;
      }
    };
    // q as fp16 into tensor memory, half a row per thread: bf16 rows times a power of two (see shift_of), which the
    // largest finite value of both halves sets
    float* const s_half = reinterpret_cast<float*>(smem + M::half);
    float qs = a.scale * 1.4426950408889634f;
    {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(smem + M::q + (16 * warp + 2 * i + (lane >> 4)) * kQPitch + 16 * (lane & 15)) = qraw[i];
      sync_rows();
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 y = *reinterpret_cast<const uint4*>(smem + M::q + r * kQPitch + 128 * t + 16 * i);
        w[4 * i] = y.x, w[4 * i + 1] = y.y, w[4 * i + 2] = y.z, w[4 * i + 3] = y.w;
      }
      if (!__is_same(T, __half)) {
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) big = max_abs_nan<T>(big, w[i]);
        big = max(big & 0xffffu, big >> 16);
        if (big >= inf_bits<T>()) {  // (rare) of the finite ones
          big = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
            big = max(big, max(lo < inf_bits<T>() ? lo : 0u, hi < inf_bits<T>() ? hi : 0u));
          }
        }
        s_half[tid] = __uint_as_float(big << 16);
        sync_rows();
        const int shift = shift_of(fmaxf(s_half[tid], s_half[tid ^ 128]));
        const float f = pow2i(-shift);
        qs *= pow2i(shift);
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pack2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
      }
      tmem_st32_async(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColQ + 32 * t, w);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_Q]);
    }
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);  // this warp's lanes
    const uint32_t to = tl + 128 * t;                                 // the stream's O
    int sb = t;                                                       // the unit's S buffer
    const int n_own = (nu - t + 1) >> 1;  // the stream's units
    float m = -INFINITY, l = 0.f, lr = 0.f;  // lr: of the rounded probabilities
    float top_w = -INFINITY;                 // the largest w so far
#pragma unroll 1
    for (int i = 0; i < n_own; ++i) {
      const int u = 2 * i + t, eo = 2 * t + (i & 1), ph = (i >> 1) & 1;  // its barrier and phase
      const uint32_t ts = tl + kColS + kKeys * sb;
      uint64_t see = ~0ull;  // keys of the unit that the row sees
      if (u >= np - 1) {
        if (u >= np) {
          if (ok) ok = held(B_TREF + u - np, 0) && (!a.parents || held(B_ANC, 0));
          uint64_t lo, hi;
          seen(lo, hi);
          see = u == np ? lo : hi;
        } else {
          const int left = c1 - (c0 + kKeys * u);
          if (left < kKeys) see = (1ull << left) - 1;
        }
      }
      const float2 e = s_unit[u];
      // (a factor that vanishes would turn hidden keys' -inf into NaN)
      const float f = fabsf(qs * e.x) < 0x1p-126f ? 0x1p-126f : qs * e.x, ve = e.y;
      if (ok) ok = held(B_SFULL + eo, ph);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && warp_on) {
        tc_fence_after();
        const bool keyed = e.x < 0.f || ve > 512.f;  // (of all threads alike, `apart` too)
        const bool apart = keyed || ve < top_w - kFar;
        top_w = fmaxf(top_w, ve > 512.f ? ve - 1024.f : ve);
        // twice through the scores, 32 at a time: the largest first
        const bool masked = __any_sync(0xffffffffu, see != ~0ull);
        auto scores = [&](int c, uint32_t (&s)[32]) {
          tmem_ld32_async(ts + 32 * c, s);
          tmem_wait_ld();
          tmem_reg_fence32(s);
          if (masked) {
            const uint32_t w = (uint32_t)(see >> (32 * c));
#pragma unroll
            for (int q = 0; q < 32; ++q) s[q] = (w >> q & 1u) ? s[q] : 0xff800000u;
          }
        };
        // exponent bytes of the unit's K, one per 16 keys or per own row; those of V lie as far behind as their arrays
        const uint8_t* const bytes = !keyed ? nullptr : smem + (u < np ? M::kexp + 4 * u : M::own + kKeys * (u - np));
        float mx = -INFINITY;
        if (__builtin_expect(keyed, 0)) {
          mx = unit_apart<false>(ts, see, bytes, u < np, qs, ve, 0.f);
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32];
            scores(c, s);
            float m0 = __uint_as_float(s[0]), m1 = __uint_as_float(s[1]);
#pragma unroll
            for (int q = 2; q < 30; q += 4) {
              m0 = fmax3(m0, __uint_as_float(s[q]), __uint_as_float(s[q + 1]));
              m1 = fmax3(m1, __uint_as_float(s[q + 2]), __uint_as_float(s[q + 3]));
            }
            mx = fmax3(mx, fmax3(m0, __uint_as_float(s[30]), __uint_as_float(s[31])), m1);
          }
          mx = fmaf(mx, f, ve);
        }
        const float unit_max = mx;
        const bool up = mx > m + 15.f;
        if (__any_sync(0xffffffffu, up)) {
          mx -= 7.f;
          const float half = up ? fast_exp2(0.5f * (m - mx)) : 1.f, keep = half * half;
          m = up ? mx : m;
          l = l * half * half;
          lr = lr * half * half;
          if (i > 0) {
            // O shrinks: the product of the stream's last unit has to be in it
            ok = __all_sync(0xffffffffu, held(B_PV + 2 * t + ((i - 1) & 1), ((i - 1) >> 1) & 1));
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                float o[16];
                tmem_ld16(to + 16 * c, o);
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] *= keep;
                tmem_st16_async(to + 16 * c, reinterpret_cast<const uint32_t*>(o));
              }
              tmem_wait_st();
            }
          }
        }
        const float m0 = m == -INFINITY ? 0.f : m, add = ve - m0;
        if (__builtin_expect(!apart, 1)) {
          const uint64_t f2 = f2_pack(f, f), a2 = f2_pack(add, add);
          uint64_t l0 = f2_pack(0.f, 0.f);
          float r0 = 0.f, r1 = 0.f;  // of the rounded probabilities
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32], p[16];
            scores(c, s);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              float y0, y1;
              f2_unpack(f2_fma(u2_pack(s[2 * q], s[2 * q + 1]), f2, a2), y0, y1);
              y0 = fast_exp2(y0);
              y1 = fast_exp2(y1);
              l0 = f2_add(l0, f2_pack(y0, y1));
              p[q] = pack2(y0, y1);
              r0 = add_half(r0, (uint16_t)(p[q] & 0xffffu));
              r1 = add_half(r1, (uint16_t)(p[q] >> 16));
            }
            tmem_st16_async(ts + 16 * c, p);  // over scores that have been read
          }
          float s0, s1;
          f2_unpack(l0, s0, s1);
          const float un = fast_exp2(kLift - ve);
          l = fmaf(s0 + s1, un, l);
          // (where all of a unit's p' are below 1, which is far below the largest: values of a small scale, whose p' may
          // have lost bits that 2^-w makes matter, and whose weight in O is small)
          lr = fmaf(unit_max < m ? s0 + s1 : r0 + r1, un, lr);
        } else {
          const float sum = unit_apart<true>(ts, see, bytes, u < np, keyed ? qs : f, ve, m0);
          l += sum;
          lr += sum;
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_PFULL + eo]);
      if ((sb += 2) >= kScores) sb -= kScores;
    }
    if (ok && nu > 0) ok = held(B_O, 0);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *abort_flag = 1;
    int place = row0 + r;
    asm volatile("" : "+r"(place));  // (computed here: a register less in the loop)
    const int qr = place;
    const bool row_ok = qr < rows;
    const int node = row_ok ? by_g(qr) : 0;
    // normalised output of this stream; two streams of the same rows join in the first one.  It is written out, or
    // staged over operands that are done with (B_O follows every MMA) where a cluster shares the prefix.
    // (2^kLift, and a quarter until the end: 448 * 2^120 is more than a float holds, a share of it may not be)
    float inv = !ok ? NAN : l == 0.f ? 0.f : 1024.f / lr;
    float lse = !ok ? NAN : l == 0.f ? -INFINITY : kv8_log2_sum(m - kLift, l);
    const bool o_on = ok && n_own > 0;  // (uniform: else O was never written)
    if (o_on) tc_fence_after();
    const uint32_t sw = (uint32_t)(r & 7) << 4;
    uint8_t* const stg = smem + M::stage + r * 512;
    uint8_t* const swap = smem + M::stage + kRowTile * 512 + r * 256;
    auto read_o = [&](int c, float (&o)[32]) {
      if (o_on) {
        uint32_t w[32];
        tmem_ld32_async(to + 32 * c, w);
        tmem_wait_ld();
        tmem_reg_fence32(w);
#pragma unroll
        for (int q = 0; q < 32; ++q) o[q] = __uint_as_float(w[q]) * inv;
      } else {
#pragma unroll
        for (int q = 0; q < 32; ++q) o[q] = ok ? 0.f : NAN;
      }
    };
    // each stream joins half of the dimensions, 64 t ..: the other half goes to the other one
    if (warp_on) {
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float o[32];
        read_o(2 * (t ^ 1) + c, o);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(swap + (t ^ 1) * kRowTile * 256 + (((8 * c + q) << 4) ^ sw)) =
              make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      }
    }
    s_half[tid] = lse;
    sync_rows();
    float w1 = 0.f;
    {
      const float other = s_half[tid ^ 128], mx = fmaxf(lse, other);
      const float a0 = lse == -INFINITY ? 0.f : fast_exp2(lse - mx), a1 = other == -INFINITY ? 0.f : fast_exp2(other - mx);
      const float sum = a0 + a1, is = sum == 0.f ? 0.f : 1.f / sum;
      inv *= a0 * is;
      w1 = a1 * is;
      lse = sum == 0.f ? -INFINITY : mx + log2f(sum);
    }
    if (warp_on) {
      const bool wild = nt > 0 && (s_vbad[0] | s_vbad[1] | s_vbad[2] | s_vbad[3]);
#pragma unroll 1
      for (int c = 2 * t; c < 2 * t + 2; ++c) {
        float o[32];
        read_o(c, o);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 y = *reinterpret_cast<const float4*>(swap + t * kRowTile * 256 + (((8 * (c & 1) + q) << 4) ^ sw));
          o[4 * q] = fmaf(w1, y.x, o[4 * q]);
          o[4 * q + 1] = fmaf(w1, y.y, o[4 * q + 1]);
          o[4 * q + 2] = fmaf(w1, y.z, o[4 * q + 2]);
          o[4 * q + 3] = fmaf(w1, y.w, o[4 * q + 3]);
        }
        if (wild && row_ok) {  // infinities and NaN in V of the step's own rows, for the rows that see them
          uint64_t anc0, anc1;
          seen(anc0, anc1);
#pragma unroll 1
          for (int k = 0; k <= top; ++k) {
            if (!(s_vbad[k >> 5] >> (k & 31) & 1u)) continue;
            if (!((k < 64 ? anc0 >> k : anc1 >> (k - 64)) & 1)) continue;
            const T* vp = reinterpret_cast<const T*>(a.v_new) + a.v_row_stride * (first + k) + a.v_head_stride * kvh + 32 * c;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const float v = to_f32<T>(vp[q]);
              if (!(fabsf(v) < INFINITY)) o[q] += v;
            }
          }
        }
        if (pl.chunks == 1) {  // rounded, so that rows can be written in whole
          uint4 w[4];
          T* e = reinterpret_cast<T*>(w);
#pragma unroll
          for (int q = 0; q < 32; ++q) e[q] = from_f32<T>(4.f * o[q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(smem + M::stage + r * 256 + (((4 * c + q) << 4) ^ sw)) = w[q];
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(stg + (((8 * c + q) << 4) ^ sw)) =
                make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (t == 0 && pl.chunks > 1) s_row[r] = lse;
      else if (t == 0 && row_ok && a.lse)
        a.lse[(size_t)(first + node) * a.n_q_heads + kvh * G + (qr - node * G)] = lse * 0.69314718055994531f;
    }
    if (pl.chunks == 1) {
      sync_rows();
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {  // half a warp per row
        const int rr = 16 * warp + 2 * i + (lane >> 4), q2 = row0 + rr, node2 = by_g(q2);
        const uint4 w = *reinterpret_cast<const uint4*>(smem + M::stage + rr * 256 + (((lane & 15) << 4) ^ ((rr & 7) << 4)));
        if (q2 < rows)
          *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + a.out_row_stride * (first + node2) +
                                    (size_t)(kvh * G + (q2 - node2 * G)) * kKv8Hd + 8 * (lane & 15)) = w;
      }
    }
  }

  if (pl.chunks > 1) {
    // merge: every CTA of the cluster writes a slice of the rows, from all CTAs' parts of them
    cluster_sync_all();
    const int valid = min(kRowTile, rows - row0);
    const int per_cta = (int)__umulhi((uint32_t)(valid + pl.chunks - 1), pl.by_chunks);
    const int rb = share * per_cta, re = min(valid, rb + per_cta);
    const uint32_t row_base = smem_u32(s_row), stage_base = smem_u32(smem + M::stage);
    static_assert(kKv8TcMaxChunks == 8, "two loads of four parts");
    // half a warp per row, dimensions 4 l .. and 64 + 4 l .. per lane
    const int l16 = lane & 15;
    for (int r2 = rb + 2 * warp; r2 < re; r2 += kThreads / 16) {
      const int rr = min(re - 1, r2 + (lane >> 4));
      const int q2 = row0 + rr, node = by_g(q2);
      const uint32_t s0 = stage_base + (uint32_t)(rr * 512 + ((l16 ^ (rr & 7)) << 4)), s1 = s0 + 256;
      // lane k of the half has part k's log-sum-exp
      float x = -INFINITY;
      if (l16 < pl.chunks) x = dsmem_ld_f32(map_peer(row_base + 4 * rr, l16));
      float4 y[4][2];
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[k][0] = dsmem_ld_f4(map_peer(s0, min(k0 + k, pl.chunks - 1)));
          y[k][1] = dsmem_ld_f4(map_peer(s1, min(k0 + k, pl.chunks - 1)));
        }
      };
      load(0);
      float mx = x;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float w = x == -INFINITY ? 0.f : fast_exp2(x - mx);
      float sum = w;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w *= sum == 0.f ? 0.f : 1.f / sum;
      const bool mine = r2 + (lane >> 4) < re;
      if (a.lse && l16 == 0 && mine)
        a.lse[(size_t)(first + node) * a.n_q_heads + kvh * G + (q2 - node * G)] =
            sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll 1
      for (int k0 = 0; k0 < pl.chunks; k0 += 4) {
        if (k0) load(k0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (lane & 16) + k0 + k);  // (0 beyond the last part)
          const float4 u = y[k][0], v = y[k][1];
          o[0] = fmaf(wk, u.x, o[0]), o[1] = fmaf(wk, u.y, o[1]), o[2] = fmaf(wk, u.z, o[2]), o[3] = fmaf(wk, u.w, o[3]);
          o[4] = fmaf(wk, v.x, o[4]), o[5] = fmaf(wk, v.y, o[5]), o[6] = fmaf(wk, v.z, o[6]), o[7] = fmaf(wk, v.w, o[7]);
        }
      }
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(4.f * o[i]);
      if (mine) {
        T* const to = reinterpret_cast<T*>(a.out) + a.out_row_stride * (first + node) +
                      (size_t)(kvh * G + (q2 - node * G)) * kKv8Hd + 4 * l16;
        *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(e);
        *reinterpret_cast<uint2*>(to + 64) = *reinterpret_cast<const uint2*>(e + 4);
      }
    }
  }
  tc_fence_before();
  // no CTA leaves while a peer reads it (what was read has been used: nothing to order but the barrier itself)
  if (pl.chunks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  else __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T>
cudaLaunchConfig_t tree_config(dim3 grid, int chunks, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = M::dyn;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = chunks;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chunks > 1 ? 1 : 0;
  return cfg;
}

template <typename T>
cudaError_t launch_tree(const Kv8View& c, const spec_kv8_attention_args& a, const TcPlan& p, int row_tiles,
                        cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = tree_config<T>(dim3(p.chunks * row_tiles, c.hkv, a.batch), p.chunks, attr);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kv8_tree_kernel<T>, c, a, p);
}

template <typename T>
cudaError_t configure_tree(int sm_count, int* clusters) {
  cudaError_t e = cudaFuncSetAttribute(kv8_tree_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)M::dyn);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv8_tree_kernel<T>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
  // how many clusters of n CTAs the GPU holds at once
  clusters[0] = 0, clusters[1] = sm_count;
  for (int n = 2; n <= kKv8TcMaxChunks && e == cudaSuccess; ++n) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = tree_config<T>(dim3(n), n, attr);
    e = cudaOccupancyMaxActiveClusters(&clusters[n], kv8_tree_kernel<T>, &cfg);
  }
  return e;
}

}  // namespace

cudaError_t kv8_tree_configure(int sm_count, int* clusters) {
  const cudaError_t e = configure_tree<__nv_bfloat16>(sm_count, clusters);
  return e == cudaSuccess ? configure_tree<__half>(sm_count, clusters) : e;
}

cudaError_t launch_kv8_tree(const Kv8View& c, const spec_kv8_attention_args& a, const int* clusters, cudaStream_t s) {
  const int G = a.n_q_heads / c.hkv;
  const int row_tiles = (a.max_nodes * G + kRowTile - 1) / kRowTile;
  const long long tiles = (long long)a.batch * c.hkv * row_tiles;
  const int units = (a.max_prefix + kKeys - 1) / kKeys;
  // The CTAs of a cluster share a prefix where that is sooner done: rounds of clusters that the GPU holds at once, each
  // as long as a share's units and a cluster's start, join and end, all in units of 0.6 us.  Measured with bf16 trees, us:
  //   CTAs of a cluster (clusters at once)   1 (148)  2 (74)  3 (45)  4 (33)  5 (26)  6 (22)  7 (15)  8 (15)
  //    8 tiles, 2048 tokens                    28.8    20.9    17.6    15.3    17.1    15.8    14.3    13.6
  //   16 tiles, 1024 tokens                    19.3    17.4    15.7    13.3    17.4    16.1    27.1    25.2
  //   16 tiles, 8192 tokens                    86.5    51.2    38.1    30.7    31.2    28.5    47.0    43.1
  //   64 tiles, 4096 tokens                    49.0    33.4    50.6    43.7    70.2    63.2    90.3    82.7
  // More tiles than SMs have a CTA each: ragged batches have fewer and shorter ones than the bounds say (10 trees of
  // 16 - 61 over 512 - 4096 tokens, 160 tiles by their bounds: 51 us with one, 60 with two; equal ones 101 with either).
  static constexpr int kEnds[kKv8TcMaxChunks + 1] = {0, 15, 19, 18, 17, 22, 21, 18, 17};
  const int least = a.max_prefix > kKv8TcMaxKeys ? (a.max_prefix + kKv8TcMaxKeys - 1) / kKv8TcMaxKeys : 1;
  TcPlan p;
  p.chunks = least;
  long long best = -1;
  for (int n = least; n <= (tiles > clusters[1] ? least : kKv8TcMaxChunks); ++n) {
    if (clusters[n] < 1) continue;
    const long long cost = (tiles + clusters[n] - 1) / clusters[n] * (kEnds[n] + (units + 2 + n - 1) / n);
    if (best < 0 || cost < best) best = cost, p.chunks = n;
  }
  // more tiles than SMs start with the longest prefixes (16 trees, 192 tiles of 630 - 4096 tokens: 78 us, 82 in the
  // batch's order)
  p.by_length = a.batch > 1 && a.batch <= kByLength && tiles > clusters[1];
  p.by_chunks = (uint32_t)((((uint64_t)1 << 32) + p.chunks - 1) / p.chunks);
  p.by_group = (uint32_t)(((1u << 20) + G - 1) / G);
  return a.dtype == SPEC_DTYPE_BF16 ? launch_tree<__nv_bfloat16>(c, a, p, row_tiles, s)
                                    : launch_tree<__half>(c, a, p, row_tiles, s);
}

}  // namespace spec
