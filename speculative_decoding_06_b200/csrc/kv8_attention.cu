// Attention over the 8-bit paged cache for few rows per kv head (plain decoding,
// short chains and trees).
//
// Rows: the G = Hq / Hkv query heads of a kv head, for every row of an entry,
// share that head's keys, so row r = node * G + g of a tile of 8 or 16 rows reads
// each K/V byte once.  With few rows the work is bound by those bytes (256 per key
// and head), not by arithmetic, so a warp keeps everything but the stream of
// codes in registers:
//
//   scores   S^T = K Q^T by mma.m16n8k16: 16 keys by 8 rows.  The contraction's
//            order is free, so lane (g, t) takes dimensions 32t .. 32t + 31 of keys
//            g and g + 8: whole 16-byte pieces, each word of codes (4 dims) one
//            k-step's two A registers after e4m3 -> fp16 conversion (exact).
//   softmax  in 32 bits, base 2.  A page's K scale multiplies the scores; its
//            V scale 2^w goes into the exponent: p' = 2^(x + w - m), so that O sums
//            p' times bare codes and l sums p' 2^(12 - w).  m is 7 below the row's running
//            maximum of x + w and moves only when exceeded by more than 15: p' <= 2^15,
//            and fp16, to which p' is rounded (2^-11 of itself) for the second product,
//            has its full 11 bits down to 2^-21 of the largest p'.  O is divided by the
//            sum of the rounded p', so that a key's rounding cancels as far as its weight
//            dominates; the log-sum-exp is that of the unrounded ones.  The weights
//            do not depend on V, so l has to hold where p' does not: see kLift and kFar.
//   output   O^T = V^T P^T: lane (g, t) holds dimensions 16g .. 16g+15 of keys 2t,
//            2t+1, 2t+8, 2t+9; two keys' bytes interleave into A registers;
//            the scores' accumulators become the B operand by movmatrix.
//
// Each warp streams tiles of 32 keys through a queue of its own in shared memory,
// two tiles deep, which one lane fills by TMA (boxes of 16 keys, each inside one
// page; the 128-byte swizzle keeps both products' reads free of bank conflicts).
// A batch of 64 at 512 - 4096 tokens (310 MB) takes 61.4 us, 5.0 TB/s, 77 % of the
// measured copy rate, with three CTAs of four warps per SM (60.1 before l was made to hold for
// pages of any scale).  Measured beside each other, 60.5 us: 68 us with three tiles
// and two CTAs, 70 - 110 us with CTAs of two or eight warps, 89 us with sixteen
// cp.async per lane and tile in place of TMA.  Tiles of 16 rows keep some 200 bytes per thread in local memory
// (168 registers for three CTAs per SM): 64 sequences of 2400 tokens with 4 rows of 32 query heads on 8 take
// 94 us, 3.3 TB/s, where 2 rows, tiles of 8, take 68.  The step's own rows (16-bit K and V) are added by
// plain 32-bit arithmetic.  Warps, then the CTAs of a sequence cut into chunks,
// merge their (m, l, O); of the latter the one that arrives last, in chunk order,
// so that results do not depend on the order of arrival.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8.h"

namespace spec {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;          // keys per step of a warp: two groups of 16, each inside one page
constexpr int kStages = 2;
constexpr int kTileBytes = kTile * 2 * kKv8Hd;
constexpr int kMaxChunk = 4096;    // keys of a CTA: its page ids and scales lie in shared memory
constexpr int kGroups = kMaxChunk / 16;
// l is the sum of 2^(x - m + kLift).  With w in [-60, 120] and m 7 to 22 below the largest x + w, its largest term lies
// between 2^-101 and 2^87: the sum neither overflows nor loses terms above 2^-25 of the largest.
constexpr float kLift = 12.f;
// Keys whose w is that far below the largest so far may have p' = 0 for weights that count in l: l then takes the weights
// themselves.  (A weight of 2^-43 of the largest has p' of 2^-126 or more at this distance.)
constexpr float kFar = 90.f;

// Workspace: arrival counters at its start, wherever a call's bounds put the rest, so that they are zero between calls
// of any bounds; then (m, l) and O of every (group, chunk).
constexpr int kMaxGroups = 16384;  // groups (sequence, kv head, row tile) of one launch
static_assert(4 * kMaxGroups == SPEC_KV8_WORKSPACE_ZERO, "counters");
struct DecodePlan {
  int chunk, chunks, row_tiles;
  int group0, groups;  // of this launch, of all
  int* counters;       // [kMaxGroups]
  float2* ml;          // [group][chunk][rows]
  float* part;         // [group][chunk][rows][128]
};

struct Smem {
  static constexpr int ring = 0;
  static constexpr int page = ring + kWarps * kStages * kTileBytes;  // int [kGroups]: offset of a group's first row / 16
  static constexpr int kscale = page + 4 * kGroups;                  // float [kGroups]: 2^e of K, NaN: no such page
  static constexpr int vexp = kscale + 4 * kGroups;                  // float [kGroups]: e of V
  static constexpr int anc = vexp + 4 * kGroups;                     // uint64 [16 rows][2]
  static constexpr int bars = anc + 16 * 16;                          // uint64 [kWarps][kStages]
  static constexpr int misc = bars + 8 * kWarps * kStages;
  static constexpr int end = misc + 16;
  static constexpr int dyn = end + 1024;                              // to a 1024-byte boundary (the swizzle's atom)
};

// two e4m3 codes (low byte first) as two fp16: exact
__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t w16) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w16));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ float finite_abs(float x) {
  const float m = fabsf(x);
  return m < INFINITY ? m : 0.f;
}

// Sixteen values of a 16-bit row as 32-bit floats.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p) + h);
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * h + i] = to_f32<T>(e[i]);
  }
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 3) kv8_decode_kernel(const __grid_constant__ CUtensorMap map, Kv8View c,
                                                              spec_kv8_attention_args a, DecodePlan pl) {
  extern __shared__ uint8_t smem_raw[];
  // (to a 1024-byte boundary by an offset, so that the compiler still knows what it points to as shared memory)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  int* s_page = reinterpret_cast<int*>(smem + Smem::page);
  float* s_kscale = reinterpret_cast<float*>(smem + Smem::kscale);
  float* s_vexp = reinterpret_cast<float*>(smem + Smem::vexp);
  uint64_t* s_anc = reinterpret_cast<uint64_t*>(smem + Smem::anc);
  int* s_last = reinterpret_cast<int*>(smem + Smem::misc);
  constexpr int kRows = 8 * NT;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = a.n_q_heads / c.hkv;
  const int group = blockIdx.x / pl.chunks, chunk_i = blockIdx.x - group * pl.chunks;  // (group of the launch)
  const int bk = (pl.group0 + group) / pl.row_tiles, row0 = (pl.group0 + group - bk * pl.row_tiles) * kRows;
  const int b = bk / c.hkv, kvh = bk - b * c.hkv;
  const int first = a.offsets[b], n = a.offsets[b + 1] - first;
  const int seq = a.seq_ids ? a.seq_ids[b] : b;
  if (a.fill && row0 == 0 && chunk_i == 0) kv8_fill_rows(a, b, kvh, G);
  if (seq < 0 || seq >= a.n_seqs || first < 0 || n < 1 || n > a.max_nodes || n > a.rows - first) return;
  const int P = a.lengths[seq];
  const int rows = n * G;
  if (P < 0 || P > a.max_prefix || row0 >= rows) return;
  const int nc = max(1, (P + pl.chunk - 1) / pl.chunk);
  if (chunk_i >= nc) return;
  const int c0 = chunk_i * pl.chunk, c1 = min(P, c0 + pl.chunk);
  const int ngroups = (c1 - c0 + 15) >> 4;
  const int ntiles = (c1 - c0 + kTile - 1) / kTile;

  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + Smem::bars) + warp * kStages;
  if (lane < kStages) mbar_init(&full[lane], 1);
  fence_barrier_init();
  // pages of the chunk's groups of 16 keys
  for (int i = tid; i < 2 * ntiles; i += kThreads) {
    const int key = c0 + 16 * i;
    int pg = 0;
    float ks = 0.f, ve = 0.f;
    if (i < ngroups) {
      pg = a.tables[(size_t)seq * a.max_blocks + (key >> c.page_log2)];
      const bool ok = pg >= 0 && pg < c.n_pages;
      if (!ok) pg = 0;
      const size_t at = (size_t)pg * c.hkv + kvh;
      const int kb = ok ? c.exps[0][at] : 255, vb = c.exps[1][at];  // 255: NaN
      ks = kb < 255 ? __int_as_float(kb << 23) : NAN;
      ve = vb < 255 ? (float)(vb - 127) : NAN;
    }
    s_page[i] = (((pg * c.hkv + kvh) << c.page_log2) + (key & (c.page - 1))) >> 4;
    s_kscale[i] = ks;
    s_vexp[i] = ve;
  }
  // ancestors of the tile's rows among the step's rows (itself included)
  if (a.k_new && tid < kRows) {
    uint64_t lo = 0, hi = 0;
    if (row0 + tid < rows) {
      int j = (row0 + tid) / G;
      if (!a.parents) {
        lo = j >= 63 ? ~0ull : (2ull << j) - 1;
        hi = j < 64 ? 0 : j >= 127 ? ~0ull : (2ull << (j - 64)) - 1;
      } else {
        while (j >= 0) {
          if (j < 64) lo |= 1ull << j;
          else hi |= 1ull << (j - 64);
          const int up = a.parents[first + j];
          j = up < j ? up : -1;
        }
      }
    }
    s_anc[2 * tid] = lo;
    s_anc[2 * tid + 1] = hi;
  }
  // this lane's part of q, as fp16 pieces of row g (+ 8): bf16 rows are scaled by a
  // power of two that puts their largest value near 2^8 (fp16 then holds every value
  // down to 2^-32 of it)
  uint32_t qf[NT][16];
  float qs[NT];  // row g's factor, with scale * log2(e)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + 8 * nt + g;
    const int rr = min(r, rows - 1);
    const int node = rr / G;
    const T* p = reinterpret_cast<const T*>(a.q) + a.q_row_stride * (first + node) +
                 a.q_head_stride * (kvh * G + (rr - node * G)) + 32 * t;
    float v[32];
    load16(p, reinterpret_cast<float(&)[16]>(v[0]));
    load16(p + 16, reinterpret_cast<float(&)[16]>(v[16]));
    int ex = 0;
    if (sizeof(T) == 2 && !__is_same(T, __half)) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = fmaxf(m, finite_abs(v[i]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      ex = max(-120, min(120, (__float_as_int(m) >> 23) - 127 - 8));
    }
    const float f = __int_as_float((127 - ex) << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i] * f, v[2 * i + 1] * f);
      qf[nt][i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    qs[nt] = a.scale * 1.4426950408889634f * __int_as_float((127 + ex) << 23);
  }
  // the factors of this lane's accumulator columns, rows 2t and 2t + 1
  float qc[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    qc[nt][0] = __shfl_sync(0xffffffffu, qs[nt], 8 * t);
    qc[nt][1] = __shfl_sync(0xffffffffu, qs[nt], 8 * t + 4);
  }
  __syncthreads();

  uint8_t* const ring = smem + Smem::ring + warp * (kStages * kTileBytes);
  const int mine = ntiles > warp ? (ntiles - warp + kWarps - 1) / kWarps : 0;
  // tile i of this warp: K of two groups of 16 keys, then V
  auto fetch = [&](int i) {
    if (lane == 0 && i < mine) {
      const int st = i % kStages, g0 = 2 * (warp + kWarps * i);
      const uint64_t pol = policy_evict_first();
      mbar_arrive_expect_tx(&full[st], kTileBytes);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tma_load_2d(ring + st * kTileBytes + q * 2048, &map, &full[st], 0, c.row0[q >> 1] + 16 * s_page[g0 + (q & 1)], pol);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) fetch(i);
  // where lane (g, t) finds its pieces: row g of K, pieces 2t and 2t + 1; rows 2t, 2t + 1, + 8, + 9 of V, piece g
  const int k_at0 = g * 128 + (((2 * t) ^ g) << 4), k_at1 = g * 128 + (((2 * t + 1) ^ g) << 4);
  const int v_at0 = 2 * t * 128 + ((g ^ (2 * t)) << 4), v_at1 = (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4);

  float m[NT][2], l[NT][2], lr[NT][2], o[NT][8][4];  // lr: the sum of the rounded probabilities
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = lr[nt][0] = lr[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[nt][i][q] = 0.f;
  }
  // a row's running maximum rises to m2: what was summed shrinks
  auto raise = [&](int nt, int col, float m2) {
    const float half = m2 > m[nt][col] ? fast_exp2(0.5f * (m[nt][col] - m2)) : 1.f;
    const float keep = half * half;
    m[nt][col] = fmaxf(m[nt][col], m2);
    l[nt][col] = l[nt][col] * half * half;
    lr[nt][col] = lr[nt][col] * half * half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[nt][i][col] *= keep;
      o[nt][i][2 + col] *= keep;
    }
  };

  bool landed = true;
  float top_w = -INFINITY;  // the largest w so far
  for (int i = 0; i < mine; ++i) {
    landed = __all_sync(0xffffffffu, mbar_wait(&full[i % kStages], (i / kStages) & 1, nullptr, nullptr));
    if (!landed) {  // a wait ran out: copies under way land before the CTA's memory is released, and the rows say so
      for (int k = i + 1; k < min(mine, i + kStages); ++k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, nullptr, nullptr);
      break;
    }
    const uint8_t* const buf = ring + (i % kStages) * kTileBytes;
    auto piece = [&](int at) { return *reinterpret_cast<const uint4*>(buf + at); };
    const int g0 = 2 * (warp + kWarps * i);
    float s[2][NT][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 ka0 = piece(2048 * u + k_at0), ka1 = piece(2048 * u + k_at1);                // key g
      const uint4 kb0 = piece(2048 * u + 1024 + k_at0), kb1 = piece(2048 * u + 1024 + k_at1);  // key g + 8
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t wa = word(ks < 4 ? ka0 : ka1, ks & 3), wb = word(ks < 4 ? kb0 : kb1, ks & 3);
        const uint32_t a0 = cvt_e4m3x2(wa), a2 = cvt_e4m3x2_hi(wa), a1 = cvt_e4m3x2(wb), a3 = cvt_e4m3x2_hi(wb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(s[u][nt], a0, a1, a2, a3, qf[nt][2 * ks], qf[nt][2 * ks + 1]);
      }
    }
    // x + w in base 2, hidden keys at -inf
    const float ks0 = s_kscale[g0], ks1 = s_kscale[g0 + 1], ve0 = s_vexp[g0], ve1 = s_vexp[g0 + 1];
    const int left = c1 - (c0 + 16 * g0);  // keys of the tile that exist
    const float low_w = left > 16 ? fminf(ve0, ve1) : ve0;
    top_w = fmaxf(top_w, left > 16 ? fmaxf(ve0, ve1) : ve0);
    const bool far = low_w < top_w - kFar;
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float ks = u ? ks1 : ks0, ve = u ? ve1 : ve0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float x = fmaf(s[u][nt][q], qc[nt][q & 1] * ks, ve);
          s[u][nt][q] = 16 * u + g + (q >> 1) * 8 < left ? x : -INFINITY;
        }
      }
      bool up = false;
      float mx[2];
#pragma unroll
      for (int col = 0; col < 2; ++col) {
        float v = fmaxf(fmaxf(s[0][nt][col], s[0][nt][2 + col]), fmaxf(s[1][nt][col], s[1][nt][2 + col]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        mx[col] = v;
        up |= v > m[nt][col] + 15.f;
      }
      if (__any_sync(0xffffffffu, up)) {
        raise(nt, 0, mx[0] - 7.f);
        raise(nt, 1, mx[1] - 7.f);
      }
      const float n0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], n1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float p0 = fast_exp2(s[u][nt][0] - n0), p1 = fast_exp2(s[u][nt][1] - n1);
        const float p2 = fast_exp2(s[u][nt][2] - n0), p3 = fast_exp2(s[u][nt][3] - n1);
        const __half2 lo = __floats2half2_rn(p0, p1), hi = __floats2half2_rn(p2, p3);
        // (below 2^-14 the rounding loses bits that 2^-w may make matter, and the weight in O is small)
        auto kept = [](float p, float rounded) { return p < 0x1p-14f ? p : rounded; };
        const float un = far ? 0.f : fast_exp2(kLift - (u ? ve1 : ve0));
        l[nt][0] = fmaf(p0 + p2, un, l[nt][0]);
        l[nt][1] = fmaf(p1 + p3, un, l[nt][1]);
        lr[nt][0] = fmaf(kept(p0, __low2float(lo)) + kept(p2, __low2float(hi)), un, lr[nt][0]);
        lr[nt][1] = fmaf(kept(p1, __high2float(lo)) + kept(p3, __high2float(hi)), un, lr[nt][1]);
        pb[u][nt][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
        pb[u][nt][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
      }
    }
    if (far) {  // (rare) the weights themselves, as squares: 2^-149 where one exponential ends at 2^-126
#pragma unroll
      for (int i2 = 0; i2 < 8 * NT; ++i2) {
        const int u = i2 & 1, q = i2 >> 1 & 3, nt = i2 >> 3, col = q & 1;
        const float n = m[nt][col] == -INFINITY ? 0.f : m[nt][col];
        const float h = fast_exp2(0.5f * (s[u][nt][q] - n + kLift - (u ? ve1 : ve0)));
        l[nt][col] = fmaf(h, h, l[nt][col]);
        lr[nt][col] = fmaf(h, h, lr[nt][col]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint4 v0 = piece(4096 + 2048 * u + v_at0), v1 = piece(4096 + 2048 * u + v_at1);
      uint4 v2 = piece(5120 + 2048 * u + v_at0), v3 = piece(5120 + 2048 * u + v_at1);
      if (left < 16 * u + 16) {  // what lies behind the sequence's end may be anything: 0 * NaN would spread
        const int k0 = left - 16 * u - 2 * t;
        if (k0 <= 0) v0 = make_uint4(0, 0, 0, 0);
        if (k0 <= 1) v1 = make_uint4(0, 0, 0, 0);
        if (k0 <= 8) v2 = make_uint4(0, 0, 0, 0);
        if (k0 <= 9) v3 = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x0 = word(v0, w), x1 = word(v1, w), x2 = word(v2, w), x3 = word(v3, w);
        const uint32_t e0 = __byte_perm(x0, x1, 0x5140), e1 = __byte_perm(x0, x1, 0x7362);
        const uint32_t f0 = __byte_perm(x2, x3, 0x5140), f1 = __byte_perm(x2, x3, 0x7362);
        const uint32_t a0 = cvt_e4m3x2(e0), a1 = cvt_e4m3x2_hi(e0), a2 = cvt_e4m3x2(f0), a3 = cvt_e4m3x2_hi(f0);
        const uint32_t b0 = cvt_e4m3x2(e1), b1 = cvt_e4m3x2_hi(e1), b2 = cvt_e4m3x2(f1), b3 = cvt_e4m3x2_hi(f1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[nt][2 * w], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
          mma16816(o[nt][2 * w + 1], b0, b1, b2, b3, pb[u][nt][0], pb[u][nt][1]);
        }
      }
    }
    __syncwarp();  // every lane has used what it read: the stage may be filled again
    fetch(i + kStages);
  }
  if (!landed) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) l[nt][0] = l[nt][1] = NAN;
  }

  // the step's own rows: the last chunk's CTA, its warps in turn
  if (a.k_new && chunk_i == nc - 1) {
    // rows of the tile see no row behind the tile's last node
    const int top = min(n - 1, (row0 + kRows - 1) / G);
    for (int j = warp; j <= top; j += kWarps) {
      const T* kp = reinterpret_cast<const T*>(a.k_new) + a.k_row_stride * (first + j) + a.k_head_stride * kvh + 32 * t;
      const T* vp = reinterpret_cast<const T*>(a.v_new) + a.v_row_stride * (first + j) + a.v_head_stride * kvh + 16 * g;
      float k[32], v[16];
      load16(kp, reinterpret_cast<float(&)[16]>(k[0]));
      load16(kp + 16, reinterpret_cast<float(&)[16]>(k[16]));
      load16(vp, v);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&qf[nt][i]));
          // (q goes up to 2^9, k to the end of the floats)
          x = fmaf(q.x, 0x1p-16f * k[2 * i], x);
          x = fmaf(q.y, 0x1p-16f * k[2 * i + 1], x);
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        x *= 0x1p16f * qs[nt];
        const bool sees = (s_anc[2 * (8 * nt + g) + (j >> 6)] >> (j & 63)) & 1;
        x = sees ? x : -INFINITY;
#pragma unroll
        for (int col = 0; col < 2; ++col) {
          const float xc = __shfl_sync(0xffffffffu, x, 8 * t + 4 * col);
          const bool see = __shfl_sync(0xffffffffu, (int)sees, 8 * t + 4 * col);
          if (!see) continue;
          if (xc > m[nt][col] + 15.f) raise(nt, col, xc - 7.f);
          const float y = xc - (m[nt][col] == -INFINITY ? 0.f : m[nt][col]);
          const float p = fast_exp2(y);
          if (g == 0) {  // (nothing is rounded here)
            const float h = fast_exp2(0.5f * (y + kLift));
            l[nt][col] = fmaf(h, h, l[nt][col]);
            lr[nt][col] = fmaf(h, h, lr[nt][col]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[nt][i][col] = fmaf(p, v[2 * i], o[nt][i][col]);
            o[nt][i][2 + col] = fmaf(p, v[2 * i + 1], o[nt][i][2 + col]);
          }
        }
      }
    }
  }

  // merge the warps: (m, l) and O of each into shared memory (the queues are empty)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      l[nt][col] += __shfl_xor_sync(0xffffffffu, l[nt][col], 4);
      l[nt][col] += __shfl_xor_sync(0xffffffffu, l[nt][col], 8);
      l[nt][col] += __shfl_xor_sync(0xffffffffu, l[nt][col], 16);
      lr[nt][col] += __shfl_xor_sync(0xffffffffu, lr[nt][col], 4);
      lr[nt][col] += __shfl_xor_sync(0xffffffffu, lr[nt][col], 8);
      lr[nt][col] += __shfl_xor_sync(0xffffffffu, lr[nt][col], 16);
      // from here on O is of the unrounded sum's size
      const float f = lr[nt][col] == 0.f ? 1.f : l[nt][col] / lr[nt][col];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[nt][i][col] *= f;
        o[nt][i][2 + col] *= f;
      }
    }
  __syncthreads();
  float* s_o = reinterpret_cast<float*>(smem + Smem::ring);             // [warp][rows][132]
  float2* s_ml = reinterpret_cast<float2*>(s_o + kWarps * kRows * 132);  // [warp][rows]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int col = 0; col < 2; ++col) {
      const int r = warp * kRows + 8 * nt + 2 * t + col;
      if (g == 0) s_ml[r] = make_float2(m[nt][col], l[nt][col]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(&s_o[r * 132 + 16 * g + 2 * i]) = make_float2(o[nt][i][col], o[nt][i][2 + col]);
    }
  __syncthreads();
  // a warp per row, a lane per four dimensions
  auto finish = [&](int r, float mm, float ll, float4 acc) {
    const int node = r / G, head = kvh * G + (r - node * G);
    const float inv = ll == 0.f ? 0.f : 4096.f / ll;  // 2^kLift
    T* out = reinterpret_cast<T*>(a.out) + a.out_row_stride * (first + node) + (size_t)head * kKv8Hd + 4 * lane;
    T w[4] = {from_f32<T>(acc.x * inv), from_f32<T>(acc.y * inv), from_f32<T>(acc.z * inv), from_f32<T>(acc.w * inv)};
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(w);
    if (a.lse && lane == 0)
      a.lse[(size_t)(first + node) * a.n_q_heads + head] =
          ll == 0.f ? -INFINITY : kv8_log2_sum(mm - kLift, ll) * 0.69314718055994531f;
  };
  const size_t slot = (size_t)group * pl.chunks + chunk_i;
  for (int r = warp; r < kRows && row0 + r < rows; r += kWarps) {
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w * kRows + r].x);
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 x = s_ml[w * kRows + r];
      const float h = x.x == -INFINITY && x.y == 0.f ? 0.f : fast_exp2(0.5f * (x.x - mm)), f = h * h;
      const float4 v = *reinterpret_cast<const float4*>(&s_o[(w * kRows + r) * 132 + 4 * lane]);
      ll = fmaf(h, h * x.y, ll);
      acc = make_float4(fmaf(f, v.x, acc.x), fmaf(f, v.y, acc.y), fmaf(f, v.z, acc.z), fmaf(f, v.w, acc.w));
    }
    if (nc == 1) {
      finish(row0 + r, mm, ll, acc);
    } else {
      __stcg(reinterpret_cast<float4*>(pl.part + (slot * kRows + r) * kKv8Hd) + lane, acc);
      if (lane == 0) __stcg(&pl.ml[slot * kRows + r], make_float2(mm, ll));
    }
  }
  if (nc == 1) return;
  // the sequence's last CTA to arrive merges the chunks and leaves the counter at zero
  __threadfence();
  __syncthreads();
  if (tid == 0) *s_last = atomicAdd(&pl.counters[group], 1) == nc - 1;
  __syncthreads();
  if (!*s_last) return;
  __threadfence();
  if (tid == 0) pl.counters[group] = 0;
  const size_t slot0 = (size_t)group * pl.chunks;
  for (int r = warp; r < kRows && row0 + r < rows; r += kWarps) {
    float mm = -INFINITY;
    for (int k = lane; k < nc; k += 32) mm = fmaxf(mm, __ldcg(&pl.ml[(slot0 + k) * kRows + r]).x);
    mm = warp_max(mm);
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < nc; ++k) {
      const float2 x = __ldcg(&pl.ml[(slot0 + k) * kRows + r]);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(pl.part + ((slot0 + k) * kRows + r) * kKv8Hd) + lane);
      const float h = x.x == -INFINITY && x.y == 0.f ? 0.f : fast_exp2(0.5f * (x.x - mm)), f = h * h;
      ll = fmaf(h, h * x.y, ll);
      acc = make_float4(fmaf(f, v.x, acc.x), fmaf(f, v.y, acc.y), fmaf(f, v.z, acc.z), fmaf(f, v.w, acc.w));
    }
    finish(row0 + r, mm, ll, acc);
  }
}

// Rows per tile, chunks and workspace for the given bounds.
DecodePlan plan_decode(int hkv, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix, int* nt,
                       size_t* bytes) {
  DecodePlan p{};
  const int rows = max_nodes * (n_q_heads / hkv);
  *nt = rows <= 8 ? 1 : 2;
  p.row_tiles = (rows + 8 * *nt - 1) / (8 * *nt);
  const long long groups = (long long)batch * hkv * p.row_tiles;
  // One round of three CTAs per SM where that makes chunks of up to 2048 keys: a CTA's start, end and partial result
  // take some 5 us (1 x 65536 tokens x 8 heads: 33 us, 43 with chunks of 1024, which are two rounds; 7 x 16385 x 4: 29
  // and 36; the same ragged, 1 - 16385: 24 and 23).  With more work than that, shares of an eighth of an SM's keys, for
  // an even load (prefixes of one length assumed: ragged ones make fewer CTAs).  64 sequences x 8 heads of 512 - 4096
  // tokens: 60.5 us with eighths, 66.6 with quarters, 63.6 with sixteenths.  At least a tile for each warp.
  long long want = groups * max_prefix / (3LL * sm_count);
  if (want > 2048) want = groups * max_prefix / (8LL * sm_count) > 1024 ? groups * max_prefix / (8LL * sm_count) : 1024;
  long long chunk = (want + 127) / 128 * 128;
  chunk = chunk < 128 ? 128 : chunk > kMaxChunk ? kMaxChunk : chunk;
  p.chunk = (int)chunk;
  p.chunks = (int)((max_prefix + chunk - 1) / chunk);
  if (p.chunks < 1) p.chunks = 1;
  p.groups = (int)groups;
  // (a launch's grid stays below 2^30)
  const int per_launch = p.chunks > (1 << 30) / kMaxGroups ? (1 << 30) / p.chunks : kMaxGroups;
  const size_t slots = (size_t)(groups < per_launch ? groups : per_launch) * p.chunks * 8 * *nt;
  p.group0 = per_launch;
  *bytes = p.chunks > 1 ? 4 * kMaxGroups + slots * (kKv8Hd * 4 + 8) : 16;
  return p;
}

bool by_tree(int hkv, int n_q_heads, int max_nodes, int max_prefix) {
  return max_nodes * (n_q_heads / hkv) > 16 && max_prefix <= kKv8TcMaxChunks * kKv8TcMaxKeys;
}

}  // namespace

size_t kv8_attention_need(const Kv8View& c, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix) {
  if (by_tree(c.hkv, n_q_heads, max_nodes, max_prefix)) return 16;
  if ((long long)batch * c.hkv * ((max_nodes * (n_q_heads / c.hkv) + 15) / 16) > kKv8MaxGroups) return 0;
  int nt = 1;
  size_t bytes = 0;
  plan_decode(c.hkv, sm_count, batch, n_q_heads, max_nodes, max_prefix, &nt, &bytes);
  return bytes;
}

// At least what every call needs whose bounds are none of them above these.  With g groups and prefixes of p keys a call
// keeps g * chunks partial results of 8 or 16 rows where it has more than one chunk:
//   chunks of kMaxChunk keys (p above it): g * ceil(p / kMaxChunk), which grows with both;
//   shorter ones: chunks < p / chunk + 1, and chunk is above 1024 / 1025 of g p / (8 SMs) (of g p / (3 SMs), 128 / 129),
//   so that g p / chunk < 9 SMs; more than one chunk means p > chunk and so g < 9 SMs: less than min(g, 9 SMs) + 9 SMs.
// More than 16 rows come here only with prefixes that the tree kernel does not take; below them its calls need nothing,
// but those of fewer rows do.
size_t kv8_attention_workspace(const Kv8View& c, int sm_count, int batch, int n_q_heads, int max_nodes, int max_prefix) {
  const int rows = max_nodes * (n_q_heads / c.hkv);
  const int nt = rows <= 8 ? 1 : 2;
  const int tiles = rows <= 16 || by_tree(c.hkv, n_q_heads, max_nodes, max_prefix) ? 1 : (rows + 15) / 16;
  const long long groups = (long long)batch * c.hkv * tiles, held = groups < kMaxGroups ? groups : kMaxGroups;
  const long long round = 9LL * sm_count;
  long long slots = (groups < round ? groups : round) + round;
  if (max_prefix > kMaxChunk) {
    const long long longest = held * (((long long)max_prefix + kMaxChunk - 1) / kMaxChunk);
    if (longest > slots) slots = longest;
  }
  return 4 * kMaxGroups + (size_t)slots * 8 * nt * (kKv8Hd * 4 + 8);
}

cudaError_t kv8_attention_configure(int sm_count, int* clusters) {
  cudaError_t e = kv8_tree_configure(sm_count, clusters);
  for (const void* f : {(const void*)kv8_decode_kernel<__nv_bfloat16, 1>, (const void*)kv8_decode_kernel<__nv_bfloat16, 2>,
                        (const void*)kv8_decode_kernel<__half, 1>, (const void*)kv8_decode_kernel<__half, 2>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::dyn);
  return e;
}

cudaError_t launch_kv8_attention(const Kv8View& c, const CUtensorMap& map, const spec_kv8_attention_args& a, const int* clusters,
                                 cudaStream_t s) {
  if (by_tree(c.hkv, a.n_q_heads, a.max_nodes, a.max_prefix)) return launch_kv8_tree(c, a, clusters, s);
  int nt = 1;
  size_t bytes = 0;
  DecodePlan p = plan_decode(c.hkv, clusters[1], a.batch, a.n_q_heads, a.max_nodes, a.max_prefix, &nt, &bytes);
  const int per_launch = p.group0;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.counters = reinterpret_cast<int*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + 4 * kMaxGroups);
  p.part = reinterpret_cast<float*>(p.ml + (size_t)(p.groups < per_launch ? p.groups : per_launch) * p.chunks * 8 * nt);
  for (p.group0 = 0; p.group0 < p.groups; p.group0 += per_launch) {
    const unsigned grid = (unsigned)(p.groups - p.group0 < per_launch ? p.groups - p.group0 : per_launch) * p.chunks;
    if (a.dtype == SPEC_DTYPE_BF16) {
      if (nt == 1) kv8_decode_kernel<__nv_bfloat16, 1><<<grid, kThreads, Smem::dyn, s>>>(map, c, a, p);
      else kv8_decode_kernel<__nv_bfloat16, 2><<<grid, kThreads, Smem::dyn, s>>>(map, c, a, p);
    } else {
      if (nt == 1) kv8_decode_kernel<__half, 1><<<grid, kThreads, Smem::dyn, s>>>(map, c, a, p);
      else kv8_decode_kernel<__half, 2><<<grid, kThreads, Smem::dyn, s>>>(map, c, a, p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace spec
