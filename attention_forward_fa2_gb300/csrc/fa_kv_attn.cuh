// fa_kv_attn.cuh -- attention of few query rows over the paged e4m3 cache, sm_103a (GB300).
//
// For query row i of a sequence (n_q rows, len_k cached keys) at position
// p = i + len_k - n_q (causal; else p = len_k - 1) and key/value head hk,
//     s_j = scale * ks(page j) * q_i . K8_j        over the keys j <= p in sight
//     o_i = sum_j softmax_j(s_j) * vs(page j) * V8_j,   lse_i = log sum_j e^{s_j}.
// Bound by reading the codes once, 2 d bytes per key and key/value head: the
// G = H / Hk query heads (times n_q rows) that share them are computed together,
// 8 or 16 rows to a unit of work (sequence, key/value head, row group).
//
// Schedule: the steps (key tiles of 128 tokens) of all units, laid end to end,
// are cut into equal ranges, one per resident CTA, so that every SM reads the
// same number of bytes whatever the lengths.  A CTA finds its range by a scan of
// the lengths, computes the units that lie in it whole, and leaves the ones cut
// by its borders in fp32 in the workspace (at most two); a second kernel joins
// them ("GPU 内核与 FlashAttention" §11.2).
// Cluster form (ONE), for few units of few steps, where latency is all: a unit is a
// cluster of up to 8 CTAs, each takes a share of its steps and leaves its part in its
// own shared memory; the cluster's warps join them row by row through distributed
// shared memory.  One launch, no workspace, no scan (one token, 16 heads on 4 of
// d 128: 1000 keys 9.8 -> 8.4 us, batch 8 on 32/8 heads and 2000 keys 15.9 -> 11.7; 33
// sequences, 4 tokens, 16/4 heads of d 64, window 1024: 20.0 -> 15.0, clusters of 3).
//
// A CTA: warp 4 walks the range ahead of the others, fills a ring of key tiles by
// TMA, a page at a time (each lane looks up and loads one page of the tile), and
// lays out the next unit's queries; warps 0-3 compute, 32 tokens of every tile
// each, with an online softmax of their own, and meet at the end of a unit.
//   Products: mma.sync m16n8k16 in f16 with fp32 sums, transposed so that tokens
//   (S^T = K Q^T) and features (O^T = V^T P^T) fill the 16 rows of a product and
//   8 or 16 query rows its columns: with 4 heads to a key/value head, queries as
//   rows would leave three quarters of every product empty.  The tensor work then
//   hides behind the loads; operands come from registers, which is where e4m3 codes become f16
//   (exact: f16 holds every e4m3 value).  q is scaled per row by a power of two
//   to below 2^8, so that f16 holds its bf16 values exactly down to 2^-22 of the
//   row's largest; P is rounded to f16 (2^-11, finer than bf16).
//   Scales: x_j = s_j log2 e + log2 vs(page j) is the exponent of the weight that
//   multiplies the codes V8_j; the running maximum and the rescale rule work on
//   x, so the rounding of P to f16 is relative to the largest term of the output
//   sum, whatever the pages' scales; the normaliser adds 2^x / vs in fp32.
//   Layout: TMA swizzles rows of d bytes; thread (g, c) = (lane / 4, lane % 4)
//   takes 16-byte chunk c of the K row of token perm(g), whose 16 values feed four
//   k-steps (a permutation of d that q's fragments share), and V through
//   ldmatrix.trans on byte pairs, one byte permute apart from the A fragment; P
//   turns from S^T's layout to the B fragment by movmatrix.  perm() places the two
//   rows that a quarter-warp reads in different banks.
//   Measured: 64 sequences of 8192 keys, 32 heads on 8 of d 128, one token each: 165 us,
//   97 % of a copy's bandwidth; four tokens each (16 rows) 193 us, 83 %.
//   Occupancy: two or three CTAs an SM: a warp's step is one dependent chain of loads,
//   products, shuffles and exponentials, and other warps have to cover it.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_f16.cuh"
#include "fa_fwd_kernel.cuh"
#include "fa_kvcache.h"
#include "ptx.cuh"

namespace fa {

constexpr int kKvThreads = 160;   // warps 0-3 compute, warp 4 loads

struct KvAttnParams {
  const __nv_bfloat16* q;   // [total_q, H, d], or [B, max_q, H, d] (cu null)
  __nv_bfloat16* o;         // like q
  float* lse;               // [B, H, max_q]
  const int *cu, *lens, *table;
  const float *k_scale, *v_scale;  // [num_pages, Hk]
  int B, max_q, max_k, total_q, H, Hk, G;
  int width, page, num_pages;
  int causal, window, sinks;
  int cluster, row_groups;  // cluster form: CTAs and row groups (see there)
  float scale_log2;
  // Workspace: a unit cut by the borders of CTA c's range is at place 2c (begun by
  // an earlier CTA) or 2c + 1 (begun by c, ended later); cut[c] names the unit
  // that ends in c and was begun by an earlier CTA.
  int4* cut;                // [ctas]: b (-1: none), key/value head, first row, CTA that began it
  float* part_o;            // [2 ctas, rows of a unit, d] normalised
  float* part_lse;          // [2 ctas, rows of a unit], log2 units
  unsigned long long timeout_ns;
  int* status;
};

enum KvSite : int { kKvSiteLoad = 201, kKvSiteLoadQ = 202, kKvSiteCompute = 203, kKvSiteComputeQ = 204, kKvSiteMeet = 205 };

// A unit of work as warp 4 hands it to the others.
struct KvUnit {
  int b;               // -1: no more units
  int hk, r0, rows;    // key/value head, first row, rows of the sequence (n_q * G)
  int row0, n_q, len;  // first packed query row, queries, keys
  int steps;           // steps of this CTA
  int ns, gap, t0;     // key tile of step t: t < ns ? t : t + gap, from t0
  int place;           // -1: whole (write o and lse), else place in the workspace
};

// NT: column tiles of 8 query rows; a unit has 8 * NT.  Resident CTAs of an SM: with
// 16 rows and d = 128 the accumulators do not fit 128 registers.
template <int D, int NT>
constexpr int kKvCtas = D == 128 && NT > 1 ? 2 : 3;
template <int D, int NT>
struct KvSmem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = kKvCtas<D, NT>;  // resident on an SM
  static constexpr int kStages = D == 128 ? (NT > 1 ? 3 : 2) : 4;
  static constexpr int kTileBytes = kKvTile * D;
  static constexpr int kStageBytes = 2 * kTileBytes;               // K then V
  static constexpr int kOffConst = kStages * kStageBytes;          // per stage and page: ks, log2 vs, 1 / vs
  static constexpr int kConstBytes = 3 * (kKvTile / 16) * 4;
  static constexpr int kOffQ = kOffConst + kStages * kConstBytes;  // two units' q as B fragments
  static constexpr int kQBytes = NT * (D / 32) * 32 * 16;
  static constexpr int kOffCoef = kOffQ + 2 * kQBytes;             // and the factor of each row's scores
  static constexpr int kOffUnit = kOffCoef + 2 * kRows * 4;
  static constexpr int kUnitBytes = 64;
  static constexpr int kOffBar = kOffUnit + 2 * kUnitBytes;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int kOffScan = kOffBar + kNumBars * 8;          // 6 long long, 2 long long, abort
  static constexpr int kOffLse = kOffScan + 80;                    // cluster form: of this CTA's part
  static constexpr int kBytes = kOffLse + kRows * 4;
  static constexpr int kAlloc = kBytes + 1024;
  // At the end of a unit its last stage takes two warps' rows: d floats, m and l.
  static constexpr int kRowStride = D + 16;                        // floats; rows of a quarter-warp in different banks
  static_assert(2 * kRows * (kRowStride + 2) * 4 <= kStageBytes, "join area");
  static_assert(sizeof(KvUnit) <= kUnitBytes && kOffQ % 16 == 0 && kOffBar % 8 == 0, "layout");
  static_assert(kCtas * (kAlloc + 1024) <= 233472, "resident CTAs");
};

// The queries and keys of a sequence, and the key tiles its rows see.
struct KvSeq {
  int row0, n_q, len, rows;
  KvRange range;
  int units_per_head;  // row groups
  bool bad;
  // Steps of a unit: a sequence without keys takes one, in which it sees nothing.
  __device__ __forceinline__ int steps() const { return range.steps > 0 ? range.steps : 1; }
};
template <int ROWS>
__device__ __forceinline__ KvSeq kv_seq(const KvAttnParams& p, int b) {
  KvSeq s;
  s.row0 = p.cu ? p.cu[b] : b * p.max_q;
  s.n_q = p.cu ? p.cu[b + 1] - s.row0 : p.max_q;
  s.len = p.lens[b];
  s.bad = s.n_q < 0 || s.n_q > p.max_q || s.row0 < 0 || s.row0 > p.total_q - s.n_q || s.len < 0 || s.len > p.max_k ||
          s.len > static_cast<long long>(p.width) * p.page;
  if (s.bad) s.n_q = 0;
  s.rows = s.n_q * p.G;
  s.units_per_head = (s.rows + ROWS - 1) / ROWS;
  s.range = kv_range(p.causal ? s.len - s.n_q : s.len - 1, s.len - 1, p.window, p.sinks);
  return s;
}
__device__ __forceinline__ long long kv_flat(const KvAttnParams& p, const KvSeq& s) {
  return static_cast<long long>(s.steps()) * s.units_per_head * p.Hk;
}

// D (16 x 8, fp32) += A (16 x 16, f16) * B (16 x 8, f16).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// The transpose of an 8 x 8 block of 16-bit values, one row a quad.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// Byte offset of 16-byte chunk `ch` of token row `t` in a tile as TMA swizzles it
// (128-byte rows: 128-byte swizzle, 64-byte rows: 64-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t kv_chunk(int t, int ch) {
  return D == 128 ? t * 128 + ((ch ^ (t & 7)) << 4) : t * 64 + ((ch ^ ((t >> 1) & 3)) << 4);
}

// Token (of 8) that fragment row g stands for.
template <int D>
__device__ __forceinline__ int kv_perm(int n) {
  return D == 128 ? (n >> 1) + ((n & 1) << 2) : n;
}

// Where a unit of the cluster form stands, for the rows' end.
struct KvPlace {
  int b, hk, r0, rows, row0;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of this CTA's shared `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

template <int D, int NT, bool ONE>
__global__ void __launch_bounds__(kKvThreads, (kKvCtas<D, NT>))
    fa_kv_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const KvAttnParams p) {
  using L = KvSmem<D, NT>;
  constexpr int kRows = L::kRows;
  constexpr int kSteps = D / 16;  // k-steps of S^T, row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw_base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  auto full = [&](int s) -> uint32_t { return base + L::kOffBar + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return base + L::kOffBar + 8u * (L::kStages + s); };
  auto q_full = [&](int s) -> uint32_t { return base + L::kOffBar + 8u * (2 * L::kStages + s); };
  auto q_empty = [&](int s) -> uint32_t { return base + L::kOffBar + 8u * (2 * L::kStages + 2 + s); };
  const uint32_t meet_bar = base + L::kOffBar + 8u * (2 * L::kStages + 4);
  long long* const s_scan = reinterpret_cast<long long*>(gbase + L::kOffScan);  // warp sums, then (sequence, its first step)
  volatile int* const s_abort = reinterpret_cast<volatile int*>(gbase + L::kOffScan + 64);
  float* const s_lse = reinterpret_cast<float*>(gbase + L::kOffLse);
  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int s = 0; s < L::kStages; ++s) {
      ptx::mbar_init(full(s), 32);
      ptx::mbar_init(empty(s), 4);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(q_full(s), 32);
      ptx::mbar_init(q_empty(s), 4);
    }
    ptx::mbar_init(meet_bar, 4);
    ptx::fence_mbar_init();
  }
  long long begin = 0, end = 1, span = 1;
  if constexpr (ONE) {
    __syncthreads();
  } else {
  // ------------------------------------------ this CTA's range of the steps of all units
  const int per = (p.B + kKvThreads - 1) / kKvThreads;  // sequences of a thread
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const KvSeq s = kv_seq<kRows>(p, b);
    if (s.bad && blockIdx.x == 0) record_error(p.status, kErrBadSeqlens, 0);
    mine += kv_flat(p, s);
  }
  long long pre = mine;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, pre, k);
    if (lane >= k) pre += v;
  }
  if (lane == 31) s_scan[warp] = pre;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kKvThreads / 32; ++w) {
    if (w < warp) pre += s_scan[w];
    total += s_scan[w];
  }
  pre -= mine;  // steps before this thread's sequences
  span = (total + gridDim.x - 1) / gridDim.x;
  begin = blockIdx.x * span;
  end = min(total, begin + span);
  if (threadIdx.x == 0) p.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (begin >= end) return;  // the whole CTA
  if (begin >= pre && begin < pre + mine) {
    long long at = pre;
    int b = b0;
    for (; b < b1; ++b) {
      const long long f = kv_flat(p, kv_seq<kRows>(p, b));
      if (begin < at + f) break;
      at += f;
    }
    s_scan[6] = b;
    s_scan[7] = at;
  }
  __syncthreads();
  }

  auto load = [&]() {
    // ================================================================ loads
    int b = ONE ? 0 : static_cast<int>(s_scan[6]);
    long long at = ONE ? 0 : s_scan[7];  // first step of sequence b
    long long pos = begin;
    const int ppt = kKvTile / p.page;  // pages per tile: one per lane
    int done = 0, units = 0;
    bool ok = true;
    while (ok && pos < end) {
      KvSeq s;
      int steps, t0, t1, hk, r0;
      if constexpr (ONE) {
        const int u = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
        r0 = u % p.row_groups * kRows;
        hk = u / p.row_groups % p.Hk;
        b = u / p.row_groups / p.Hk;
        s = kv_seq<kRows>(p, b);
        if (s.bad && lane == 0 && hk == 0 && r0 == 0 && rank == 0) record_error(p.status, kErrBadSeqlens, 0);
        if (lane == 0) *reinterpret_cast<KvPlace*>(s_scan) = KvPlace{b, hk, r0, s.rows, s.row0};
        steps = s.steps();
        t0 = steps * rank / p.cluster;
        t1 = steps * (rank + 1) / p.cluster;
        if (r0 >= s.rows || t0 == t1) break;
      } else {
        s = kv_seq<kRows>(p, b);
        while (pos >= at + kv_flat(p, s)) {
          at += kv_flat(p, s);
          s = kv_seq<kRows>(p, ++b);
        }
        steps = s.steps();
        const long long local = pos - at;
        const int unit = static_cast<int>(local / steps);
        t0 = static_cast<int>(local - static_cast<long long>(unit) * steps);
        t1 = static_cast<int>(min(static_cast<long long>(steps), t0 + (end - pos)));
        hk = unit / s.units_per_head;
        r0 = (unit % s.units_per_head) * kRows;
      }
      // ---- the unit and its queries, as B fragments: k-step kk = 4 h + wd takes
      // d = 16 (c + 4 h) + 4 wd + {0, 1 | 2, 3} of row 8 nt + g.
      uint4 raw[NT][D / 64][2];  // read ahead of the first tile's copies, laid out behind them
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 8 * nt + g;
        const bool in = r < s.rows;
        const __nv_bfloat16* src =
            p.q + (static_cast<size_t>(s.row0 + (in ? r / p.G : 0)) * p.H + hk * p.G + (in ? r % p.G : 0)) * D;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            raw[nt][h][v] = in ? *reinterpret_cast<const uint4*>(src + 16 * (c + 4 * h) + 8 * v) : make_uint4(0, 0, 0, 0);
      }
      auto put_unit = [&]() -> bool {
        const int us = units & 1;
        if (!ptx::mbar_wait_warp(q_empty(us), ((units >> 1) & 1u) ^ 1u, s_abort, p.timeout_ns)) {
          if (lane == 0) record_error(p.status, kErrTimeout, kKvSiteLoadQ);
          return false;
        }
        if (lane == 0) {
          KvUnit* const u = reinterpret_cast<KvUnit*>(gbase + L::kOffUnit + us * L::kUnitBytes);
          u->b = b;
          u->hk = hk;
          u->r0 = r0;
          u->rows = s.rows;
          u->row0 = s.row0;
          u->n_q = s.n_q;
          u->len = s.len;
          u->steps = t1 - t0;
          u->ns = s.range.ns;
          u->gap = s.range.gap;
          u->t0 = t0;
          u->place = ONE ? 0 : t0 > 0 ? 2 * blockIdx.x : t1 < steps ? 2 * blockIdx.x + 1 : -1;
          if (!ONE && t0 > 0 && t1 == steps)
            p.cut[blockIdx.x] = make_int4(b, hk, r0, static_cast<int>((pos - t0) / span));
        }
        {
          float* const coef = reinterpret_cast<float*>(gbase + L::kOffCoef) + us * kRows;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t amax = 0;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                const uint32_t wd[4] = {raw[nt][h][v].x, raw[nt][h][v].y, raw[nt][h][v].z, raw[nt][h][v].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) amax = max(amax, max((wd[k] << 16) & 0x7fffffffu, wd[k] & 0x7fff0000u));
              }
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // Exponent that brings the row's largest magnitude to [2^7, 2^8).
            const int ex = min(max(static_cast<int>(amax >> 23) - 127 - 7, -119), 119);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            if (c == 0) coef[8 * nt + g] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * p.scale_log2;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                // Two k-steps: 16 bytes a lane.
                const uint32_t wd[4] = {raw[nt][h][v].x, raw[nt][h][v].y, raw[nt][h][v].z, raw[nt][h][v].w};
                uint32_t f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  f[k] = pack_f16x2(__uint_as_float(wd[k] << 16) * down, __uint_as_float(wd[k] & 0xffff0000u) * down);
                ptx::st_shared_v4(base + L::kOffQ + us * L::kQBytes + ((nt * (D / 32) + 2 * h + v) * 32 + lane) * 16, f[0],
                                  f[1], f[2], f[3]);
              }
          }
        }
        ptx::mbar_arrive(q_full(us));
        ++units;
        return true;
      };
      // ---- the unit's key tiles
      auto page_of = [&](int t) -> int {  // this lane's page of step t; -1: nothing to load
        if (t >= t1 || lane >= ppt) return -1;
        const int a = (t < s.range.ns ? t : t + s.range.gap) * kKvTile + lane * p.page;
        if (!kv_needed(s.range, a, p.page)) return -1;
        const int id = p.table[static_cast<size_t>(b) * p.width + a / p.page];
        if (kv_page_ok(id, p.num_pages)) return id;
        record_error(p.status, kErrBadPage, 0);
        return -1;
      };
      int next = page_of(t0);
      for (int t = t0; t < t1; ++t, ++done) {
        const int st = done % L::kStages;
        const int id = next;
        next = page_of(t + 1);
        const size_t ph = static_cast<size_t>(id < 0 ? 0 : id) * p.Hk + hk;
        float ks = 0.f, vs = 1.f;
        if (id >= 0) {
          ks = p.k_scale[ph];
          vs = p.v_scale[ph];
          // A page that was never written has scale 0: its codes are weighed with the
          // smallest scale there is, so that its keys still count in the normaliser.
          if (vs == 0.f) vs = __uint_as_float(static_cast<uint32_t>(kKvMinExp + 127) << 23);
        }
        if (!ptx::mbar_wait_warp(empty(st), ((done / L::kStages) & 1u) ^ 1u, s_abort, p.timeout_ns)) {
          if (lane == 0) record_error(p.status, kErrTimeout, kKvSiteLoad);
          ok = false;
          break;
        }
        if (id >= 0) {
          mbar_expect_tx(full(st), 2 * p.page * D);
          const uint32_t dst = base + st * L::kStageBytes + lane * p.page * D;
          const int row = static_cast<int>(ph) * p.page;
          tma_load_2d(dst, &tm_k, full(st), 0, row);
          tma_load_2d(dst + L::kTileBytes, &tm_v, full(st), 0, row);
        }
        if (lane < ppt) {
          float* const cst = reinterpret_cast<float*>(gbase + L::kOffConst + st * L::kConstBytes) + 3 * lane;
          cst[0] = ks;
          cst[1] = log2f(vs);
          cst[2] = 1.f / vs;
        }
        ptx::mbar_arrive(full(st));
        // The unit follows its first tile's copies, whose latency covers it.
        if (t == t0 && !put_unit()) {
          ok = false;
          ++done;
          break;
        }
      }
      pos += ONE ? 1 : t1 - t0;
    }
    // The end of the units.
    if (ok && ptx::mbar_wait_warp(q_empty(units & 1), ((units >> 1) & 1u) ^ 1u, s_abort, p.timeout_ns)) {
      if (lane == 0) reinterpret_cast<KvUnit*>(gbase + L::kOffUnit + (units & 1) * L::kUnitBytes)->b = -1;
      ptx::mbar_arrive(q_full(units & 1));
    }
    if constexpr (!ONE) grid_dependents_launch();  // the join's blocks may be set up; they wait for this grid's end
    // Nothing may land in shared memory after the CTA is gone.
    for (int s = 0; s < L::kStages; ++s)
      if (done > s) ptx::mbar_wait_drain(full(s), ((done - 1 - s) / L::kStages) & 1u, p.timeout_ns);
  };

  auto compute = [&]() {
  // ================================================================ compute
  const int page_shift = 31 - __clz(p.page);
  int done = 0;
  // The four warps wait for one another (bounded like every wait: a warp that gave
  // up never comes, and bar.sync would wait for it for ever).
  uint32_t met = 0;
  auto meet = [&]() -> bool {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(meet_bar);
    const bool all = ptx::mbar_wait_warp(meet_bar, met & 1u, s_abort, p.timeout_ns);
    ++met;
    if (!all && lane == 0) record_error(p.status, kErrTimeout, kKvSiteMeet);
    return all;
  };
#pragma unroll 1
  for (int units = 0;; ++units) {
    const int us = units & 1;
    if (!ptx::mbar_wait_warp(q_full(us), (units >> 1) & 1u, s_abort, p.timeout_ns)) {
      if (lane == 0) record_error(p.status, kErrTimeout, kKvSiteComputeQ);
      return;
    }
    const KvUnit w = *reinterpret_cast<const KvUnit*>(gbase + L::kOffUnit + us * L::kUnitBytes);
    if (w.b < 0) return;
    const uint32_t qf = base + L::kOffQ + us * L::kQBytes + lane * 16;
    const float* const s_coef = reinterpret_cast<const float*>(gbase + L::kOffCoef) + us * kRows;
    const int off = w.len - w.n_q;
    const int p_min = p.causal ? off : w.len - 1, p_max = w.len - 1;
    const KvRange range = kv_range(p_min, p_max, p.window, p.sinks);
    const int lo_max = p.window > 0 ? p_max - p.window + 1 : 0;  // the last row's window starts here
    // This thread's columns of S^T and O^T: rows 8 nt + 2 c + e of the unit.
    float coef[NT][2];
    int pos[NT][2];  // position of the row; -1 for rows behind the last (nothing visible)
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = w.r0 + 8 * nt + 2 * c + e;
        coef[nt][e] = s_coef[8 * nt + 2 * c + e];
        pos[nt][e] = r >= w.rows ? -1 : p.causal ? r / p.G + off : w.len - 1;
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
    uint4 qr[NT == 1 ? D / 32 : 1];  // q's fragments, where the registers hold them
    if constexpr (NT == 1) {
#pragma unroll
      for (int k = 0; k < D / 32; ++k) qr[k] = ld_shared_v4(qf + k * 512);
    }
    float acc[NT][kSteps][4];  // O^T: features 16 k + 2 g (0, 1) and 16 k + 2 g + 1 (2, 3), rows 2 c and 2 c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][k][e] = 0.f;
#pragma unroll 1
    for (int i = 0; i < w.steps; ++i, ++done) {
      const int s = done % L::kStages;
      const int t = w.t0 + i;
      const int tok0 = (t < w.ns ? t : t + w.gap) * kKvTile + 32 * warp;
      if (!ptx::mbar_wait_warp(full(s), (done / L::kStages) & 1u, s_abort, p.timeout_ns)) {
        if (lane == 0) record_error(p.status, kErrTimeout, kKvSiteCompute);
        return;
      }
      if (kv_needed(range, tok0, 32)) {
        const uint32_t kt = base + s * L::kStageBytes + 32 * warp * D;
        const uint32_t vt = kt + L::kTileBytes;
        const float* const cst = reinterpret_cast<const float*>(gbase + L::kOffConst + s * L::kConstBytes);
        // 32 tokens at once, or with 16 rows 16 and 16: their sums leave registers for
        // half the scores only.
        constexpr int MTN = NT == 1 ? 2 : 1;
#pragma unroll 1
        for (int t8 = 0; t8 < 32; t8 += 16 * MTN) {
          // S^T: 8-token group j = 2 mt + half is rows half * 8 + g of row tile mt.
          float sc[NT][MTN][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4 * MTN; ++e) sc[nt][e >> 2][e & 3] = 0.f;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            uint4 raw[2 * MTN];
#pragma unroll
            for (int j = 0; j < 2 * MTN; ++j) raw[j] = ld_shared_v4(kt + kv_chunk<D>(t8 + 8 * j + kv_perm<D>(g), c + 4 * h));
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint4 qv[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (NT == 1)
                  qv[nt] = qr[2 * h + v];
                else
                  qv[nt] = ld_shared_v4(qf + (nt * (D / 32) + 2 * h + v) * 512);
              }
#pragma unroll
              for (int wd = 0; wd < 2; ++wd) {
                uint32_t lo[2 * MTN], hi[2 * MTN];
#pragma unroll
                for (int j = 0; j < 2 * MTN; ++j)
                  e4m3x4_to_f16(v == 0 ? (wd == 0 ? raw[j].x : raw[j].y) : (wd == 0 ? raw[j].z : raw[j].w), lo[j], hi[j]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int mt = 0; mt < MTN; ++mt)
                    mma_f16(sc[nt][mt], lo[2 * mt], lo[2 * mt + 1], hi[2 * mt], hi[2 * mt + 1],
                            wd == 0 ? qv[nt].x : qv[nt].z, wd == 0 ? qv[nt].y : qv[nt].w);
              }
            }
          }
          // Exponents x, masked where a border runs through these tokens.
          const int tk = tok0 + t8;
          const bool border = tk + 16 * MTN - 1 > p_min || (tk < lo_max && tk + 16 * MTN - 1 >= p.sinks);
          float inv[2 * MTN];
          uint32_t vmask[2 * MTN];  // bytes of V fragments whose token some row sees
#pragma unroll
          for (int j = 0; j < 2 * MTN; ++j) {
            vmask[j] = ~0u;
            const float* pc = cst + 3 * ((32 * warp + t8 + 8 * j) >> page_shift);
            const float ck = pc[0], lv = pc[1];
            inv[j] = pc[2];
            const int tok = tk + 8 * j + kv_perm<D>(g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = fmaf(sc[nt][j >> 1][2 * (j & 1) + e], coef[nt][e] * ck, lv);
                if (border) {
                  const int pr = pos[nt][e], lo = p.window > 0 ? pr - p.window + 1 : 0;
                  if (tok > pr || (tok < lo && tok >= p.sinks)) x = -INFINITY;
                }
                sc[nt][j >> 1][2 * (j & 1) + e] = x;
              }
            if (border) {
              const int ta = tk + 8 * j + kv_perm<D>(2 * c), tb = tk + 8 * j + kv_perm<D>(2 * c + 1);
              if (!kv_needed(range, ta, 1)) vmask[j] &= 0xff00ff00u;
              if (!kv_needed(range, tb, 1)) vmask[j] &= 0x00ff00ffu;
            }
          }
          // The reference maximum moves when a row's maximum passes it by 2^8.
          bool move = false;
          float mx[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[nt][e] = fmaxf(sc[nt][0][e], sc[nt][0][2 + e]);
              if constexpr (MTN == 2) mx[nt][e] = fmaxf(mx[nt][e], fmaxf(sc[nt][MTN - 1][e], sc[nt][MTN - 1][2 + e]));
              move = move || mx[nt][e] > m[nt][e] + 8.f;
            }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float al[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // The eight threads of a row agree on its maximum.
                float v = mx[nt][e];
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
                const bool up = v > m[nt][e] + 8.f;
                al[e] = up ? ptx::ex2(m[nt][e] - v) : 1.f;  // 0 from m = -inf
                if (up) m[nt][e] = v;
                l[nt][e] *= al[e];
              }
#pragma unroll
              for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][k][e] *= al[e & 1];
            }
          }
          uint32_t pb[NT][2 * MTN];  // P^T of the 8-token groups as halves of B fragments
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float n0 = m[nt][0] == -INFINITY ? 0.f : -m[nt][0], n1 = m[nt][1] == -INFINITY ? 0.f : -m[nt][1];
#pragma unroll
            for (int j = 0; j < 2 * MTN; ++j) {
              const float e0 = ptx::ex2(sc[nt][j >> 1][2 * (j & 1)] + n0), e1 = ptx::ex2(sc[nt][j >> 1][2 * (j & 1) + 1] + n1);
              l[nt][0] = fmaf(e0, inv[j], l[nt][0]);
              l[nt][1] = fmaf(e1, inv[j], l[nt][1]);
              pb[nt][j] = movmatrix_trans(pack_f16x2(e0, e1));
            }
          }
#pragma unroll
          for (int kk = 0; kk < MTN; ++kk) {
            // Matrix lane / 8: tokens 8 (bit 0) of the 16, chunk (bit 1) of the pair.
            const int trow = t8 + 16 * kk + ((lane >> 3) & 1) * 8 + kv_perm<D>(lane & 7);
#pragma unroll
            for (int ch = 0; ch < kSteps; ch += 2) {
              uint32_t r[4];
              ldmatrix_x4_trans(vt + kv_chunk<D>(trow, ch + (lane >> 4)), r);
#pragma unroll
              for (int q2 = 0; q2 < 2; ++q2) {
                uint32_t u0 = __byte_perm(r[2 * q2], 0, 0x3120), u1 = __byte_perm(r[2 * q2 + 1], 0, 0x3120);
                if (border) {
                  u0 &= vmask[2 * kk];
                  u1 &= vmask[2 * kk + 1];
                }
                uint32_t a0, a1, a2, a3;  // even and odd features, tokens 0-7 and 8-15
                e4m3x4_to_f16(u0, a0, a1);
                e4m3x4_to_f16(u1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][ch + q2], a0, a1, a2, a3, pb[nt][2 * kk], pb[nt][2 * kk + 1]);
              }
            }
          }
        }
      }
      __syncwarp();
      // The unit's last stage is kept for the warps' meeting below.
      if (lane == 0 && i + 1 < w.steps) ptx::mbar_arrive(empty(s));
    }
    if (lane == 0) ptx::mbar_arrive(q_empty(us));

    // ----------------------------------------------- the warps' parts: 2, 3 to 0, 1; 1 to 0
    const int last = (done - 1) % L::kStages;
    float* const area = reinterpret_cast<float*>(gbase + last * L::kStageBytes);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], k);
    auto put = [&](float* a) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* const dst = a + (8 * nt + 2 * c + e) * (L::kRowStride + 2);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
            *reinterpret_cast<float2*>(dst + 16 * k + 2 * g) = make_float2(acc[nt][k][e], acc[nt][k][2 + e]);
          if (g == 0) *reinterpret_cast<float2*>(dst + L::kRowStride) = make_float2(m[nt][e], l[nt][e]);
        }
    };
    auto take = [&](const float* a) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* const src = a + (8 * nt + 2 * c + e) * (L::kRowStride + 2);
          const float2 ml = *reinterpret_cast<const float2*>(src + L::kRowStride);
          const float M = fmaxf(m[nt][e], ml.x);
          const float f0 = M == -INFINITY ? 0.f : ptx::ex2(m[nt][e] - M), f1 = M == -INFINITY ? 0.f : ptx::ex2(ml.x - M);
          m[nt][e] = M;
          l[nt][e] = l[nt][e] * f0 + ml.y * f1;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const float2 x = *reinterpret_cast<const float2*>(src + 16 * k + 2 * g);
            acc[nt][k][e] = acc[nt][k][e] * f0 + x.x * f1;
            acc[nt][k][2 + e] = acc[nt][k][2 + e] * f0 + x.y * f1;
          }
        }
    };
    constexpr int kArea = kRows * (L::kRowStride + 2);
    if (!meet()) return;  // all four have read the stage
    if (warp >= 2) put(area + (warp - 2) * kArea);
    if (!meet()) return;
    if (warp < 2) take(area + warp * kArea);
    if (warp == 1) put(area + kArea);
    if (!meet()) return;
    if (warp == 0) {
      take(area + kArea);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = w.r0 + 8 * nt + 2 * c + e;
          if (r >= w.rows) continue;
          const float lt = l[nt][e];
          const float il = lt > 0.f ? 1.f / lt : lt;  // NaN stays
          const float lse2 = lt > 0.f ? m[nt][e] + log2f(lt) : lt == 0.f ? -INFINITY : lt;
          if constexpr (ONE) {
            float* const part = reinterpret_cast<float*>(gbase) + (8 * nt + 2 * c + e) * D + 2 * g;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
              *reinterpret_cast<float2*>(part + 16 * k) = make_float2(acc[nt][k][e] * il, acc[nt][k][2 + e] * il);
            if (g == 0) s_lse[8 * nt + 2 * c + e] = lse2;
          } else if (w.place >= 0) {
            const size_t row = static_cast<size_t>(w.place) * kRows + 8 * nt + 2 * c + e;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
              *reinterpret_cast<float2*>(p.part_o + row * D + 16 * k + 2 * g) =
                  make_float2(acc[nt][k][e] * il, acc[nt][k][2 + e] * il);
            if (g == 0) p.part_lse[row] = lse2;
          } else {
            const int i = r / p.G, h = w.hk * p.G + r % p.G;
            __nv_bfloat16* const dst = p.o + (static_cast<size_t>(w.row0 + i) * p.H + h) * D + 2 * g;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
              *reinterpret_cast<uint32_t*>(dst + 16 * k) = ptx::pack_bf16x2(acc[nt][k][e] * il, acc[nt][k][2 + e] * il);
            if (g == 0) p.lse[(static_cast<size_t>(w.b) * p.H + h) * p.max_q + i] = lse2 * 0.69314718055994530942f;
          }
        }
    }
    // The stage goes back to TMA: order the writes above before its copies.
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty(last));
  }
  };

  if (ONE && warp == 0 && lane < kRows) s_lse[lane] = -INFINITY;  // stays where the CTA has no steps
  if (warp == 4)
    load();
  else
    compute();
  if constexpr (ONE) {
    // ------------------------------------- the cluster's parts, row by row
    __syncwarp();
    cluster_sync();  // every thread of the cluster comes here: each wait above ends
    const KvPlace u = *reinterpret_cast<const KvPlace*>(s_scan);
    const int rank = blockIdx.x % p.cluster;
    for (int r = rank + p.cluster * warp; r < kRows && u.r0 + r < u.rows; r += p.cluster * (kKvThreads / 32)) {
      const float mine = lane < p.cluster ? ld_cluster(cluster_addr(ptx::smem_u32(s_lse + r), lane)) : -INFINITY;
      float M = mine;
#pragma unroll
      for (int k = 4; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
      M = __shfl_sync(0xffffffffu, M, 0);
      const float f = mine == -INFINITY ? 0.f : ptx::ex2(mine - M);
      constexpr int kPer = D / 32;
      float acc[kPer], l = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
      for (int s = 0; s < p.cluster; ++s) {
        const float fs = __shfl_sync(0xffffffffu, f, s);
        const bool none = __shfl_sync(0xffffffffu, mine, s) == -INFINITY;  // no values in that part
        const uint32_t src = cluster_addr(base + (r * D + lane * kPer) * 4, s);
        l += fs;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const float x = ld_cluster(src + 4 * e);
          acc[e] = none ? acc[e] : fmaf(fs, x, acc[e]);
        }
      }
      const float il = l > 0.f ? 1.f / l : l;  // NaN stays
      const int i = (u.r0 + r) / p.G, h = u.hk * p.G + (u.r0 + r) % p.G;
      __nv_bfloat16* const dst = p.o + (static_cast<size_t>(u.row0 + i) * p.H + h) * D + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = ptx::pack_bf16x2(acc[e] * il, acc[e + 1] * il);
      if (lane == 0)
        p.lse[(static_cast<size_t>(u.b) * p.H + h) * p.max_q + i] =
            l > 0.f ? (M + log2f(l)) * 0.69314718055994530942f : l == 0.f ? -INFINITY : l;
    }
    cluster_sync();  // no CTA leaves while another reads its parts
  }
}

// The parts of the unit that ends in CTA blockIdx.x's range and was begun before
// it: o = sum_s w_s O_s / sum_s w_s with w_s = 2^(lse2_s - max).  One block per row;
// each warp adds every fourth part.  Bound by reading the parts, a few per cent of
// the codes; a single sequence and head has one part per CTA.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) fa_kv_join_kernel(const KvAttnParams p) {
  grid_dependency_wait();
  const int4 cut = p.cut[blockIdx.x];
  if (cut.x < 0) return;
  const int r = cut.z + blockIdx.y;
  const int row0 = p.cu ? p.cu[cut.x] : cut.x * p.max_q;
  const int n_q = p.cu ? p.cu[cut.x + 1] - row0 : p.max_q;
  if (r >= n_q * p.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = static_cast<int>(blockIdx.x) - cut.w + 1;
  // Part s lies with CTA cut.w + s: the first is that CTA's tail, the others are heads.
  auto at = [&](int s) -> size_t {
    return (2 * static_cast<size_t>(cut.w + s) + (s == 0 ? 1 : 0)) * ROWS + blockIdx.y;
  };
  float M = -INFINITY;
  for (int s = lane; s < parts; s += 32) M = fmaxf(M, p.part_lse[at(s)]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
  constexpr int kPer = D / 32;
  float acc[kPer], l = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  if (M > -INFINITY) {
#pragma unroll 4
    for (int s = warp; s < parts; s += 4) {
      const float f = ptx::ex2(p.part_lse[at(s)] - M);
      const float* src = p.part_o + at(s) * D + lane * kPer;
      l += f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(f, src[e], acc[e]);
    }
  }
  __shared__ float s_acc[4][D], s_l[4];
#pragma unroll
  for (int e = 0; e < kPer; ++e) s_acc[warp][lane * kPer + e] = acc[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const float il = l > 0.f ? 1.f / l : 0.f;
  const int i = r / p.G, h = cut.y * p.G + r % p.G;
  if (threadIdx.x < D / 2) {
    const int e = 2 * threadIdx.x;
    const float a = (s_acc[0][e] + s_acc[1][e]) + (s_acc[2][e] + s_acc[3][e]);
    const float c = (s_acc[0][e + 1] + s_acc[1][e + 1]) + (s_acc[2][e + 1] + s_acc[3][e + 1]);
    *reinterpret_cast<uint32_t*>(p.o + (static_cast<size_t>(row0 + i) * p.H + h) * D + e) =
        ptx::pack_bf16x2(a * il, c * il);
  }
  if (threadIdx.x == 0)
    p.lse[(static_cast<size_t>(cut.x) * p.H + h) * p.max_q + i] =
        l > 0.f ? (M + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace fa
