// fa_kv_attn.cuh -- attention of few query rows over the paged e4m3 cache, sm_103a (GB300).
//
// For query row i of a sequence (n_q rows, len_k cached keys) at position
// p = i + len_k - n_q (causal; else p = len_k - 1) and key/value head hk,
//     s_j = scale * ks(page j) * q_i . K8_j        over the keys j <= p in sight
//     o_i = sum_j softmax_j(s_j) * vs(page j) * V8_j,   lse_i = log sum_j e^{s_j}.
// Bound by reading the codes once, 2 d bytes per key and key/value head: the
// G = H / Hk query heads (times n_q rows) that share them run in one CTA, and long
// sequences are cut over keys (splits) so that every SM reads; a second kernel
// joins the splits ("GPU 内核与 FlashAttention" §11.2).
//
// A CTA holds up to 16 * MT query rows, and walks key tiles of 128 tokens through
// a ring in shared memory that one warp fills by TMA, a page at a time (each lane
// looks up and loads one page of the tile).  Four warps compute, 32 tokens of
// every tile each, with an online softmax of their own; they meet once at the end.
//   Products: mma.sync m16n8k16 in f16 with fp32 sums.  With at most 32 rows the
//   tensor work is 1/8 to 1/4 of a 128-row tcgen05 tile and hides behind the
//   loads; operands come from registers, which is where e4m3 codes become f16
//   (exact: f16 holds every e4m3 value).  q is scaled per row by a power of two
//   to below 2^8, so that f16 holds its bf16 values exactly down to 2^-22 of the
//   row's largest; P is rounded to f16 (2^-11, finer than bf16).
//   Scales: x_j = s_j log2 e + log2 vs(page j) is the exponent of the weight that
//   multiplies the codes V8_j; the running maximum and the rescale rule work on
//   x, so the rounding of P to f16 is relative to the largest term of the output
//   sum, whatever the pages' scales; the normaliser adds 2^x / vs in fp32.
//   Layout: TMA swizzles rows of d bytes; thread (n, c) = (lane / 4, lane % 4)
//   takes 16-byte chunk c of the K row of token perm(n), whose 16 values feed four
//   k-steps (a permutation of d that q's fragments share), and V through
//   ldmatrix.trans on byte pairs, one byte permute apart from the B fragment;
//   perm() places the two rows that a quarter-warp reads in different banks.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_fwd_kernel.cuh"
#include "fa_kvcache.h"
#include "ptx.cuh"

namespace fa {

struct KvAttnParams {
  const __nv_bfloat16* q;   // [total_q, H, d], or [B, max_q, H, d] (cu null)
  __nv_bfloat16* o;         // like q
  float* lse;               // [B, H, max_q]
  const int *cu, *lens, *table;
  const float *k_scale, *v_scale;  // [num_pages, Hk]
  int B, max_q, max_k, total_q, H, Hk, G;
  int width, page, num_pages;
  int causal, window, sinks;
  int row_groups;           // CTAs of 16 * MT rows per (sequence, key/value head)
  int splits, split_steps;  // key splits, steps per split
  float scale_log2;
  float *ws_o, *ws_lse;     // [splits, B, H, max_q, d] and [splits, B, H, max_q] (log2 units)
  unsigned long long timeout_ns;
  int* status;
};

constexpr int kKvThreads = 160;  // warps 0-3 compute, warp 4 loads

enum KvSite : int { kKvSiteLoad = 201, kKvSiteCompute = 202 };

template <int D, int MT>
struct KvSmem {
  static constexpr int kStages = D == 128 ? (MT > 1 ? 6 : 3) : 6;
  static constexpr int kTileBytes = kKvTile * D;
  static constexpr int kStageBytes = 2 * kTileBytes;  // K then V
  static constexpr int kRowStride = D + 16;           // floats; rows of a quarter-warp in different banks
  static constexpr int kOffConst = kStages * kStageBytes;         // per stage and page: coefficient, log2 vs, 1 / vs
  static constexpr int kConstBytes = 3 * (kKvTile / 16) * 4;
  static constexpr int kOffQ = kOffConst + kStages * kConstBytes;  // q fragments (MT > 1)
  static constexpr int kQBytes = MT > 1 ? MT * (D / 16) * 32 * 16 : 0;
  static constexpr int kOffBar = kOffQ + kQBytes;
  static constexpr int kOffAbort = kOffBar + 2 * kStages * 8;
  static constexpr int kBytes = kOffAbort + 16;
  static constexpr int kAlloc = kBytes + 1024;
  // The join at the end reuses the ring: per warp and row m, l and d floats.
  static_assert(4 * 16 * MT * (kRowStride + 2) * 4 <= kStages * kStageBytes, "join area");
  static_assert(kOffQ % 16 == 0 && kOffBar % 8 == 0, "alignment");
};

// The query rows and key range of one CTA.
struct KvWork {
  int row0;            // first packed query row of the sequence
  int n_q, len;
  int rows;            // rows of this key/value head: n_q * G, row r is query r / G, head r % G
  int r0, r1;          // rows of this group
  KvRange range;
  int p_min, p_max;
  bool bad;
};
template <int RG>
__device__ __forceinline__ KvWork kv_work(const KvAttnParams& p, int b, int rg) {
  KvWork w;
  w.row0 = p.cu ? p.cu[b] : b * p.max_q;
  w.n_q = p.cu ? p.cu[b + 1] - w.row0 : p.max_q;
  w.len = p.lens[b];
  w.bad = w.n_q < 0 || w.n_q > p.max_q || w.row0 < 0 || w.row0 > p.total_q - w.n_q || w.len < 0 || w.len > p.max_k ||
          w.len > static_cast<long long>(p.width) * p.page;
  if (w.bad) w.n_q = 0;
  w.rows = w.n_q * p.G;
  w.r0 = rg * RG;
  w.r1 = min(w.rows, w.r0 + RG);
  const int i0 = w.r0 / p.G, i1 = (w.r1 - 1) / p.G;
  w.p_min = p.causal ? i0 + w.len - w.n_q : w.len - 1;
  w.p_max = p.causal ? i1 + w.len - w.n_q : w.len - 1;
  w.range = kv_range(w.p_min, w.p_max, p.window, p.sinks);
  if (w.r0 >= w.rows) w.range.steps = 0;
  return w;
}

__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// D (16 x 8, fp32) += A (16 x 16, f16) * B (16 x 8, f16).
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Token (of 8) that fragment row / column n stands for.
template <int D>
__device__ __forceinline__ int kv_perm(int n) {
  return D == 128 ? (n >> 1) + ((n & 1) << 2) : n;
}

template <int D, int MT>
__global__ void __launch_bounds__(kKvThreads, D == 128 && MT > 1 ? 1 : 2)
    fa_kv_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const KvAttnParams p) {
  using L = KvSmem<D, MT>;
  constexpr int RG = 16 * MT;
  constexpr int kSteps = D / 16;  // k-steps of S
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw_base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x;
  const int hk = blockIdx.y / p.row_groups, rg = blockIdx.y % p.row_groups;
  const int b = blockIdx.z;

  const KvWork w = kv_work<RG>(p, b, rg);
  if (w.bad && split == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(p.status, kErrBadSeqlens, 0);
  if (w.r0 >= w.rows) return;
  const int t0 = split * p.split_steps;
  const int t1 = min(w.range.steps, t0 + p.split_steps);
  if (t0 >= t1 && p.splits > 1) return;  // the join knows which splits hold keys

  auto full = [&](int s) -> uint32_t { return base + L::kOffBar + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return base + L::kOffBar + 8u * (L::kStages + s); };
  volatile int* const s_abort = reinterpret_cast<volatile int*>(gbase + L::kOffAbort);
  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int s = 0; s < L::kStages; ++s) {
      ptx::mbar_init(full(s), 32);
      ptx::mbar_init(empty(s), 4);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();

  const int n = lane >> 2, c = lane & 3;
  float m[MT][2], l[MT][2];
  float acc[MT][kSteps][2][4];  // [chunk of 16 d][even / odd d][C fragment]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[mt][e] = -INFINITY;
      l[mt][e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[mt][k][e >> 2][e & 3] = 0.f;
  }

  if (warp == 4) {
    // ================================================================ loads
    const int ppt = kKvTile / p.page;  // pages per tile: one per lane
    auto first_token = [&](int t) { return (t < w.range.ns ? t : t + w.range.gap) * kKvTile + lane * p.page; };
    auto page_of = [&](int t) -> int {  // -1: nothing to load
      if (t >= t1 || lane >= ppt) return -1;
      const int a = first_token(t);
      if (!kv_needed(w.range, a, p.page)) return -1;
      const int id = p.table[static_cast<size_t>(b) * p.width + a / p.page];
      if (kv_page_ok(id, p.num_pages)) return id;
      record_error(p.status, kErrBadPage, 0);
      return -1;
    };
    int next = page_of(t0);
    int done = 0;
    for (int t = t0; t < t1; ++t, ++done) {
      const int s = done % L::kStages;
      const int id = next;
      next = page_of(t + 1);
      const size_t ph = static_cast<size_t>(id < 0 ? 0 : id) * p.Hk + hk;
      float ks = 0.f, vs = 1.f;
      if (id >= 0) {
        ks = p.k_scale[ph];
        vs = p.v_scale[ph];
      }
      if (!ptx::mbar_wait_warp(empty(s), ((done / L::kStages) & 1u) ^ 1u, s_abort, p.timeout_ns)) {
        if (lane == 0) record_error(p.status, kErrTimeout, kKvSiteLoad);
        break;
      }
      if (id >= 0) {
        mbar_expect_tx(full(s), 2 * p.page * D);
        const uint32_t dst = base + s * L::kStageBytes + lane * p.page * D;
        const int row = static_cast<int>(ph) * p.page;
        tma_load_2d(dst, &tm_k, full(s), 0, row);
        tma_load_2d(dst + L::kTileBytes, &tm_v, full(s), 0, row);
      }
      if (lane < ppt) {
        float* const cst = reinterpret_cast<float*>(gbase + L::kOffConst + s * L::kConstBytes) + 3 * lane;
        cst[0] = ks;
        cst[1] = log2f(vs);
        cst[2] = 1.f / vs;
      }
      ptx::mbar_arrive(full(s));
    }
    // Nothing may land in shared memory after this: each lane sees the last fills complete.
    for (int s = 0; s < L::kStages; ++s)
      if (done > s) ptx::mbar_wait_drain(full(s), ((done - 1 - s) / L::kStages) & 1u, p.timeout_ns);
  } else {
    // ============================================================== compute
    // q of this thread's rows n and n + 8 of each row tile, scaled to below 2^8, as
    // A fragments: k-step kk = 4 h + wd takes d = 16 (c + 4 h) + 4 wd + {0, 1 | 2, 3}.
    uint32_t qa[MT == 1 ? kSteps : 1][4];
    float coef[MT][2];
    int pos[MT][2];  // position of the row; -1 for rows behind the last (nothing visible)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t frag[kSteps][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = w.r0 + 16 * mt + 8 * e + n;
        const bool in = r < w.r1;
        const int i = r / p.G, g = r % p.G;
        pos[mt][e] = !in ? -1 : p.causal ? i + w.len - w.n_q : w.len - 1;
        const __nv_bfloat16* src = p.q + (static_cast<size_t>(w.row0 + i) * p.H + hk * p.G + g) * D;
        float x[kSteps][4];
        uint32_t amax = 0;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (in) raw = *reinterpret_cast<const uint4*>(src + 16 * (c + 4 * h) + 8 * v);
            const uint32_t wd[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[4 * h + 2 * v + (k >> 1)][2 * (k & 1)] = __uint_as_float(wd[k] << 16);
              x[4 * h + 2 * v + (k >> 1)][2 * (k & 1) + 1] = __uint_as_float(wd[k] & 0xffff0000u);
              amax = max(amax, max((wd[k] << 16) & 0x7fffffffu, wd[k] & 0x7fff0000u));
            }
          }
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // Exponent that brings the row's largest magnitude to [2^7, 2^8).
        const int ex = min(max(static_cast<int>(amax >> 23) - 127 - 7, -119), 119);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        coef[mt][e] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * p.scale_log2;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          frag[k][e] = pack_f16x2(x[k][0] * down, x[k][1] * down);
          frag[k][2 + e] = pack_f16x2(x[k][2] * down, x[k][3] * down);
        }
      }
      if constexpr (MT == 1) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) qa[k][e] = frag[k][e];
      } else if (warp == mt % 4) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          ptx::st_shared_v4(base + L::kOffQ + ((mt * kSteps + k) * 32 + lane) * 16, frag[k][0], frag[k][1], frag[k][2],
                            frag[k][3]);
      }
    }
    if constexpr (MT > 1) asm volatile("bar.sync 1, 128;" ::: "memory");

    const int page_shift = 31 - __clz(p.page);
    const int lo_max = p.window > 0 ? w.p_max - p.window + 1 : 0;  // the last row's window starts here
    bool ok = true;
    int done = 0;
#pragma unroll 1
    for (int t = t0; t < t1 && ok; ++t, ++done) {
      const int s = done % L::kStages;
      const int tok0 = (t < w.range.ns ? t : t + w.range.gap) * kKvTile + 32 * warp;
      if (!ptx::mbar_wait_warp(full(s), (done / L::kStages) & 1u, s_abort, p.timeout_ns)) {
        if (lane == 0) record_error(p.status, kErrTimeout, kKvSiteCompute);
        ok = false;
        break;
      }
      if (kv_needed(w.range, tok0, 32)) {
        const uint32_t kt = base + s * L::kStageBytes + 32 * warp * D;
        const uint32_t vt = kt + L::kTileBytes;
        const float* const cst = reinterpret_cast<const float*>(gbase + L::kOffConst + s * L::kConstBytes);
        float sc[MT][4][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[mt][e >> 2][e & 3] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint4 raw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) raw[j] = ld_shared_v4(kt + kv_chunk<D>(8 * j + kv_perm<D>(n), c + 4 * h));
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) {
            uint32_t a[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (MT == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[mt][e] = qa[4 * h + wd][e];
              } else {
                const uint4 f = ld_shared_v4(base + L::kOffQ + ((mt * kSteps + 4 * h + wd) * 32 + lane) * 16);
                a[mt][0] = f.x;
                a[mt][1] = f.y;
                a[mt][2] = f.z;
                a[mt][3] = f.w;
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b0, b1;
              e4m3x4_to_f16(wd == 0 ? raw[j].x : wd == 1 ? raw[j].y : wd == 2 ? raw[j].z : raw[j].w, b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_f16(sc[mt][j], a[mt], b0, b1);
            }
          }
        }
        // Exponents x, masked where a border runs through these 32 tokens.
        const bool border = tok0 + 31 > w.p_min || (tok0 < lo_max && tok0 + 31 >= p.sinks);
        float inv[4];
        uint32_t vmask[4] = {~0u, ~0u, ~0u, ~0u};  // bytes of V fragments whose token no row sees
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* pc = cst + 3 * ((32 * warp + 8 * j) >> page_shift);
          const float ck = pc[0], lv = pc[1];
          inv[j] = pc[2];
          const int ta = tok0 + 8 * j + kv_perm<D>(2 * c), tb = tok0 + 8 * j + kv_perm<D>(2 * c + 1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = coef[mt][e] * ck;
              float x0 = fmaf(sc[mt][j][2 * e], f, lv), x1 = fmaf(sc[mt][j][2 * e + 1], f, lv);
              if (border) {
                const int pr = pos[mt][e], lo = p.window > 0 ? pr - p.window + 1 : 0;
                if (ta > pr || (ta < lo && ta >= p.sinks)) x0 = -INFINITY;
                if (tb > pr || (tb < lo && tb >= p.sinks)) x1 = -INFINITY;
              }
              sc[mt][j][2 * e] = x0;
              sc[mt][j][2 * e + 1] = x1;
            }
          if (border) {
            if (!kv_needed(w.range, ta, 1)) vmask[j] &= 0xff00ff00u;
            if (!kv_needed(w.range, tb, 1)) vmask[j] &= 0x00ff00ffu;
          }
        }
        // The reference maximum moves when a row's maximum passes it by 2^8.
        bool move = false;
        float mx[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(sc[mt][0][2 * e], sc[mt][0][2 * e + 1]);
#pragma unroll
            for (int j = 1; j < 4; ++j) v = ptx::fmax3(v, sc[mt][j][2 * e], sc[mt][j][2 * e + 1]);
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            mx[mt][e] = v;
            move = move || v > m[mt][e] + 8.f;
          }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float al[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool up = mx[mt][e] > m[mt][e] + 8.f;
              al[e] = up ? ptx::ex2(m[mt][e] - mx[mt][e]) : 1.f;  // 0 from m = -inf
              if (up) m[mt][e] = mx[mt][e];
              l[mt][e] *= al[e];
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[mt][k][e >> 2][e & 3] *= al[(e >> 1) & 1];
          }
        }
        uint32_t pa[MT][2][4];  // P as A fragments of two k-steps of 16 tokens
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float neg = m[mt][e] == -INFINITY ? 0.f : -m[mt][e];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float e0 = ptx::ex2(sc[mt][j][2 * e] + neg), e1 = ptx::ex2(sc[mt][j][2 * e + 1] + neg);
              l[mt][e] = fmaf(e0 + e1, inv[j], l[mt][e]);
              pa[mt][j >> 1][2 * (j & 1) + e] = pack_f16x2(e0, e1);
            }
          }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          // Matrix lane / 8: tokens 8 (bit 0) of the 16, chunk (bit 1) of the pair.
          const int trow = 16 * kk + ((lane >> 3) & 1) * 8 + kv_perm<D>(lane & 7);
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
              uint32_t e0, o0, e1, o1;
              e4m3x4_to_f16(u0, e0, o0);
              e4m3x4_to_f16(u1, e1, o1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_f16(acc[mt][ch + q2][0], pa[mt][kk], e0, e1);
                mma_f16(acc[mt][ch + q2][1], pa[mt][kk], o0, o1);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty(s));
    }
  }

  // ------------------------------------------------- the four warps' parts joined
  __syncthreads();
  float* const sm_m = reinterpret_cast<float*>(gbase);
  float* const sm_l = sm_m + 4 * RG;
  float* const sm_o = sm_l + 4 * RG;
  if (warp < 4) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * mt + 8 * e + n;
        float lt = l[mt][e] + __shfl_xor_sync(0xffffffffu, l[mt][e], 1);
        lt += __shfl_xor_sync(0xffffffffu, lt, 2);
        if (c == 0) {
          sm_m[warp * RG + r] = m[mt][e];
          sm_l[warp * RG + r] = lt;
        }
        float* const dst = sm_o + (warp * RG + r) * L::kRowStride + 4 * c;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          *reinterpret_cast<float4*>(dst + 16 * k) = make_float4(acc[mt][k][0][2 * e], acc[mt][k][1][2 * e],
                                                                 acc[mt][k][0][2 * e + 1], acc[mt][k][1][2 * e + 1]);
      }
  }
  __syncthreads();
  const size_t all_rows = static_cast<size_t>(p.B) * p.H * p.max_q;
  for (int idx = threadIdx.x; idx < (w.r1 - w.r0) * (D / 4); idx += kKvThreads) {
    const int r = idx / (D / 4), d4 = idx % (D / 4);
    const int i = (w.r0 + r) / p.G, h = hk * p.G + (w.r0 + r) % p.G;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) M = fmaxf(M, sm_m[k * RG + r]);
    float lt = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = M == -INFINITY ? 0.f : ptx::ex2(sm_m[k * RG + r] - M);
      const float4 v = *reinterpret_cast<const float4*>(sm_o + (k * RG + r) * L::kRowStride + 4 * d4);
      lt = fmaf(f, sm_l[k * RG + r], lt);
      o0 = fmaf(f, v.x, o0);
      o1 = fmaf(f, v.y, o1);
      o2 = fmaf(f, v.z, o2);
      o3 = fmaf(f, v.w, o3);
    }
    const float il = lt > 0.f ? 1.f / lt : 0.f;
    const float lse2 = lt > 0.f ? M + log2f(lt) : -INFINITY;
    const size_t row = (static_cast<size_t>(b) * p.H + h) * p.max_q + i;
    if (p.splits > 1) {
      const size_t at = static_cast<size_t>(split) * all_rows + row;
      *reinterpret_cast<float4*>(p.ws_o + at * D + 4 * d4) = make_float4(o0 * il, o1 * il, o2 * il, o3 * il);
      if (d4 == 0) p.ws_lse[at] = lse2;
    } else {
      uint2 pk = make_uint2(ptx::pack_bf16x2(o0 * il, o1 * il), ptx::pack_bf16x2(o2 * il, o3 * il));
      if (!(lt > 0.f) && M == -INFINITY) pk = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(p.o + (static_cast<size_t>(w.row0 + i) * p.H + h) * D + 4 * d4) = pk;
      if (d4 == 0) p.lse[row] = lse2 * 0.69314718055994530942f;
    }
  }
}

// The splits of each row joined: o = sum_s w_s O_s / sum_s w_s with w_s = 2^(lse2_s - max).
// One warp per row; bound by reading the fp32 parts (a few per cent of the codes).
template <int D, int RG>
__global__ void __launch_bounds__(128) fa_kv_join_kernel(const KvAttnParams p) {
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long all_rows = static_cast<long long>(p.B) * p.H * p.max_q;
  if (row >= all_rows) return;
  const int i = static_cast<int>(row % p.max_q);
  const int h = static_cast<int>((row / p.max_q) % p.H);
  const int b = static_cast<int>(row / p.max_q / p.H);
  const KvWork w = kv_work<RG>(p, b, (i * p.G + h % p.G) / RG);
  if (i >= w.n_q) return;
  const int parts = (w.range.steps + p.split_steps - 1) / p.split_steps;
  float M = -INFINITY;
  for (int s = lane; s < parts; s += 32) M = fmaxf(M, p.ws_lse[s * all_rows + row]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
  constexpr int kPer = D / 32;
  float acc[kPer], l = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  if (M > -INFINITY) {
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float f = ptx::ex2(p.ws_lse[s * all_rows + row] - M);
      const float* src = p.ws_o + (s * all_rows + row) * D + lane * kPer;
      l += f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(f, src[e], acc[e]);
    }
  }
  const float il = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* const dst = p.o + (static_cast<size_t>(w.row0 + i) * p.H + h) * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = ptx::pack_bf16x2(acc[e] * il, acc[e + 1] * il);
  if (lane == 0) p.lse[row] = l > 0.f ? (M + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace fa
