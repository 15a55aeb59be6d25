// fa_win_bwd_kernel.cuh -- gradients of attention with a sliding window and sinks, sm_103a (GB300).
//
// With the forward's rule (query i stands at p = i + len_k - len_q and sees the
// keys j <= p with p - j < window or j < sinks) the gradients are those of
// "GPU 内核与 FlashAttention" §13 with P = 0 outside it:
//     P = exp(scale Q K^T - L),  dV = P^T dO,  dS = P o (dO V^T - D),  D_i = do_i . o_i,
//     dQ = scale dS K,  dK = scale dS^T Q.
// The products, roles, barriers and the shared and tensor memory of a CTA are
// those of fa_bwd_kernel (fa_bwd_kernel.cuh: 128 keys of one key/value head per
// unit, dK and dV on chip, dQ by line-wide fp32 reductions); what differs is
// which query blocks a unit walks.
//   Key block without sinks: the query blocks from the one that holds position
//     kb * 128 to the one that holds kb * 128 + 127 + window - 1, so the work of
//     a unit is bound by the window.
//   Key block with sinks: every later query sees its sinks, which for a long
//     sequence is many times the work of the other units and would end the
//     kernel with one CTA per head running.  Its query blocks are cut into
//     chunks of chunk_qb blocks (about a window's worth), one unit each; a
//     chunk writes its dK and dV in fp32 to a place of its own in the
//     workspace, and the last kernel adds the chunks in their order (no
//     atomics: dK and dV come out the same on every run).
//   Few units for the SMs: the steps (heads of the group times query blocks) of every
//     unit are cut into `split` parts, handled like the chunks.
// Bound by the chain of a step (see the MMA thread): two sequences of 4096, 16 heads on
// 4 of d 128, window 512, 4 sinks: 119 us, tensor pipe 47 % busy; 151 us with the
// kernels before and behind it.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_bwd_kernel.cuh"
#include "fa_f16.cuh"
#include "fa_win_kernel.cuh"
#include "ptx.cuh"

namespace fa {

// BwdParams' lse2 and delta hold the negated values here.
struct WinBwdParams : BwdParams {
  int window, sinks;
  int num_skb;         // key blocks that can hold sinks: ceil(min(sinks, Nk) / 128)
  int chunk_qb;        // query blocks per chunk of such a block
  int num_chunks;      // chunks of the longest sequence
  int split;           // parts of a unit
  int num_sink_units;  // B * Hk * num_skb * num_chunks * split
  int total_q, total_k;  // variable-length form: packed rows (sequences past them are rejected)
  int* order;          // packed: the units that have work, the longest first; their number behind place num_units
  float* part;         // [num_chunks * split, B, Hk, num_skb * 128, 2 (dV, dK), d] fp32
  float* part2;        // split > 1: [split, B, Hk, (num_kb - num_skb) * 128, 2, d], the other blocks
};

// Part `n` of a key's dV and dK, for key blocks that are not one unit.
template <int D>
__device__ __forceinline__ float* win_part(const WinBwdParams& p, int n, int b, int hk, int kb, int key) {
  const bool sink = kb < p.num_skb;
  const int first = sink ? 0 : p.num_skb, blocks = sink ? p.num_skb : p.num_kb - p.num_skb;
  const size_t row = ((static_cast<size_t>(n) * p.B + b) * p.Hk + hk) * (static_cast<size_t>(blocks) * kBwdBK) +
                     (key - first * kBwdBK);
  return (sink ? p.part : p.part2) + row * (2 * D);
}
// The steps [lo, hi) of n that part s takes.
__host__ __device__ __forceinline__ int win_share(int n, int s, int split) {
  return static_cast<int>(static_cast<long long>(n) * s / split);
}

// Query blocks [qb0, qb0 + nqb) that see a key of block kb; `sink`: the block
// holds sinks of this sequence, so every later query does.
__host__ __device__ __forceinline__ void win_query_blocks(int kb, int len_q, int len_k, int window, bool sink, int& qb0,
                                                          int& nqb) {
  qb0 = 0;
  nqb = 0;
  if (kb * kBwdBK >= len_k) return;
  const int off = len_k - len_q;
  const int num_qb = (len_q + kBwdBQ - 1) / kBwdBQ;
  const int first = kb * kBwdBK - off;  // query at the position of the block's first key
  qb0 = first <= 0 ? 0 : first / kBwdBQ;
  int end = num_qb;
  if (!sink) {
    const int last_key = min(kb * kBwdBK + kBwdBK, len_k) - 1;
    // Last query whose window reaches last_key (64 bits: window goes up to 2^30).
    const long long last = static_cast<long long>(last_key) + window - 1 - off;
    if (last < 0) return;
    if (last / kBwdBQ + 1 < end) end = static_cast<int>(last / kBwdBQ + 1);
  }
  nqb = end > qb0 ? end - qb0 : 0;
}

struct WinBwdUnit {
  int b, hk, kb;
  int chunk;           // chunk of a sink block, -1 for a block without sinks
  int part;            // place of its dK and dV in the workspace, -1: bf16 to dk and dv
  int q_start, len_q, k_start, len_k, off;
  RowWindow kw;
  int qb0, nqb;        // query blocks qb0 .. qb0 + nqb - 1 of each head of the group in turn,
  int h0, q0, nsteps;  // from head h0 (of all) and block qb0 + q0 on
};
// The steps of a unit in turn: head and query block.
struct WinBwdStep {
  int h, q;
  __device__ __forceinline__ explicit WinBwdStep(const WinBwdUnit& w) : h(w.h0), q(w.q0) {}
  __device__ __forceinline__ void next(const WinBwdUnit& w) {
    if (++q == w.nqb) {
      q = 0;
      ++h;
    }
  }
};

template <bool VARLEN>
__device__ __forceinline__ void win_bwd_seq(const WinBwdParams& p, int b, int& q_start, int& len_q, int& k_start,
                                            int& len_k, bool& bad) {
  q_start = 0;
  len_q = p.Nq;
  k_start = 0;
  len_k = p.Nk;
  bad = false;
  if constexpr (VARLEN) {
    q_start = p.cu_q[b];
    len_q = p.cu_q[b + 1] - q_start;
    k_start = p.cu_k[b];
    len_k = p.cu_k[b + 1] - k_start;
    bad = len_q < 0 || len_k < 0 || len_q > p.Nq || len_k > p.Nk || q_start < 0 || k_start < 0 ||
          q_start > p.total_q - len_q || k_start > p.total_k - len_k;
    if (bad) len_q = len_k = 0;
  }
}

// SPLIT: p.split > 1 (without it the kernel is 5 % faster).
template <bool VARLEN, bool SPLIT>
__device__ __forceinline__ WinBwdUnit win_bwd_decode(const WinBwdParams& p, int u) {
  WinBwdUnit w;
  int r;
  const int split = SPLIT ? p.split : 1;
  const int s = (u < p.num_sink_units ? u : u - p.num_sink_units) % split;
  if (u < p.num_sink_units) {
    r = u / split;
    w.chunk = r % p.num_chunks;
    r /= p.num_chunks;
    w.kb = r % p.num_skb;
    r /= p.num_skb;
  } else {
    // Key block by key block: under a long window the first blocks are seen by the
    // most queries, and the round-robin over units of falling work stays even.
    w.chunk = -1;
    r = (u - p.num_sink_units) / split;
    w.kb = p.num_skb + r / (p.B * p.Hk);
    r %= p.B * p.Hk;
  }
  w.hk = r % p.Hk;
  w.b = r / p.Hk;
  bool bad;
  win_bwd_seq<VARLEN>(p, w.b, w.q_start, w.len_q, w.k_start, w.len_k, bad);
  if (bad)
    record_error(p.status, kErrBadSeqlens, 0);
  w.off = w.len_k - w.len_q;
  w.kw = make_window<VARLEN>(w.k_start, w.k_start + w.len_k, w.k_start + w.kb * kBwdBK, kBwdBK);
  win_query_blocks(w.kb, w.len_q, w.len_k, p.window, w.chunk >= 0, w.qb0, w.nqb);
  if (w.chunk >= 0) {
    const int skip = min(w.nqb, w.chunk * p.chunk_qb);
    w.qb0 += skip;
    w.nqb = min(w.nqb - skip, p.chunk_qb);
  }
  const int n = p.group * w.nqb;
  w.h0 = w.hk * p.group;
  w.q0 = 0;
  w.nsteps = n;
  if (SPLIT && n > 0) {
    const int i0 = win_share(n, s, split);
    w.nsteps = win_share(n, s + 1, split) - i0;
    w.h0 += i0 / w.nqb;
    w.q0 = i0 % w.nqb;
  }
  w.part = w.chunk >= 0 ? w.chunk * split + s : SPLIT ? s : -1;
  return w;
}

// The units of a CTA: round by round, packed ones (where listed) in the order of the
// list, every other round from its end, so that units of falling length even out.
#define FA_WIN_BWD_FOR_EACH_UNIT(u)                                                                              \
  for (int round = 0, u = unit_at(0); round * static_cast<int>(gridDim.x) < num_units && ok; u = unit_at(++round)) \
    if (u >= 0)

// Lists the units that have work (one block; behind the list their number): a counting
// sort by steps into 64 bins, the longest first.  Without it, ragged sequences leave
// the static rounds uneven: nine of 386 to 2048 tokens, 2 key/value heads, window 300:
// 43 steps on the busiest SM where 34 are possible.
constexpr int kOrderMax = 16384;  // units up to which they are listed
template <bool SPLIT>
__device__ __forceinline__ void win_bwd_list(const WinBwdParams& p) {
  constexpr int kBins = 64;
  __shared__ int bins[kBins];
  const int most = p.group * (p.nq_pad / kBwdBQ);
  auto bin = [&](int u) -> int {  // -1: no work
    const WinBwdUnit w = win_bwd_decode<true, SPLIT>(p, u);
    if (w.kb * kBwdBK >= w.len_k || (w.nsteps == 0 && w.part >= 0)) return -1;
    return kBins - 1 - static_cast<int>(static_cast<long long>(w.nsteps) * (kBins - 1) / max(most, 1));
  };
  if (threadIdx.x < kBins) bins[threadIdx.x] = 0;
  __syncthreads();
  for (int u = threadIdx.x; u < p.num_units; u += blockDim.x) {
    const int b = bin(u);
    if (b >= 0) atomicAdd(&bins[b], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int sum = 0;
    for (int b = 0; b < kBins; ++b) {
      const int n = bins[b];
      bins[b] = sum;
      sum += n;
    }
    p.order[p.num_units] = sum;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < p.num_units; u += blockDim.x) {
    const int b = bin(u);
    if (b >= 0) p.order[atomicAdd(&bins[b], 1)] = u;
  }
}

template <int D, int STAGES, bool VARLEN, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    fa_win_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                  const WinBwdParams p) {
  static_assert(D == 64 || D == 128, "backward kernel: d = 64 or 128");
  static_assert(STAGES >= 2, "backward ring depth");
  using L = BwdSmem<D, STAGES>;
  constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 384;
  constexpr int kDPanels = D / 64;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw_base);
  if ((base - raw_base) + static_cast<uint32_t>(L::kBytes) > static_cast<uint32_t>(L::kAlloc)) {
    // The aligned layout would run past the allocation (uniform over the CTA,
    // decided before any barrier or tensor-memory use).
    if (threadIdx.x == 0) record_error(p.status, kErrUnsupported, kBSiteSmemWindow);
    return;
  }

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t bar0 = base + L::kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* const s_tmem = reinterpret_cast<volatile uint32_t*>(gbase + L::kOffTmem);
  volatile int* const s_abort = reinterpret_cast<volatile int*>(gbase + L::kOffAbort);
  const uint64_t tmo = p.timeout_ns;

  if (warp == 13 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_do);
  }
  if (threadIdx.x == 0) {
    *s_abort = 0;
    ptx::mbar_init(bar(L::kBarKVFull), 1);
    ptx::mbar_init(bar(L::kBarKVEmpty), 1);
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(bar(L::kBarQFull + s), 1);
      ptx::mbar_init(bar(L::kBarQEmpty + s), 1);
    }
    ptx::mbar_init(bar(L::kBarSFull), 1);
    ptx::mbar_init(bar(L::kBarDPFull), 1);
    ptx::mbar_init(bar(L::kBarPFull), 256);
    ptx::mbar_init(bar(L::kBarDSFull), 256);
    ptx::mbar_init(bar(L::kBarDQFull), 1);
    ptx::mbar_init(bar(L::kBarDQEmpty), 128);
    ptx::mbar_init(bar(L::kBarAccFull), 1);
    ptx::mbar_init(bar(L::kBarAccEmpty), 128);
    ptx::mbar_init(bar(L::kBarTeardown), 1);
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(ptx::smem_u32(const_cast<uint32_t*>(s_tmem)), 512);
    ptx::tmem_relinquish();
  }
  if constexpr (D < 128) {
    // The K panels beyond d are never loaded: zero them once, visible to the
    // tensor core (async proxy) before any MMA reads them.
    for (uint32_t i = threadIdx.x; i < (L::kKBytes - L::kKVBytes) / 16; i += blockDim.x)
      ptx::st_shared_v4(base + L::kOffK + L::kKVBytes + 16 * i, 0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if constexpr (VARLEN) grid_dependency_wait();  // the prep kernel wrote the list
  const bool listed = VARLEN && p.order != nullptr;
  const int num_units = listed ? p.order[p.num_units] : p.num_units;
  auto unit_at = [&](int round) -> int {
    const int c = static_cast<int>(blockIdx.x), n = static_cast<int>(gridDim.x);
    const int at = round * n + (listed && (round & 1) ? n - 1 - c : c);
    return at >= num_units ? -1 : listed ? p.order[at] : at;
  };

  // Handshake barriers are single: each one's next completion needs an action
  // of its own waiter first (S(g+1) is issued after P(g) is seen, dP(g+1)
  // after the drain has read dQ^T(g), which follows dS(g), and so on).
  if (warp >= 12) {
    ptx::setmaxnreg_dec<BwdRegSplit::kOther>();
    if (warp == 13 && lane == 0) {
      // ============================================================ TMA loads
      uint32_t g = 0, uc = 0;
      bool ok = true;
      if constexpr (!VARLEN) grid_dependency_wait();  // what it wrote is read, and added to, behind the first copy
#pragma unroll 1
      FA_WIN_BWD_FOR_EACH_UNIT(u) {
        const WinBwdUnit w = win_bwd_decode<VARLEN, SPLIT>(p, u);
        if (w.nsteps == 0) continue;
        if (uc > 0 && !ptx::mbar_wait(bar(L::kBarKVEmpty), (uc - 1) & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kBSiteLoadKV);
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(bar(L::kBarKVFull), 2 * L::kKVBytes);  // K and V, D features each
#pragma unroll
        for (int pn = 0; pn < kDPanels; ++pn) {
          if constexpr (VARLEN) {
            // Packed rows; a tile shifted back below row 0 is zero-filled there.
            ptx::tma_load_3d(base + L::kOffK + pn * L::kKVPanel, &tm_k, bar(L::kBarKVFull), pn * 64, w.hk,
                             w.kw.load_row);
            ptx::tma_load_3d(base + L::kOffV + pn * L::kKVPanel, &tm_v, bar(L::kBarKVFull), pn * 64, w.hk,
                             w.kw.load_row);
          } else {
            ptx::tma_load_4d(base + L::kOffK + pn * L::kKVPanel, &tm_k, bar(L::kBarKVFull), pn * 64, w.hk,
                             w.kb * kBwdBK, w.b);
            ptx::tma_load_4d(base + L::kOffV + pn * L::kKVPanel, &tm_v, bar(L::kBarKVFull), pn * 64, w.hk,
                             w.kb * kBwdBK, w.b);
          }
        }
        ++uc;
        WinBwdStep st(w);
#pragma unroll 1
        for (int i = 0; i < w.nsteps && ok; ++i, ++g, st.next(w)) {
          const uint32_t slot = g % STAGES;
          if (g >= STAGES && !ptx::mbar_wait(bar(L::kBarQEmpty + slot), ((g / STAGES) - 1) & 1u, s_abort, tmo)) {
            record_error(p.status, kErrTimeout, kBSiteLoadQ);
            ok = false;
            break;
          }
          const int h = st.h, qb = w.qb0 + st.q;
          const uint32_t fb = bar(L::kBarQFull + slot);
          ptx::mbar_arrive_expect_tx(fb, L::kSlotBytes + L::kLDBytes);
          const uint32_t sq = base + L::kOffQ + slot * L::kSlotBytes;
#pragma unroll
          for (int pn = 0; pn < kDPanels; ++pn) {
            if constexpr (VARLEN) {
              const int qrow = make_window<true>(w.q_start, w.q_start + w.len_q, w.q_start + qb * kBwdBQ, kBwdBQ).load_row;
              ptx::tma_load_3d(sq + pn * L::kQPanel, &tm_q, fb, pn * 64, h, qrow);
              ptx::tma_load_3d(sq + L::kQBytes + pn * L::kQPanel, &tm_do, fb, pn * 64, h, qrow);
            } else {
              ptx::tma_load_4d(sq + pn * L::kQPanel, &tm_q, fb, pn * 64, h, qb * kBwdBQ, w.b);
              ptx::tma_load_4d(sq + L::kQBytes + pn * L::kQPanel, &tm_do, fb, pn * 64, h, qb * kBwdBQ, w.b);
            }
          }
          // The block's scaled LSE and D rows (512 bytes each, 512-byte aligned:
          // nq_pad is a multiple of the block) for the softmax warps.
          const size_t ro = (static_cast<size_t>(w.b) * p.H + h) * p.nq_pad + static_cast<size_t>(qb) * kBwdBQ;
          const uint32_t sld = base + L::kOffLD + slot * L::kLDBytes;
          ptx::bulk_load(sld, p.lse2 + ro, kBwdBQ * 4, fb);
          ptx::bulk_load(sld + kBwdBQ * 4, p.delta + ro, kBwdBQ * 4, fb);
        }
      }
      grid_dependents_launch();  // the kernels behind this one may be set up; they wait for its end
      // Drain: every issued copy must land before the CTA exits.
      if (uc > 0) ptx::mbar_wait_drain(bar(L::kBarKVFull), (uc - 1) & 1u, tmo);
      for (uint32_t s = 0; s < STAGES; ++s) {
        if (g > s) {
          const uint32_t rounds = (g - 1 - s) / STAGES + 1;
          ptx::mbar_wait_drain(bar(L::kBarQFull + s), (rounds - 1) & 1u, tmo);
        }
      }
    } else if (warp == 12 && lane == 0) {
      // ============================================================ MMA issue
      constexpr uint32_t id_s = ptx::idesc_bf16_f32(128, kBwdBQ, 0, 0);   // K Q^T, V dO^T
      constexpr uint32_t id_acc = ptx::idesc_bf16_f32(128, D, 0, 1);      // P^T dO, dS^T Q
      constexpr uint32_t id_dq = ptx::idesc_bf16_f32(128, kBwdBQ, 1, 1);  // K^T dS^T (K padded to 128 rows)
      uint32_t g = 0, uc = 0;
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t par, int site) -> bool {
        if (ptx::mbar_wait(b, par, s_abort, tmo)) return true;
        record_error(p.status, kErrTimeout, site);
        ok = false;
        return false;
      };
      // Shared-memory descriptors advance by byte offset / 16 in their low
      // word (the address field cannot carry below 256 KiB), so each MMA
      // costs the issuing thread an add instead of a descriptor build.
      const uint64_t kdesc = ptx::sw128_desc(base + L::kOffK, 16, 1024);
      const uint64_t vdesc = ptx::sw128_desc(base + L::kOffV, 16, 1024);
      const uint64_t kdesc_mn = ptx::sw128_desc(base + L::kOffK, L::kKVPanel, 1024);
      const uint64_t dsdesc_mn = ptx::sw128_desc(base + L::kOffDS, L::kDSPanel, 1024);
      const uint64_t dsdesc_k = ptx::sw128_desc(base + L::kOffDS, 16, 1024);
      auto issue_s = [&](uint32_t t) {
        const uint64_t qdesc = ptx::sw128_desc(base + L::kOffQ + (t % STAGES) * L::kSlotBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t oa = (kk / 4) * L::kKVPanel + (kk % 4) * 32;
          const uint32_t ob = (kk / 4) * L::kQPanel + (kk % 4) * 32;
          ptx::mma_ss(tmem + kColS, kdesc + (oa >> 4), qdesc + (ob >> 4), id_s, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit(bar(L::kBarSFull));
      };
      auto issue_dp = [&](uint32_t t) {
        const uint64_t dodesc =
            ptx::sw128_desc(base + L::kOffQ + (t % STAGES) * L::kSlotBytes + L::kQBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t oa = (kk / 4) * L::kKVPanel + (kk % 4) * 32;
          const uint32_t ob = (kk / 4) * L::kQPanel + (kk % 4) * 32;
          ptx::mma_ss(tmem + kColDP, vdesc + (oa >> 4), dodesc + (ob >> 4), id_s, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit(bar(L::kBarDPFull));
      };
#pragma unroll 1
      FA_WIN_BWD_FOR_EACH_UNIT(u) {
        const WinBwdUnit w = win_bwd_decode<VARLEN, SPLIT>(p, u);
        if (w.nsteps == 0) continue;
        if (!wait(bar(L::kBarKVFull), uc & 1u, kBSiteMmaKV)) break;
        ptx::tc_fence_after();
        if (!wait(bar(L::kBarQFull + g % STAGES), (g / STAGES) & 1u, kBSiteMmaQ)) break;
        ptx::tc_fence_after();
        issue_s(g);
        // dP's columns last held dQ^T(g - 1) (the previous unit's last step).
        if (g > 0 && !wait(bar(L::kBarDQEmpty), (g - 1) & 1u, kBSiteMmaDQ)) break;
        ptx::tc_fence_after();
        issue_dp(g);
#pragma unroll 1
        for (int i = 0; i < w.nsteps && ok; ++i, ++g) {
          const uint32_t slot = g % STAGES;
          const uint32_t sq = base + L::kOffQ + slot * L::kSlotBytes;
          const uint32_t sdo = sq + L::kQBytes;
          // dV += P^T dO (P^T of warpgroup c at columns 64c .. 64c + 31).
          if (!wait(bar(L::kBarPFull), g & 1u, kBSiteMmaP)) break;
          if (i == 0 && uc > 0 && !wait(bar(L::kBarAccEmpty), (uc - 1) & 1u, kBSiteMmaAcc)) break;
          ptx::tc_fence_after();
          const uint64_t dodesc_mn = ptx::sw128_desc(sdo, L::kQPanel, 1024);
#pragma unroll
          for (int kk = 0; kk < kBwdBQ / 16; ++kk)
            ptx::mma_ts(tmem + kColDV, tmem + kColS + (kk >> 2) * 64 + (kk & 3) * 8, dodesc_mn + kk * 128, id_acc,
                        (i > 0 || kk > 0) ? 1u : 0u);
          // S(g + 1) over P(g) (read by the dV just issued, which runs first).
          if (i + 1 < w.nsteps) {
            if (!wait(bar(L::kBarQFull + (g + 1) % STAGES), ((g + 1) / STAGES) & 1u, kBSiteMmaQ)) break;
            ptx::tc_fence_after();
            issue_s(g + 1);
          }
          // dK += dS^T Q, then dQ^T = K^T dS^T over dP, both from shared memory.  (dQ^T
          // first, with dK under the drain, was measured 14 % slower; for d = 64, dQ^T
          // in columns of its own no faster: what bounds the step is the chain of the
          // softmax warps, 1.5 k cycles for P and 2.0 k for dS of 5.5 k, while the
          // reductions of dQ, 64 KB a step, move 23 bytes a cycle for 2.8 k of them.)
          if (!wait(bar(L::kBarDSFull), g & 1u, kBSiteMmaDS)) break;
          ptx::tc_fence_after();
          const uint64_t qdesc_mn = ptx::sw128_desc(sq, L::kQPanel, 1024);
#pragma unroll
          for (int kk = 0; kk < kBwdBQ / 16; ++kk) {
            const uint32_t oa = (kk / 4) * L::kDSPanel + (kk % 4) * 32;
            ptx::mma_ss(tmem + kColDK, dsdesc_k + (oa >> 4), qdesc_mn + kk * 128, id_acc, (i > 0 || kk > 0) ? 1u : 0u);
          }
          ptx::mma_commit(bar(L::kBarQEmpty + slot));  // Q(g) and dO(g) read
#pragma unroll
          for (int kk = 0; kk < kBwdBK / 16; ++kk)
            ptx::mma_ss(tmem + kColDP, kdesc_mn + kk * 128, dsdesc_mn + kk * 128, id_dq, kk > 0 ? 1u : 0u);
          ptx::mma_commit(bar(L::kBarDQFull));
          // dP(g + 1) once the drain has read dQ^T(g) out of those columns.
          if (i + 1 < w.nsteps) {
            if (!wait(bar(L::kBarDQEmpty), g & 1u, kBSiteMmaDQ)) break;
            ptx::tc_fence_after();
            issue_dp(g + 1);
          }
        }
        if (!ok) break;
        ptx::mma_commit(bar(L::kBarAccFull));
        ptx::mma_commit(bar(L::kBarKVEmpty));
        ++uc;
      }
      ptx::mma_commit(bar(L::kBarTeardown));
      if (!ptx::mbar_wait_drain(bar(L::kBarTeardown), 0, tmo)) record_error(p.status, kErrTimeout, kBSiteTeardown);
    }
  } else if (warp < 8) {
    // (softmax warpgroups keep the launch allocation, BwdRegSplit::kSoftmax)
    // ================================================================ softmax
    const int c = warp >> 2;                    // query columns [64c, 64c + 64)
    const int r = ((warp & 3) << 5) + lane;     // key row of the block
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tSc = tmem + lane_off + kColS + c * 64;
    const uint32_t tDc = tmem + lane_off + kColDP + c * 64;  // dP^T columns of this warpgroup
    const float c2 = p.scale_log2;
    uint32_t g = 0;
    bool ok = true;
#pragma unroll 1
    FA_WIN_BWD_FOR_EACH_UNIT(u) {
      const WinBwdUnit w = win_bwd_decode<VARLEN, SPLIT>(p, u);
      if (w.nsteps == 0) continue;
      const int kj0 = w.kw.load_row - w.k_start;          // first key of the tile (sequence index)
      const int kj = kj0 + r;                             // this thread's key
      const bool key_ok = r >= w.kw.lo && r < w.kw.hi;  // a key of this block
      WinBwdStep st(w);
#pragma unroll 1
      for (int i = 0; i < w.nsteps && ok; ++i, ++g, st.next(w)) {
        const int qb = w.qb0 + st.q;
        // First query (sequence index) of this warpgroup's columns of the tile as loaded.
        const int q0 = make_window<VARLEN>(w.q_start, w.q_start + w.len_q, w.q_start + qb * kBwdBQ, kBwdBQ).load_row -
                       w.q_start + c * 64;
        // Scaled LSE and D of this warpgroup's 64 queries, staged with Q(g)
        // (shared-memory broadcasts instead of dependent global loads).
        const uint32_t slot = g % STAGES;
        // Pairs of -L log2 e, then of -D: the operands of the packed sums below.
        const ulonglong2* l2g = reinterpret_cast<const ulonglong2*>(gbase + L::kOffLD + slot * L::kLDBytes) + c * 16;
        const ulonglong2* dlg = l2g + kBwdBQ / 4;
        if (!ptx::mbar_wait_warp(bar(L::kBarSFull), g & 1u, s_abort, tmo) ||
            !ptx::mbar_wait_warp(bar(L::kBarQFull + slot), (g / STAGES) & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kBSiteSoftS);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        // P^T = 2^(S^T c2 - L log2 e), 32 columns at a time; 0 where the query does
        // not see the key (only tiles that hold a border are masked: the
        // diagonal, the window's end, the end of the sinks, keys of the next
        // block); the bf16 pairs of half hh go to columns 16 hh .. 16 hh + 15
        // (already read).  f16 pairs stay in registers for dS: S(g + 1)
        // overwrites these columns as soon as dV(g) has read them.
        const int q_pos = q0 + w.off;  // position of this warpgroup's first column
        const bool border = w.kw.lo != 0 || w.kw.hi != kBwdBK || kj0 + kBwdBK - 1 > q_pos ||
                            (kj0 <= q_pos + 63 - p.window && kj0 + kBwdBK > p.sinks);
        uint32_t ph[32];  // P^T in f16: its rounding (2^-11) does not add to that of dS
        const uint64_t c2x2 = ptx::f2_pack(c2, c2);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t sr[32];
          ptx::tmem_ld32(tSc + hh * 32, sr);
          ptx::tmem_wait_ld();
          float e[32];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const ulonglong2 l = l2g[hh * 8 + k / 4];
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              float x0, x1;
              ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(sr[k + 2 * h2]), __uint_as_float(sr[k + 2 * h2 + 1])),
                                         c2x2, h2 == 0 ? l.x : l.y),
                             x0, x1);
              e[k + 2 * h2] = ptx::ex2(x0);
              e[k + 2 * h2 + 1] = ptx::ex2(x1);
            }
          }
          if (border) {
            // Column k is the query at position q_pos + 32 hh + k: it sees key kj
            // from k0 on, and up to k1 - 1 unless kj is a sink.
            const int k0 = key_ok ? kj - q_pos - hh * 32 : 32;
            const int k1 = kj < p.sinks ? 32 : kj + p.window - q_pos - hh * 32;
            const uint32_t seen = bits_below(k1) & ~bits_below(k0);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if ((seen & (1u << k)) == 0u) e[k] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 32; k += 2) ph[16 * hh + k / 2] = pack_f16x2(e[k], e[k + 1]);
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) pk[k / 2] = ptx::pack_bf16x2(e[k], e[k + 1]);
          ptx::tmem_st16(tSc + hh * 16, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(L::kBarPFull));
        // dS^T = P^T o (dP^T - D), from the f16 P^T pairs held above.
        if (!ptx::mbar_wait_warp(bar(L::kBarDPFull), g & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kBSiteSoftDP);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        // The previous step's dQ^T MMA must have read the shared dS^T buffer.
        if (g > 0 && !ptx::mbar_wait_warp(bar(L::kBarDQFull), (g - 1) & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kBSiteSoftDQ);
          ok = false;
          break;
        }
        // Row r of panel c (64 queries) of the shared dS^T: 128 bytes, 128-byte swizzle.
        const uint32_t row_addr = base + L::kOffDS + c * L::kDSPanel + r * 128;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t dr[32], ds[16];
          ptx::tmem_ld32(tDc + hh * 32, dr);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const ulonglong2 dl = dlg[hh * 8 + k / 4];
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const int e = k + 2 * h2;
              float y0, y1;
              ptx::f2_unpack(ptx::f2_mul(ptx::f2_add(ptx::f2_pack(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])),
                                                     h2 == 0 ? dl.x : dl.y),
                                         unpack_f16x2(ph[16 * hh + e / 2])),
                             y0, y1);
              ds[e / 2] = ptx::pack_bf16x2(y0, y1);
            }
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int chunk = 4 * hh + q4;
            ptx::st_shared_v4(row_addr + ((chunk ^ (r & 7)) << 4), ds[4 * q4], ds[4 * q4 + 1], ds[4 * q4 + 2],
                              ds[4 * q4 + 3]);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();  // the dP loads above precede dQ^T overwriting those columns
        ptx::mbar_arrive(bar(L::kBarDSFull));
      }
    }
  } else {
    ptx::setmaxnreg_inc<BwdRegSplit::kDrain>();
    // ======================================== dQ drain and the dK / dV epilogue
    const int wq = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(wq << 5) << 16;
    uint32_t g = 0, uc = 0;
    bool ok = true;
#pragma unroll 1
    FA_WIN_BWD_FOR_EACH_UNIT(u) {
      const WinBwdUnit w = win_bwd_decode<VARLEN, SPLIT>(p, u);
      const int kr = (wq << 5) + lane;  // this thread's key row of the tile
      const bool key_ok = kr >= w.kw.lo && kr < w.kw.hi;
      const size_t prow = VARLEN ? static_cast<size_t>(w.kw.load_row + kr)
                                 : static_cast<size_t>(w.b) * p.Nk + w.kw.load_row + kr;
      const size_t krow = (prow * p.Hk + w.hk) * D;
      if (w.nsteps == 0) {
        // No query sees these keys: dK = dV = 0 (a part without steps is left out of
        // the sum of the parts).
        if (key_ok && w.part < 0) {
          for (int e = 0; e < D; e += 8) {
            ptx::st_global_v4(p.dk + krow + e, 0u, 0u, 0u, 0u);
            ptx::st_global_v4(p.dv + krow + e, 0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      WinBwdStep st(w);
#pragma unroll 1
      for (int i = 0; i < w.nsteps && ok; ++i, ++g, st.next(w)) {
        const int h = st.h, qb = w.qb0 + st.q;
        if (!ptx::mbar_wait_warp(bar(L::kBarDQFull), g & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kBSiteDrainDQ);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if ((wq << 5) < D) {
          uint32_t v[128];
#pragma unroll
          for (int q32 = 0; q32 < 4; ++q32) ptx::tmem_ld32(tmem + lane_off + kColDP + q32 * 32, v + 32 * q32);
          ptx::tmem_wait_ld();
          ptx::tc_fence_before();
          ptx::mbar_arrive(bar(L::kBarDQEmpty));
          // Query q of the block: the warp's 32 features are one 128-byte line.
          float* const dst = p.dq_acc +
                             (static_cast<size_t>(w.b * p.H + h) * p.nq_pad + static_cast<size_t>(qb) * kBwdBQ) * D +
                             (wq << 5) + lane;
#pragma unroll
          for (int q = 0; q < kBwdBQ; ++q) ptx::red_add(dst + static_cast<size_t>(q) * D, __uint_as_float(v[q]));
        } else {
          // Lanes (features) at or beyond d hold the zero rows of the padded product.
          ptx::mbar_arrive(bar(L::kBarDQEmpty));
        }
      }
      if (!ok) break;
      // Unit done, one key row per thread: dK (times the scale) and dV in bf16, or
      // for a part both in fp32 to its place in the workspace.
      float* const prt = w.part < 0 || !key_ok
                             ? nullptr
                             : win_part<D>(p, w.part, w.b, w.hk, w.kb, w.kw.load_row - w.k_start + kr);
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const uint32_t col = which == 0 ? kColDV : kColDK;
        const float mul = which == 0 ? 1.f : p.scale;
        __nv_bfloat16* const dst = which == 0 ? p.dv : p.dk;
#pragma unroll
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t a[32];
          ptx::tmem_ld32(tmem + lane_off + col + c4 * 32, a);
          ptx::tmem_wait_ld();
          if (key_ok && w.part >= 0) {
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
              ptx::st_global_v4(prt + which * D + c4 * 32 + q4 * 4, __float_as_uint(__uint_as_float(a[4 * q4]) * mul),
                                __float_as_uint(__uint_as_float(a[4 * q4 + 1]) * mul),
                                __float_as_uint(__uint_as_float(a[4 * q4 + 2]) * mul),
                                __float_as_uint(__uint_as_float(a[4 * q4 + 3]) * mul));
          } else if (key_ok) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              uint32_t wv[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                wv[e] = ptx::pack_bf16x2(__uint_as_float(a[8 * q4 + 2 * e]) * mul,
                                         __uint_as_float(a[8 * q4 + 2 * e + 1]) * mul);
              ptx::st_global_v4(dst + krow + c4 * 32 + q4 * 8, wv[0], wv[1], wv[2], wv[3]);
            }
          }
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(L::kBarAccEmpty));
      ++uc;
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}


// Before and after the key-block kernel.  Both give 16 (d = 128) or 8 (d = 64)
// lanes to a row, 16 bytes of bf16 a lane, and are bound by their bytes (the
// accumulator's 4 d, and 4 d of o and dout, a row).  PASSES rows a group, 128 a block,
// where most rows are those of no sequence (a long and many short packed ones).
//
// -D_i, the scaled log-sum-exp negated and a cleared accumulator row for every
// entry of the tile order (see BwdParams): entries without a row of their own, and
// rows without keys, carry -inf, so that their P and dS are 0.
template <int D, bool VARLEN, bool SPLIT, int PASSES>
__global__ void __launch_bounds__(256) fa_win_prep_kernel(const WinBwdParams p) {
  grid_dependents_launch();
  constexpr int kLanes = D / 8;
  uint32_t block = blockIdx.x;
  if (VARLEN && p.order != nullptr && block-- == 0) {  // the first block lists the units
    win_bwd_list<SPLIT>(p);
    return;
  }
  const int lane = threadIdx.x % kLanes;
  const uint32_t rows = static_cast<uint32_t>(p.B) * p.H * p.nq_pad;  // less than 2^31
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
    const uint32_t row = (block * PASSES + pass) * (256 / kLanes) + threadIdx.x / kLanes;
    const bool in = row < rows;
    const int t = in ? row % p.nq_pad : 0;
    const uint32_t bh = in ? row / p.nq_pad : 0;
    const int h = bh % p.H;
    const int b = bh / p.H;
    int q_start, len_q, k_start, len_k;
    bool bad;
    win_bwd_seq<VARLEN>(p, b, q_start, len_q, k_start, len_k, bad);
    const int qb = t / kBwdBQ, c = t % kBwdBQ;
    if (qb * kBwdBQ >= len_q) {  // a query block of no sequence: nobody reads it
      if (PASSES > 1) return;    // the block's rows are those of one query block
      continue;                  // and the warp's
    }
    const RowWindow qw = make_window<VARLEN>(q_start, q_start + len_q, q_start + qb * kBwdBQ, kBwdBQ);
    float acc = 0.f, l2 = INFINITY;
    if (in && c >= qw.lo && c < qw.hi) {
      const int i = qw.load_row - q_start + c;
      const size_t prow = VARLEN ? static_cast<size_t>(qw.load_row + c) : static_cast<size_t>(b) * p.Nq + i;
      const size_t off = (prow * p.H + h) * D + lane * 8;
      const uint4 a = *reinterpret_cast<const uint4*>(p.dout + off), o = *reinterpret_cast<const uint4*>(p.o + off);
      const uint32_t av[4] = {a.x, a.y, a.z, a.w}, ov[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc += __uint_as_float(av[e] << 16) * __uint_as_float(ov[e] << 16);
        acc += __uint_as_float(av[e] & 0xffff0000u) * __uint_as_float(ov[e] & 0xffff0000u);
      }
      const float L = p.lse[static_cast<size_t>(bh) * p.Nq + i];
      if (L > -INFINITY) l2 = L * 1.44269504088896340736f;
      else acc = 0.f;
    }
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (!in) continue;
    if (lane == 0) {
      p.delta[row] = -acc;
      p.lse2[row] = -l2;
    }
    float* const dst = p.dq_acc + static_cast<size_t>(row) * D + lane * 4;
    ptx::st_global_v4(dst, 0u, 0u, 0u, 0u);
    ptx::st_global_v4(dst + D / 2, 0u, 0u, 0u, 0u);
  }
}

// dq = bf16(scale * accumulator).
template <int D, bool VARLEN, int PASSES>
__device__ __forceinline__ void win_bwd_dq(const WinBwdParams& p, uint32_t block) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x % kLanes;
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
    const uint32_t row = (block * PASSES + pass) * (256 / kLanes) + threadIdx.x / kLanes;
    if (row >= static_cast<uint32_t>(p.B) * p.H * p.nq_pad) return;
    const int i = row % p.nq_pad;
    const uint32_t bh = row / p.nq_pad;
    const int h = bh % p.H;
    const int b = bh / p.H;
    int q_start, len_q, k_start, len_k;
    bool bad;
    win_bwd_seq<VARLEN>(p, b, q_start, len_q, k_start, len_k, bad);
    if (i >= len_q) {
      if (PASSES > 1 && i - i % kBwdBQ >= len_q) return;  // nor do the block's other rows
      continue;
    }
    const int qb = i / kBwdBQ;
    const RowWindow qw = make_window<VARLEN>(q_start, q_start + len_q, q_start + qb * kBwdBQ, kBwdBQ);
    const int t = qb * kBwdBQ + (q_start + i - qw.load_row);
    const size_t prow = VARLEN ? static_cast<size_t>(q_start + i) : static_cast<size_t>(b) * p.Nq + i;
    const float4* src = reinterpret_cast<const float4*>(p.dq_acc + (static_cast<size_t>(bh) * p.nq_pad + t) * D + lane * 8);
    const float4 x = src[0], y = src[1];
    ptx::st_global_v4(p.dq + (prow * p.H + h) * D + lane * 8, ptx::pack_bf16x2(x.x * p.scale, x.y * p.scale),
                      ptx::pack_bf16x2(x.z * p.scale, x.w * p.scale), ptx::pack_bf16x2(y.x * p.scale, y.y * p.scale),
                      ptx::pack_bf16x2(y.z * p.scale, y.w * p.scale));
  }
}

// dK and dV of the keys whose blocks are not one unit: the fp32 parts, added in
// their order, to bf16.  One warp per (sequence, key/value head, key);
// bound by reading the parts once (a few MB).
template <int D, bool VARLEN, bool SPLIT>
__device__ __forceinline__ void win_bwd_sum(const WinBwdParams& p, uint32_t block) {
  const int keys = (SPLIT ? p.num_kb : p.num_skb) * kBwdBK;
  const long long row = static_cast<long long>(block) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(p.B) * p.Hk * keys) return;
  const int key = static_cast<int>(row % keys);
  const int hk = static_cast<int>((row / keys) % p.Hk);
  const int b = static_cast<int>(row / keys / p.Hk);
  int q_start, len_q, k_start, len_k;
  bool bad;
  win_bwd_seq<VARLEN>(p, b, q_start, len_q, k_start, len_k, bad);
  if (key >= len_k) return;
  int qb0, nqb;
  const int kb = key / kBwdBK;
  const bool sink = !SPLIT || kb < p.num_skb;
  win_query_blocks(kb, len_q, len_k, p.window, sink, qb0, nqb);
  const int chunks = sink ? (nqb + p.chunk_qb - 1) / p.chunk_qb : 1;
  constexpr int kPer = 2 * D / 32;  // floats per lane: lanes 0-15 hold dV, 16-31 dK
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  auto add = [&](int part) {
    const float4* src = reinterpret_cast<const float4*>(win_part<D>(p, part, b, hk, kb, key)) + lane * (kPer / 4);
#pragma unroll
    for (int e = 0; e < kPer / 4; ++e) {
      const float4 x = src[e];
      acc[4 * e] += x.x;
      acc[4 * e + 1] += x.y;
      acc[4 * e + 2] += x.z;
      acc[4 * e + 3] += x.w;
    }
  };
  if constexpr (!SPLIT) {
    for (int c = 0; c < chunks; ++c) add(c);
  } else {
    for (int c = 0; c < chunks; ++c) {
      const int n = p.group * (sink ? min(nqb - c * p.chunk_qb, p.chunk_qb) : nqb);
      for (int s = 0; s < p.split; ++s)
        if (win_share(n, s, p.split) < win_share(n, s + 1, p.split)) add(c * p.split + s);
    }
  }
  const size_t prow = VARLEN ? static_cast<size_t>(k_start) + key : static_cast<size_t>(b) * p.Nk + key;
  __nv_bfloat16* const dst = (lane < 16 ? p.dv : p.dk) + (prow * p.Hk + hk) * D + (lane & 15) * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = ptx::pack_bf16x2(acc[e], acc[e + 1]);
}

// Behind the key-block kernel: the first sum_blocks blocks add parts, the others round
// dQ; the sums' latency hides behind dQ's bytes.
template <int D, bool VARLEN, bool SPLIT, int PASSES>
__global__ void __launch_bounds__(256, 6) fa_win_finish_kernel(const WinBwdParams p, uint32_t sum_blocks) {
  grid_dependency_wait();
  if (blockIdx.x < sum_blocks)
    win_bwd_sum<D, VARLEN, SPLIT>(p, blockIdx.x);
  else
    win_bwd_dq<D, VARLEN, PASSES>(p, blockIdx.x - sum_blocks);
}

}  // namespace fa
