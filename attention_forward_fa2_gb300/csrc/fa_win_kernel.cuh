// fa_win_kernel.cuh -- attention forward with a sliding window and sinks, sm_103a (GB300).
//
// What it computes: query i of a sequence stands at position p = i + len_k - len_q
// and sees the keys j <= p with p - j < window or j < sinks ("GPU 内核与
// FlashAttention" §14.4's causal mask, cut off behind the window, with the
// first keys kept);  O = softmax(scale Q K^T over those keys) V  and the fp32
// natural-log log-sum-exp of every row, by the online recurrence of §11.3.
// With `full` set every query stands at len_k - 1 (no causal border).
//
// Keys and values come dense, packed like the queries, or (KPAD: the dequantised
// cache) padded to whole key tiles per sequence with a length for each.
//
// The CTA is built like fa_fwd_kernel (fa_fwd_kernel.cuh: two 128-row query
// tiles of one head, softmax warpgroup per tile, MMA and load threads, epilogue
// warpgroup, the same shared and tensor memory layout); what differs is the
// sequence of key tiles.  A unit walks the steps j = 0 .. nsteps-1 over the key
// tiles
//     kt(j) = j            for j < ns     (tiles that hold sinks, below the windows)
//     kt(j) = j + gap      for j >= ns    (from the first tile of tile 0's window
//                                          to the diagonal of tile 1)
// and query tile t takes part in step j only when it sees a key of kt(j).  Where two
// query heads share their keys, the tiles of a unit are the same rows of two heads
// (`pair`): both see the same key tiles, and every step runs both.  Else they are
// 256 rows of one head; tile 1's window starts and ends one key tile after tile 0's,
// so each runs its own products.  Nothing runs for tiles between the sinks and the
// window.
// The work of a unit is thus bound by the window, whatever the length; what is
// lost is the masked part of the first and last key tile of the window and of
// the sink tile (window 1024, 64 sinks: 10 products of 128 x 128 for 8.5 x 128
// visible keys a row).
// Element masks are applied only in tiles that hold a border: the diagonal, the
// window's start, the end of the sinks, the sequence's end.
// Bound by each tile's chain S -> softmax -> P V hidden behind the other tile's, as the
// forward without a window: 1.03 us a pair of tiles and step.  Two sequences of 4096,
// 16 heads on 4 of d 128, window 512, 4 sinks: 60 us, tensor pipe 42 % busy; 512 units
// on 152 SMs leave the fourth round 3/8 full, border tiles take half as long again.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fa_f16.cuh"
#include "fa_fwd_kernel.cuh"
#include "ptx.cuh"

namespace fa {

// The steps of a unit that a query tile takes part in: j < s (tiles with sinks) and
// a <= j < e (its window).
struct WinSteps {
  int s, a, e;
};
// Key tiles [0, nsk) hold sinks; the query tile's window starts in key tile `lo`
// and its diagonal ends in `hi`; step j of the unit is key tile j for j < ns, else
// j + gap (gap > 0 only behind all sink tiles).
__host__ __device__ __forceinline__ WinSteps win_steps(int lo, int hi, int nsk, int ns, int gap) {
  WinSteps w;
  w.s = gap > 0 ? ns : (nsk < hi + 1 ? nsk : hi + 1);
  w.a = lo - gap;
  w.e = hi - gap + 1;
  return w;
}
__host__ __device__ __forceinline__ bool win_sees(const WinSteps& w, int j) { return j < w.s || (j >= w.a && j < w.e); }
// The last such step in [j0, j1), -1 if there is none.
__host__ __device__ __forceinline__ int win_last(const WinSteps& w, int j0, int j1) {
  const int x = (j1 < w.e ? j1 : w.e) - 1, y = (j1 < w.s ? j1 : w.s) - 1;
  return x >= w.a && x >= j0 ? x : y >= j0 ? y : -1;
}

// The low n bits set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u; }

struct WinUnit {
  int b, h, hk;
  int dh;         // query tile t is of head h + t * dh
  int q_start, q_end, k_start, k_end;
  int q_row0;
  int off;        // position of query i is i + off
  int ns, gap;    // steps [0, ns) are key tiles 0..ns-1; step j >= ns is key tile j + gap
  int nsteps;
  int j0, j1;     // the steps of this item: all, or (KPAD) a range of them
  int place;      // -1: o and lse are written; else the item's place for partial results
  int lse_base, lse_next;  // of query tile t: lse_base + t * lse_next
  bool run, nokeys;
  bool rows[kQT];    // tile t has rows
  bool active[kQT];  // tile t has rows and sees keys of these steps
  WinSteps st[kQT];  // empty where tile t is not active
  int last[kQT];     // the last step that tile t takes part in
  RowWindow qwin[kQT];
  __device__ __forceinline__ int kt(int j) const { return j < ns ? j : j + gap; }
  __device__ __forceinline__ bool sees(int t, int j) const { return win_sees(t == 0 ? st[0] : st[1], j); }
};

struct WinParams {
  int B, Nq, Nk, H;            // variable-length form: Nq / Nk are the maximum lengths
  int group;                   // query heads per key/value head
  int window, sinks;
  int full;                    // 1: no causal border
  int by_block;                // 1: units numbered query block by query block
  int whole;                   // KPAD: units are not cut (see WinItem)
  int pair;                    // 1: the query tiles of a unit are the same rows of two heads
  int tiles;                   // query tiles of a unit: 2, or 1 (few units)
  int unit_rows;               // query rows of a unit in its sequence: kBR * kQT, or kBR (pair, one tile)
  int unit_heads;              // units across the heads: H, or H / 2 (pair)
  int num_mblocks;             // ceil(Nq / unit_rows)
  int num_units;               // B * unit_heads * num_mblocks
  int total_q, total_k;        // variable-length form: packed rows (sequences past them are rejected)
  const int* cu_q;             // variable-length form: int32 [B + 1]
  const int* cu_k;             // KPAD: key lengths, int32 [B]
  float* lse;                  // [B, H, Nq] fp32
  __nv_bfloat16* o;
  float scale, scale_log2;
  float rescale_threshold;
  // KPAD: a unit cut by the borders of CTA c's range of steps lies at place 2c (begun
  // by an earlier CTA) or 2c + 1 (begun by c, ended later); cut[c] names the unit
  // that ends in c and was begun by an earlier CTA.
  int2* cut;                   // [ctas]: unit (-1: none), CTA that began it
  float* part_o;               // [2 ctas, 256, d], normalised
  float* part_lse;             // [2 ctas, 256]
  unsigned long long timeout_ns;
  int* status;
};

// Row of the unit (0 .. 255) that holds packed row `row` of query tile t.
__device__ __forceinline__ int win_unit_row(const WinUnit& w, int t, int row) {
  return row - w.q_row0 + (w.dh ? t * kBR : 0);
}

// Restricts a unit to the steps [j0, j1).
__device__ __forceinline__ void win_restrict(WinUnit& w, int j0, int j1, int place) {
  w.j0 = j0;
  w.j1 = j1;
  w.place = place;
#pragma unroll
  for (int t = 0; t < kQT; ++t) {
    w.last[t] = win_last(w.st[t], j0, j1);
    w.active[t] = w.last[t] >= 0;
  }
  w.run = w.active[0] || w.active[1];
}

template <int BC, bool VARLEN, bool KPAD>
__device__ __forceinline__ WinUnit win_decode(const WinParams& p, int u) {
  WinUnit w;
  // Head by head, so that the units in flight share keys in L2; packed batches
  // last query blocks first (under a long window the longest units), so that the
  // running CTAs even out at the end.  by_block (dense, windows over half the keys
  // or more): the longest block of every head first, which keeps the round-robin
  // over units of falling work even.
  int mb = u % p.num_mblocks, r = u / p.num_mblocks;
  if (p.by_block) {
    mb = u / (p.B * p.unit_heads);
    r = u % (p.B * p.unit_heads);
  }
  if (VARLEN || p.by_block) mb = p.num_mblocks - 1 - mb;
  w.dh = p.pair;
  w.h = (r % p.unit_heads) << p.pair;
  w.b = r / p.unit_heads;
  w.hk = w.h / p.group;
  w.q_start = 0;
  w.q_end = p.Nq;
  w.k_start = 0;
  w.k_end = p.Nk;
  bool bad = false;
  if constexpr (VARLEN || KPAD) {
    if constexpr (VARLEN) {
      w.q_start = p.cu_q[w.b];
      w.q_end = p.cu_q[w.b + 1];
    }
    if constexpr (KPAD) {
      w.k_end = p.cu_k[w.b];
    } else {
      w.k_start = p.cu_k[w.b];
      w.k_end = p.cu_k[w.b + 1];
    }
    const int len_q = w.q_end - w.q_start, len_k = w.k_end - w.k_start;
    bad = len_q < 0 || len_k < 0 || len_q > p.Nq || len_k > p.Nk || w.q_start < 0 || w.k_start < 0 ||
          (VARLEN && w.q_start > p.total_q - len_q) || (VARLEN && !KPAD && w.k_start > p.total_k - len_k);
  }
  const int len_k = bad ? 0 : w.k_end - w.k_start;
  w.q_row0 = w.q_start + mb * p.unit_rows;
  w.off = (w.k_end - w.k_start) - (w.q_end - w.q_start);
  w.lse_base = (w.b * p.H + w.h) * p.Nq;
  w.lse_next = p.pair ? p.Nq : 0;
  const bool has_rows = !bad && w.q_row0 < w.q_end;
  const int nsk = (min(p.sinks, len_k) + BC - 1) / BC;  // key tiles that hold sinks
  int first = 0x7fffffff, end = -1, lo[kQT], hi[kQT];
#pragma unroll
  for (int t = 0; t < kQT; ++t) {
    const int r0 = w.q_row0 + (p.pair ? 0 : t * kBR);
    w.qwin[t] = make_window<VARLEN>(w.q_start, w.q_end, r0, kBR);
    w.rows[t] = has_rows && r0 < w.q_end && t < p.tiles;
    // Positions of the tile's first and last row of its own.
    const int p0 = p.full ? len_k - 1 : w.qwin[t].load_row - w.q_start + w.qwin[t].lo + w.off;
    const int p1 = p.full ? len_k - 1 : w.qwin[t].load_row - w.q_start + w.qwin[t].hi - 1 + w.off;
    w.active[t] = w.rows[t] && len_k > 0 && p1 >= 0;
    lo[t] = max(0, p0 - p.window + 1) / BC;  // window <= the longest sequence
    hi[t] = p1 < 0 ? -1 : p1 / BC;           // p1 <= len_k - 1
    if (w.active[t]) {
      first = min(first, lo[t]);
      end = max(end, hi[t]);
    }
  }
  w.run = w.active[0] || w.active[1];
  w.nokeys = has_rows && len_k == 0;
  w.ns = w.run ? min(nsk, first) : 0;
  w.gap = w.run ? first - w.ns : 0;
  w.nsteps = w.run ? w.ns + end - first + 1 : 0;
#pragma unroll
  for (int t = 0; t < kQT; ++t) w.st[t] = w.active[t] ? win_steps(lo[t], hi[t], nsk, w.ns, w.gap) : WinSteps{0, 0, 0};
  win_restrict(w, 0, w.nsteps, -1);
  if (bad && mb == 0 && w.h == 0) {
    if (threadIdx.x == 0 || threadIdx.x == 13 * 32) record_error(p.status, kErrBadSeqlens, 0);
  }
  return w;
}

// Items reach the roles in one of three ways.
//   Dense: units blockIdx.x + k * gridDim.x on a grid of one CTA per SM.
//   Packed: one CTA per unit is launched, a running CTA takes over units not yet
//     started (cluster launch control), through the ring of fa_fwd_kernel.cuh.
//   KPAD (few queries, many keys): the steps of all units, laid end to end, are cut
//     into one range per SM; the load thread hands units, and the parts of units
//     cut by the range's borders, through the ring; fa_win_join_kernel joins the
//     parts.  (Three prompts of at most 1024 queries over 8192 keys, 16 heads: as
//     whole units 195 us, most SMs idle behind the longest; cut 98.)  With many
//     units an SM (`whole`) they are handed out whole, as packed ones are, which
//     keeps the units in flight on the keys of a few heads in L2.
struct WinItem {
  int u, j0, j1, place;  // u < 0: no more
};

// Shared memory behind the tiles: the ring's items, and the scan of the lengths.
template <int D, int STAGES>
struct WinSmem {
  using L = SmemLayout<D, 128, STAGES>;
  static constexpr int kOffItems = (L::kBytes + 15) / 16 * 16;
  static constexpr int kOffScan = kOffItems + kItemSlots * 16;
  static constexpr int kBytes = kOffScan + (kThreads / 32 + 2) * 8;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget exceeded");
};

// KPAD: steps of unit (b, query block mb) of any head, at least one where it has rows,
// behind kUnitCost more that stand for what its beginning and end take (with them
// left out, SMs with three or four short units ended 20 % behind those with one).
constexpr int kUnitCost = 2;
template <bool VARLEN>
__device__ __forceinline__ int win_flat(const WinParams& p, int b, int mb) {
  const WinUnit w = win_decode<128, VARLEN, true>(p, b * p.unit_heads * p.num_mblocks + (VARLEN ? p.num_mblocks - 1 - mb : mb));
  return w.rows[0] ? kUnitCost + max(w.nsteps, 1) : 0;
}

#define FA_WIN_FOR_EACH_ITEM(it) \
  for (WinItem it = next_item(-1); it.u >= 0 && it.u < p.num_units && ok; it = next_item(it.u))
#define FA_WIN_UNIT(it)                                       \
  WinUnit w = win_decode<BC, VARLEN, KPAD>(p, (it).u);        \
  if constexpr (KPAD) {                                       \
    if (!p.whole) win_restrict(w, (it).j0, (it).j1, (it).place); \
  }

template <int D, int STAGES, bool VARLEN, bool KPAD>
__global__ void __launch_bounds__(kThreads, 1)
    fa_win_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                  const WinParams p) {
  constexpr int BC = 128;
  using L = SmemLayout<D, BC, STAGES>;
  constexpr int kTmemCols = 512;
  constexpr bool kKShift = VARLEN && !KPAD;  // key tiles of packed sequences are shifted back at the end
  constexpr int kDPanels = D / kPanel;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw_base);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  const uint32_t bar0 = base + L::kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  float* const s_invl = reinterpret_cast<float*>(gbase + L::kOffInvL);
  volatile uint32_t* const s_tmem = reinterpret_cast<volatile uint32_t*>(gbase + L::kOffTmem);
  volatile int* const s_abort = reinterpret_cast<volatile int*>(gbase + L::kOffAbort);
  volatile WinItem* const s_items = reinterpret_cast<volatile WinItem*>(gbase + WinSmem<D, STAGES>::kOffItems);
  const uint64_t tmo = p.timeout_ns;
  uint32_t item_n_ = 0;
  constexpr bool kRing = VARLEN || KPAD;
  auto next_item = [&](int prev) -> WinItem {
    if constexpr (!kRing) {
      return WinItem{prev < 0 ? static_cast<int>(blockIdx.x) : prev + static_cast<int>(gridDim.x), 0, 0, -1};
    } else {
      const bool whole = warp != 12;  // the MMA thread reads alone, the other roles warp-wide
      const uint32_t slot = item_n_ % kItemSlots, parity = (item_n_ / kItemSlots) & 1u;
      const bool got = whole ? ptx::mbar_wait_warp(bar(L::kBarItemFull) + 8u * slot, parity, s_abort, tmo)
                             : ptx::mbar_wait(bar(L::kBarItemFull) + 8u * slot, parity, s_abort, tmo);
      if (!got) {
        if (!whole || lane == 0) record_error(p.status, kErrTimeout, kSiteItem);
        return WinItem{-1, 0, 0, -1};
      }
      const WinItem it{s_items[slot].u, s_items[slot].j0, s_items[slot].j1, s_items[slot].place};
      if (whole) __syncwarp();
      if (!whole || lane == 0) ptx::mbar_arrive(bar(L::kBarItemEmpty) + 8u * slot);
      ++item_n_;
      return it;
    }
  };

  // ------------------------------------------------------------------ setup
  if (warp == 13 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    ptx::prefetch_tmap(&tm_o);
  }
  if (threadIdx.x == 0) {
    *s_abort = 0;
    ptx::mbar_init(bar(L::kBarQFull), 1);
    ptx::mbar_init(bar(L::kBarQEmpty), 1);
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(bar(L::kBarKVFull + s), 1);
      ptx::mbar_init(bar(L::kBarKVEmpty + s), 1);
    }
    for (int t = 0; t < kQT; ++t) {
      ptx::mbar_init(bar(L::kBarSFull + t), 1);
      ptx::mbar_init(bar(L::kBarPFull + t), kBR);
      ptx::mbar_init(bar(L::kBarLReady + t), kBR);
      ptx::mbar_init(bar(L::kBarOFinal + t), 1);
      ptx::mbar_init(bar(L::kBarOEmpty + t), kBR);
    }
    ptx::mbar_init(bar(L::kBarTeardown), 1);
    for (int i = 0; i < kItemSlots; ++i) {
      ptx::mbar_init(bar(L::kBarItemFull + i), 1);
      ptx::mbar_init(bar(L::kBarItemEmpty + i), kItemConsumers);
    }
    ptx::mbar_init(bar(L::kBarClc), 1);
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(base + L::kOffTmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  // KPAD: this CTA's range [begin, end) of the steps of all units (sequence by
  // sequence, query blocks in order, heads innermost), from a scan of the lengths.
  long long begin = 0, end = 0, span = 1;
  long long* const s_scan = reinterpret_cast<long long*>(gbase + WinSmem<D, STAGES>::kOffScan);
  if (KPAD && !p.whole) {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    auto flat = [&](int b) -> long long {
      long long sum = 0;
      for (int mb = 0; mb < p.num_mblocks; ++mb) sum += win_flat<VARLEN>(p, b, mb);
      return sum * p.unit_heads;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += flat(b);
    long long pre = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, pre, k);
      if (lane >= k) pre += v;
    }
    if (lane == 31) s_scan[warp] = pre;
    __syncthreads();
    long long total = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) pre += s_scan[k];
      total += s_scan[k];
    }
    pre -= mine;
    span = max((total + gridDim.x - 1) / gridDim.x, 1LL);
    begin = blockIdx.x * span;
    end = min(total, begin + span);
    if (begin < end && begin >= pre && begin < pre + mine) {
      long long at = pre;
      int b = b0;
      for (; b < b1; ++b) {
        const long long f = flat(b);
        if (begin < at + f) break;
        at += f;
      }
      s_scan[kThreads / 32] = b;
      s_scan[kThreads / 32 + 1] = at;
    }
    if (threadIdx.x == 0) p.cut[blockIdx.x] = make_int2(-1, 0);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= 12) {
    ptx::setmaxnreg_dec<RegSplit<VARLEN>::kOther>();
    if (warp == 13 && lane == 0) {
      // =========================================================== TMA loads
      uint32_t qcount = 0, g = 0;
      bool ok = true;
      uint32_t n_pub = 0, n_clc = 0;
      bool clc_pending = false;
      auto publish = [&](const WinItem& item) -> bool {
        const uint32_t slot = n_pub % kItemSlots;
        if (!ptx::mbar_wait(bar(L::kBarItemEmpty + slot), ((n_pub / kItemSlots) & 1u) ^ 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kSiteItem);
          return false;
        }
        s_items[slot].u = item.u;
        s_items[slot].j0 = item.j0;
        s_items[slot].j1 = item.j1;
        s_items[slot].place = item.place;
        ptx::mbar_arrive(bar(L::kBarItemFull + slot));
        ++n_pub;
        return true;
      };
      auto request = [&]() {
        ptx::fence_proxy_async_smem();  // the previous answer was read before it is overwritten
        ptx::mbar_arrive_expect_tx(bar(L::kBarClc), 16);
        ptx::clc_try_cancel(base + L::kOffClc, bar(L::kBarClc));
        clc_pending = true;
      };
      // KPAD: where the range stands: sequence, its first step, query block, its first step.
      int kb = 0, kmb = 0, kw = 0;
      long long kat = 0, pos = begin;
      if (KPAD && !p.whole) {
        if (begin < end) {
          kb = static_cast<int>(s_scan[kThreads / 32]);
          kat = s_scan[kThreads / 32 + 1];
          kw = win_flat<VARLEN>(p, kb, 0);
        }
      }
      auto range_item = [&]() -> WinItem {
        while (pos < end) {
          while (pos >= kat + static_cast<long long>(kw) * p.unit_heads) {
            kat += static_cast<long long>(kw) * p.unit_heads;
            if (++kmb == p.num_mblocks) {
              kmb = 0;
              ++kb;
            }
            kw = win_flat<VARLEN>(p, kb, kmb);
          }
          const int h = static_cast<int>((pos - kat) / kw), at = static_cast<int>((pos - kat) % kw);
          const int to = static_cast<int>(min(static_cast<long long>(kw), at + (end - pos)));
          const long long step0 = pos - at + kUnitCost;  // where the unit's steps begin
          pos += to - at;
          const int j0 = max(at - kUnitCost, 0), j1 = to - kUnitCost;
          if (j1 <= j0) continue;  // the range ends ahead of the unit's first step
          const int u = (kb * p.unit_heads + h) * p.num_mblocks + (VARLEN ? p.num_mblocks - 1 - kmb : kmb);
          const int c = static_cast<int>(blockIdx.x);
          if (j0 > 0 && to == kw) p.cut[c] = make_int2(u, static_cast<int>(step0 / span));
          return WinItem{u, j0, j1, j0 > 0 ? 2 * c : to < kw ? 2 * c + 1 : -1};
        }
        return WinItem{-1, 0, 0, -1};
      };
      WinItem cur{static_cast<int>(blockIdx.x), 0, 0, -1};
      const bool ranges = KPAD && !p.whole;
      if (ranges) cur = range_item();
      if constexpr (KPAD) grid_dependency_wait();  // the copy of the keys is made by the kernel before this one
      if constexpr (kRing) ok = publish(cur);
      if (kRing && !ranges && ok) request();
#pragma unroll 1
      while (ok && cur.u >= 0 && cur.u < p.num_units) {
        FA_WIN_UNIT(cur)
        if (w.run) {
          if (!ptx::mbar_wait(bar(L::kBarQEmpty), (qcount & 1u) ^ 1u, s_abort, tmo)) {
            record_error(p.status, kErrTimeout, kSiteLoadQ);
            break;
          }
          ptx::mbar_arrive_expect_tx(bar(L::kBarQFull),
                                     (w.active[0] ? L::kQTileBytes : 0) + (w.active[1] ? L::kQTileBytes : 0));
          ++qcount;
#pragma unroll
          for (int t = 0; t < kQT; ++t) {
            if (!w.active[t]) continue;
#pragma unroll
            for (int pnl = 0; pnl < kDPanels; ++pnl) {
              const uint32_t dst = base + L::kOffQ + t * L::kQTileBytes + pnl * L::kQPanelBytes;
              if constexpr (VARLEN)
                ptx::tma_load_3d(dst, &tm_q, bar(L::kBarQFull), pnl * kPanel, w.h + t * w.dh, w.qwin[t].load_row);
              else
                ptx::tma_load_4d(dst, &tm_q, bar(L::kBarQFull), pnl * kPanel, w.h + t * w.dh, w.qwin[t].load_row, w.b);
            }
          }
          auto load_tile = [&](uint32_t dst0, const CUtensorMap* tm, uint32_t full, int kt) {
            const RowWindow kw = make_window<kKShift>(w.k_start, w.k_end, w.k_start + kt * BC, BC);
#pragma unroll
            for (int pnl = 0; pnl < kDPanels; ++pnl) {
              const uint32_t dst = dst0 + pnl * L::kKVPanelBytes;
              if constexpr (kKShift)
                ptx::tma_load_3d(dst, tm, full, pnl * kPanel, w.hk, kw.load_row);
              else
                ptx::tma_load_4d(dst, tm, full, pnl * kPanel, w.hk, kw.load_row, w.b);
            }
          };
#pragma unroll 1
          for (int j = w.j0; j <= w.j1; ++j) {
            const uint32_t slot = g % STAGES;
            if (!ptx::mbar_wait(bar(L::kBarKVEmpty + slot), ((g / STAGES) & 1u) ^ 1u, s_abort, tmo)) {
              record_error(p.status, kErrTimeout, kSiteLoadKV);
              ok = false;
              break;
            }
            const uint32_t bytes = (j < w.j1 ? L::kKVTileBytes : 0) + (j > w.j0 ? L::kKVTileBytes : 0);
            const uint32_t full = bar(L::kBarKVFull + slot);
            ptx::mbar_arrive_expect_tx(full, bytes);
            ++g;
            const uint32_t sbase = base + L::kOffKV + slot * L::kSlotBytes;
            if (j < w.j1) load_tile(sbase, &tm_k, full, w.kt(j));
            if (j > w.j0) load_tile(sbase + L::kKVTileBytes, &tm_v, full, w.kt(j - 1));
          }
          if (!ok) break;
        }
        if (ranges) {
          cur = range_item();
          if (!publish(cur)) break;
        } else if constexpr (kRing) {
          if (!ptx::mbar_wait(bar(L::kBarClc), n_clc & 1u, s_abort, tmo)) {
            record_error(p.status, kErrTimeout, kSiteItem);
            break;
          }
          ++n_clc;
          clc_pending = false;
          cur.u = ptx::clc_cancelled_x(base + L::kOffClc);
          // Units without rows (packed batches are walked up to the longest length) go no
          // further than here.
          while (cur.u >= 0 && cur.u < p.num_units && !win_decode<BC, VARLEN, KPAD>(p, cur.u).rows[0]) {
            request();
            if (!ptx::mbar_wait(bar(L::kBarClc), n_clc & 1u, s_abort, tmo)) {
              record_error(p.status, kErrTimeout, kSiteItem);
              ok = false;
              break;
            }
            ++n_clc;
            clc_pending = false;
            cur.u = ptx::clc_cancelled_x(base + L::kOffClc);
          }
          if (!ok || !publish(cur)) break;
          if (cur.u >= 0) request();
        } else {
          cur.u += gridDim.x;
        }
      }
      if constexpr (KPAD) grid_dependents_launch();  // the join's blocks may be set up; they wait for this grid's end
      // Nothing may land in shared memory after the CTA is gone.
      if (clc_pending) ptx::mbar_wait_drain(bar(L::kBarClc), n_clc & 1u, tmo);
      if (qcount > 0) ptx::mbar_wait_drain(bar(L::kBarQFull), (qcount - 1) & 1u, tmo);
      for (uint32_t s = 0; s < STAGES; ++s) {
        if (g > s) {
          const uint32_t rounds = (g - 1 - s) / STAGES + 1;
          ptx::mbar_wait_drain(bar(L::kBarKVFull + s), (rounds - 1) & 1u, tmo);
        }
      }
    } else if (warp == 12 && lane == 0) {
      // ========================================================== MMA issue
      constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(kBR, BC, 0, 0);
      constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(kBR, D, 0, 1);
      uint32_t qcount = 0, g = 0;
      uint32_t pc[kQT] = {0, 0};  // P-full completions consumed, per tile
      uint32_t uc[kQT] = {0, 0};  // units with the tile active, per tile
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t parity, int site) -> bool {
        if (ptx::mbar_wait(b, parity, s_abort, tmo)) return true;
        record_error(p.status, kErrTimeout, site);
        ok = false;
        return false;
      };
#pragma unroll 1
      FA_WIN_FOR_EACH_ITEM(it) {
        FA_WIN_UNIT(it)
        if (!w.run) continue;
        if (!wait(bar(L::kBarQFull), qcount & 1u, kSiteMmaQ)) break;
        ++qcount;
        ptx::tc_fence_after();
        bool begun[kQT] = {false, false};  // O_t holds a partial sum of this unit
        bool held[kQT] = {false, false};   // P_t of the previous step waits for its product
#pragma unroll 1
        for (int j = w.j0; j <= w.j1 && ok; ++j) {
          const uint32_t slot = g % STAGES;
          if (!wait(bar(L::kBarKVFull + slot), (g / STAGES) & 1u, kSiteMmaK)) break;
          ptx::tc_fence_after();
          const uint32_t k_base = base + L::kOffKV + slot * L::kSlotBytes;
          const uint32_t v_base = k_base + L::kKVTileBytes;
#pragma unroll
          for (int t = 0; t < kQT; ++t) {
            const uint32_t tS = tmem + static_cast<uint32_t>(t * BC);
            const uint32_t tP = tS + BC / 2;
            const uint32_t tO = tmem + static_cast<uint32_t>(2 * BC + t * D);
            if (held[t]) {
              // O_t += P_t(j-1) V(j-1), once P is written and O rescaled.
              if (!wait(bar(L::kBarPFull + t), pc[t] & 1u, kSiteMmaP)) break;
              ++pc[t];
              if (!begun[t] && !wait(bar(L::kBarOEmpty + t), (uc[t] & 1u) ^ 1u, kSiteMmaOEmpty)) break;
              ptx::tc_fence_after();
              const uint64_t vdesc = ptx::sw128_desc(v_base, L::kKVPanelBytes, 1024);
#pragma unroll
              for (int kk = 0; kk < BC / 16; ++kk)
                ptx::mma_ts(tO, tP + kk * 8, vdesc + static_cast<uint64_t>(kk * 128), idesc_pv,
                            (begun[t] || kk > 0) ? 1u : 0u);
              begun[t] = true;
              if (j - 1 == w.last[t]) ptx::mma_commit(bar(L::kBarOFinal + t));
            }
            held[t] = j < w.j1 && w.sees(t, j);
            if (held[t]) {
              // S_t = Q_t K(j)^T
              const uint64_t qdesc = ptx::sw128_desc(base + L::kOffQ + t * L::kQTileBytes, 16, 1024);
              const uint64_t kdesc = ptx::sw128_desc(k_base, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off_q = (kk / 4) * L::kQPanelBytes + (kk % 4) * 32;
                const uint32_t off_k = (kk / 4) * L::kKVPanelBytes + (kk % 4) * 32;
                ptx::mma_ss(tS, qdesc + static_cast<uint64_t>(off_q >> 4), kdesc + static_cast<uint64_t>(off_k >> 4),
                            idesc_qk, kk > 0 ? 1u : 0u);
              }
              ptx::mma_commit(bar(L::kBarSFull + t));
            }
          }
          if (!ok) break;
          if (j == w.j1 - 1) ptx::mma_commit(bar(L::kBarQEmpty));
          ptx::mma_commit(bar(L::kBarKVEmpty + slot));
          ++g;
        }
#pragma unroll
        for (int t = 0; t < kQT; ++t) uc[t] += w.active[t] ? 1u : 0u;
      }
      // Teardown: all MMAs must be complete before TMEM is released.
      ptx::mma_commit(bar(L::kBarTeardown));
      if (!ptx::mbar_wait_drain(bar(L::kBarTeardown), 0, tmo)) record_error(p.status, kErrTimeout, kSiteTeardown);
    }
  } else if (warp < 8) {
    ptx::setmaxnreg_inc<RegSplit<VARLEN>::kSoftmax>();
    // ================================================================ softmax
    const int t = warp >> 2;
    const int row = ((warp & 3) << 5) + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(t * BC);
    const uint32_t tP = tS + BC / 2;
    const float c2 = p.scale_log2;
    const float accept_sum = exp2f(p.rescale_threshold) * 0.9990234375f;
    uint32_t sc = 0;      // S-full completions consumed
    uint32_t units = 0;   // units of this tile finished
    bool ok = true;
#pragma unroll 1
    FA_WIN_FOR_EACH_ITEM(it) {
      FA_WIN_UNIT(it)
      const RowWindow qw = t == 0 ? w.qwin[0] : w.qwin[1];
      // Place of this row's partial results (row of the unit).
      const size_t part = KPAD && w.place >= 0
                              ? static_cast<size_t>(w.place) * (kBR * kQT) + win_unit_row(w, t, qw.load_row + row)
                              : 0;
      if (!(t == 0 ? w.active[0] : w.active[1])) {
        // No key of these steps in sight: a part of weight zero.
        if (KPAD && w.place >= 0 && (t == 0 ? w.rows[0] : w.rows[1]) && row >= qw.lo && row < qw.hi)
          p.part_lse[part] = -INFINITY;
        continue;
      }
      // Positions of this row and of the tile's first and last row of its own.
      const int len_k = w.k_end - w.k_start;
      const int pos = p.full ? len_k - 1 : qw.load_row - w.q_start + row + w.off;
      const int pos_first = p.full ? len_k - 1 : qw.load_row - w.q_start + qw.lo + w.off;
      const int pos_last = p.full ? len_k - 1 : qw.load_row - w.q_start + qw.hi - 1 + w.off;
      float m_ref = -INFINITY;
      float l = 0.f;
      int taken = 0;  // steps of this unit taken part in
#pragma unroll 1
      for (int j = w.j0; j < w.j1; ++j) {
        if (!w.sees(t, j)) continue;
        if (!ptx::mbar_wait_warp(bar(L::kBarSFull + t), sc & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kSiteSoftS);
          ok = false;
          break;
        }
        ++sc;
        ptx::tc_fence_after();
        const RowWindow kw = make_window<kKShift>(w.k_start, w.k_end, w.k_start + w.kt(j) * BC, BC);
        const int kbase = kw.load_row - w.k_start;  // key of column 0 (sequence index)
        const bool border = kw.lo != 0 || kw.hi != BC || kbase + BC - 1 > pos_first ||
                            (kbase <= pos_last - p.window && kbase + BC > p.sinks);
        float s[BC];
        uint32_t pk[BC / 2];
        auto exp_range = [&](int c0, int c1, float ng, uint64_t (&acc)[4]) {
          const uint64_t c2x2 = ptx::f2_pack(c2, c2);
          const uint64_t negx2 = ptx::f2_pack(ng, ng);
#pragma unroll
          for (int c = c0; c < c1; c += 2) {
            float x0, x1;
            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[c], s[c + 1]), c2x2, negx2), x0, x1);
            const float e0 = ptx::ex2(x0), e1 = ptx::ex2(x1);
            acc[(c >> 1) & 3] = ptx::f2_add(acc[(c >> 1) & 3], ptx::f2_pack(e0, e1));
            pk[c >> 1] = ptx::pack_bf16x2(e0, e1);
          }
        };
        auto sum_acc = [&](const uint64_t (&acc)[4]) -> float {
          float a0, a1, a2, a3, a4, a5, a6, a7;
          ptx::f2_unpack(acc[0], a0, a1);
          ptx::f2_unpack(acc[1], a2, a3);
          ptx::f2_unpack(acc[2], a4, a5);
          ptx::f2_unpack(acc[3], a6, a7);
          return ((a0 + a1) + (a2 + a3)) + ((a4 + a5) + (a6 + a7));
        };
        // The speculative maximum of fa_fwd_kernel: exponentials against the
        // current reference first; a block sum of at most 2^T proves that the
        // rescale rule leaves the reference in place.  Tiles with a border, and
        // a row's first, go another way below.
        float alpha = 1.f, lblk = 0.f;
        bool slow = border || __all_sync(0xffffffffu, m_ref == -INFINITY);
        if (!slow) {
          const float ng_ref = m_ref == -INFINITY ? 0.f : -m_ref * c2;
          uint32_t sr[BC];
#pragma unroll
          for (int c = 0; c < BC / 64; ++c) ptx::tmem_ld32(tS + c * 32, &sr[c * 32]);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int c = BC / 64; c < BC / 32; ++c) ptx::tmem_ld32(tS + c * 32, &sr[c * 32]);
#pragma unroll
          for (int c = 0; c < BC / 2; ++c) s[c] = __uint_as_float(sr[c]);
          uint64_t acc[4] = {0, 0, 0, 0};
          exp_range(0, BC / 2, ng_ref, acc);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int c = BC / 2; c < BC; ++c) s[c] = __uint_as_float(sr[c]);
          exp_range(BC / 2, BC, ng_ref, acc);
          lblk = sum_acc(acc);
          slow = __any_sync(0xffffffffu, m_ref == -INFINITY || !(lblk <= accept_sum));
        }
        if (slow) {
          uint32_t sr[BC];
#pragma unroll
          for (int c = 0; c < BC / 32; ++c) ptx::tmem_ld32(tS + c * 32, &sr[c * 32]);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < BC; ++c) s[c] = __uint_as_float(sr[c]);
          if (border) {
            // The row's visible columns as 32-bit words, [a, e) (window and diagonal)
            // and [kw.lo, f) (sinks): a bit test and a select per score (four
            // comparisons per score made a border tile cost several others).
            const int e = min(kw.hi, pos - kbase + 1);
            const int a = max(kw.lo, pos - p.window - kbase + 1);
            const int f = min(e, p.sinks - kbase);
#pragma unroll
            for (int c0 = 0; c0 < BC; c0 += 32) {
              const uint32_t seen = (bits_below(e - c0) & ~bits_below(a - c0)) | (bits_below(f - c0) & ~bits_below(kw.lo - c0));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if ((seen & (1u << c)) == 0u) s[c0 + c] = -INFINITY;
            }
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < BC; c += 8) {
            mx[0] = ptx::fmax3(mx[0], s[c], s[c + 1]);
            mx[1] = ptx::fmax3(mx[1], s[c + 2], s[c + 3]);
            if (c + 4 < BC) {
              mx[2] = ptx::fmax3(mx[2], s[c + 4], s[c + 5]);
              mx[3] = ptx::fmax3(mx[3], s[c + 6], s[c + 7]);
            }
          }
          const float bm = fmaxf(ptx::fmax3(mx[0], mx[1], mx[2]), mx[3]);
          float m_new = m_ref;
          if (bm > m_ref && (m_ref == -INFINITY || (bm - m_ref) * c2 > p.rescale_threshold)) m_new = bm;
          alpha = (m_new == m_ref) ? 1.f : ptx::ex2((m_ref - m_new) * c2);
          m_ref = m_new;
          const float ng = m_ref == -INFINITY ? 0.f : -m_ref * c2;
          uint64_t acc[4] = {0, 0, 0, 0};
          exp_range(0, BC, ng, acc);
          lblk = sum_acc(acc);
        }
#pragma unroll
        for (int c0 = 0; c0 < BC; c0 += 32) ptx::tmem_st16(tP + c0 / 2, &pk[c0 / 2]);
        l = l * alpha + lblk;
        if (taken > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O_t of this warp's rows holds the sum over the earlier steps (their
          // products precede S(j) in issue order), referenced to the old maximum.
          const uint32_t tO = tmem + lane_off + static_cast<uint32_t>(2 * BC + t * D);
          const uint64_t ax2 = ptx::f2_pack(alpha, alpha);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            ptx::tmem_ld32(tO + c * 32, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), ax2), x0, x1);
              r[e] = __float_as_uint(x0);
              r[e + 1] = __float_as_uint(x1);
            }
            ptx::tmem_st32(tO + c * 32, r);
          }
        }
        ++taken;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(L::kBarPFull + t));
      }
      if (!ok) break;
      // A unit of one step: the epilogue must have taken the previous unit's
      // 1 / l before it is overwritten (with more steps the MMA thread's
      // O-empty wait orders the two).
      if (taken == 1 && !ptx::mbar_wait_warp(bar(L::kBarOEmpty + t), (units & 1u) ^ 1u, s_abort, tmo)) {
        if (lane == 0) record_error(p.status, kErrTimeout, kSiteSoftFinal);
        ok = false;
        break;
      }
      const bool has = l > 0.f;
      s_invl[t * kBR + row] = has ? 1.f / l : 0.f;
      if (row >= qw.lo && row < qw.hi) {
        float* const dst = KPAD && w.place >= 0 ? p.part_lse + part : p.lse + w.lse_base + t * w.lse_next + (qw.load_row - w.q_start + row);
        *dst = has ? m_ref * p.scale + log2f(l) * 0.69314718055994530942f : -INFINITY;
      }
      ptx::mbar_arrive(bar(L::kBarLReady + t));
      ++units;
    }
  } else {
    ptx::setmaxnreg_dec<RegSplit<VARLEN>::kCorrection>();
    // =============================================================== epilogue
    const int wq = warp & 3;
    const int row = (wq << 5) + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq << 5) << 16;
    const uint32_t stage = base + L::kOffStage + wq * L::kStageWarpBytes;
    uint32_t uc[kQT] = {0, 0};
    bool pending = false;  // a TMA store from the staging area may still be reading it
    bool ok = true;
    // Rows without a visible key: o = 0, LSE = -inf.
    auto zero_rows = [&](const WinUnit& w, int t, int row0, int rows) {
      const size_t rs = static_cast<size_t>(p.H) * D;
      const size_t first = VARLEN ? static_cast<size_t>(row0) : static_cast<size_t>(w.b) * p.Nq + row0;
      for (int e = threadIdx.x - 256; e < rows * (D / 8); e += 128)
        ptx::st_global_v4(p.o + (first + e / (D / 8)) * rs + static_cast<size_t>(w.h + t * w.dh) * D + (e % (D / 8)) * 8, 0u, 0u, 0u, 0u);
      for (int r = threadIdx.x - 256; r < rows; r += 128) p.lse[w.lse_base + t * w.lse_next + (row0 - w.q_start) + r] = -INFINITY;
    };
#pragma unroll 1
    FA_WIN_FOR_EACH_ITEM(it) {
      FA_WIN_UNIT(it)
      if (w.nokeys) {
        for (int t = 0; t <= w.dh; ++t) zero_rows(w, t, w.q_row0, min(p.unit_rows, w.q_end - w.q_row0));
        continue;
      }
#pragma unroll
      for (int t = 0; t < kQT; ++t) {
        const RowWindow qw = w.qwin[t];
        if (w.rows[t] && !w.active[t] && !(KPAD && w.place >= 0)) zero_rows(w, t, qw.load_row + qw.lo, qw.hi - qw.lo);
        if (!w.active[t]) continue;
        if (!ptx::mbar_wait_warp(bar(L::kBarLReady + t), uc[t] & 1u, s_abort, tmo) ||
            !ptx::mbar_wait_warp(bar(L::kBarOFinal + t), uc[t] & 1u, s_abort, tmo)) {
          record_error(p.status, kErrTimeout, kSiteCorrFinal);
          ok = false;
          break;
        }
        ++uc[t];
        ptx::tc_fence_after();
        const float inv_l = s_invl[t * kBR + row];
        const uint32_t tO = tmem + lane_off + static_cast<uint32_t>(2 * BC + t * D);
        const bool warp_full = (wq << 5) >= qw.lo && (wq << 5) + 32 <= qw.hi;
        const bool parted = KPAD && w.place >= 0;
        const bool use_tma = !parted && (!VARLEN || warp_full);  // dense: rows past Nq are clipped by the map
        const bool row_ok = row >= qw.lo && row < qw.hi;
        __nv_bfloat16* const grow =
            row_ok ? p.o + (static_cast<size_t>(qw.load_row + row) * p.H + w.h + t * w.dh) * D : p.o;
        float* const prow =
            parted && row_ok
                ? p.part_o + (static_cast<size_t>(w.place) * (kBR * kQT) + win_unit_row(w, t, qw.load_row + row)) * D
                : nullptr;
        if (use_tma && pending) {
          if (lane == 0) ptx::bulk_wait_group_read_0();
          __syncwarp();
          pending = false;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          ptx::tmem_ld32(tO + c * 32, r);
          ptx::tmem_wait_ld();
          if (parted) {
            if (row_ok) {
#pragma unroll
              for (int q4 = 0; q4 < 8; ++q4)
                ptx::st_global_v4(prow + c * 32 + q4 * 4, __float_as_uint(__uint_as_float(r[4 * q4]) * inv_l),
                                  __float_as_uint(__uint_as_float(r[4 * q4 + 1]) * inv_l),
                                  __float_as_uint(__uint_as_float(r[4 * q4 + 2]) * inv_l),
                                  __float_as_uint(__uint_as_float(r[4 * q4 + 3]) * inv_l));
            }
            continue;
          }
          uint32_t wv[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            wv[e] = ptx::pack_bf16x2(__uint_as_float(r[2 * e]) * inv_l, __uint_as_float(r[2 * e + 1]) * inv_l);
          if (use_tma) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const int c16 = 4 * c + q4;
              const int pnl = c16 / 8, chunk = c16 % 8;
              ptx::st_shared_v4(stage + pnl * 4096 + lane * 128 + ((chunk ^ (lane & 7)) << 4), wv[4 * q4],
                                wv[4 * q4 + 1], wv[4 * q4 + 2], wv[4 * q4 + 3]);
            }
          } else if (row_ok) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              ptx::st_global_v4(grow + c * 32 + q4 * 8, wv[4 * q4], wv[4 * q4 + 1], wv[4 * q4 + 2], wv[4 * q4 + 3]);
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(L::kBarOEmpty + t));
        if (use_tma) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int pnl = 0; pnl < kDPanels; ++pnl) {
              if constexpr (VARLEN)
                ptx::tma_store_3d(&tm_o, stage + pnl * 4096, pnl * kPanel, w.h + t * w.dh, qw.load_row + (wq << 5));
              else
                ptx::tma_store_4d(&tm_o, stage + pnl * 4096, pnl * kPanel, w.h + t * w.dh, qw.load_row + (wq << 5), w.b);
            }
            ptx::bulk_commit_group();
          }
          pending = true;
        }
      }
    }
    if (lane == 0 && pending) ptx::bulk_wait_group_read_0();
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();  // single-lane roles rejoin their warp before the CTA barrier
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// The parts of the unit that ends in CTA blockIdx.x's range and was begun before
// it ("GPU 内核与 FlashAttention" §11.2): o = sum_s w_s O_s / sum_s w_s with w_s =
// e^(LSE_s - max).  One warp per row; bound by reading the parts (twice 256 rows a
// CTA at most).
template <int D, bool VARLEN>
__global__ void __launch_bounds__(256) fa_win_join_kernel(const WinParams p) {
  grid_dependency_wait();
  const int2 cut = p.cut[blockIdx.x];
  if (cut.x < 0) return;
  const WinUnit w = win_decode<128, VARLEN, true>(p, cut.x);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int t = w.dh ? r / kBR : 0, i = w.q_row0 + (w.dh ? r % kBR : r);  // head of the unit, query row
  if (i >= w.q_end) return;
  const int parts = static_cast<int>(blockIdx.x) - cut.y + 1;
  constexpr int kPer = D / 32;
  auto at = [&](int s) -> size_t { return (2 * static_cast<size_t>(cut.y + s) + (s == 0 ? 1 : 0)) * (kBR * kQT) + r; };
  float M = -INFINITY;
  for (int s = lane; s < parts; s += 32) M = fmaxf(M, p.part_lse[at(s)]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
  float acc[kPer], l = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float ls = p.part_lse[at(s)];
    const bool none = ls == -INFINITY;  // a part without keys holds no values
    const float f = none ? 0.f : ptx::ex2((ls - M) * 1.44269504088896340736f);
    const float* src = p.part_o + at(s) * D + lane * kPer;
    l += f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const float x = src[e];
      acc[e] = none ? acc[e] : fmaf(f, x, acc[e]);
    }
  }
  const float il = l > 0.f ? 1.f / l : l;
  const size_t row = VARLEN ? static_cast<size_t>(i) : static_cast<size_t>(w.b) * p.Nq + i;
  __nv_bfloat16* const dst = p.o + (row * p.H + w.h + t) * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = ptx::pack_bf16x2(acc[e] * il, acc[e + 1] * il);
  if (lane == 0) p.lse[w.lse_base + t * w.lse_next + (i - w.q_start)] = l > 0.f ? M + logf(l) : l == 0.f ? -INFINITY : l;
}

}  // namespace fa
