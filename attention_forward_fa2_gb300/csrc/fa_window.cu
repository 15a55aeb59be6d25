// fa_window.cu -- C entries of attention with a sliding window and sinks
// (fa_fwd_window, fa_bwd_window), kernel instantiations and launchers.
#include "fa_window.h"

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa.h"

namespace fa {
namespace {

// Ring depth: two K/V slots of 64 KB fit beside the query tiles for d = 128,
// three of 32 KB for d = 64 (as in the forward without a window).
template <int D>
constexpr int kWinStages = D == 128 ? 2 : 3;
template <int D>
constexpr int kWinBwdStages = D == 128 ? 2 : 4;

template <int D, bool VARLEN, bool KPAD>
cudaError_t launch_win(const WinLaunchArgs& a) {
  auto* kern = &fa_win_kernel<D, kWinStages<D>, VARLEN, KPAD>;
  constexpr int smem = WinSmem<D, kWinStages<D>>::kAlloc;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  const int grid = KPAD && !a.p.whole ? a.num_sms
                   : KPAD || VARLEN   ? a.p.num_units
                                      : std::min(a.p.num_units, a.num_sms);
  if constexpr (KPAD) {
    const cudaError_t le = launch_dependent(kern, dim3(grid), kThreads, smem, a.stream, a.tm_q, a.tm_k, a.tm_v, a.tm_o, a.p);
    if (le != cudaSuccess || a.p.whole) return le;
    const dim3 rows(grid, a.p.pair ? kBR * kQT / 8 : (std::min(a.p.Nq, kBR * kQT) + 7) / 8);
    return launch_dependent(&fa_win_join_kernel<D, VARLEN>, rows, 256, 0, a.stream, a.p);
  }
  kern<<<grid, kThreads, smem, a.stream>>>(a.tm_q, a.tm_k, a.tm_v, a.tm_o, a.p);
  return cudaGetLastError();
}

// KPAD: units an SM from which they are handed out whole (WinItem in fa_win_kernel.cuh).
constexpr long long kWholeUnits = 6;

template <int D>
cudaError_t dispatch_win(const WinLaunchArgs& a, bool varlen, bool kpad) {
  if (kpad) return varlen ? launch_win<D, true, true>(a) : launch_win<D, false, true>(a);
  return varlen ? launch_win<D, true, false>(a) : launch_win<D, false, false>(a);
}

// bf16 rows as a map: packed [rows, heads, d] (rank 3) or dense [B, n, heads, d]
// (rank 4), boxes of `box_rows` rows of one head and 64 columns.
int encode_rows(CUtensorMap* m, const void* ptr, bool packed, int B, int n, int heads, int d, int box_rows) {
  const cuuint64_t row = static_cast<cuuint64_t>(heads) * d * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, row, row * n};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1};
  return host_encode(m, ptr, packed ? 3 : 4, dims, strides, box);
}

template <int D, bool VARLEN, bool SPLIT, int PASSES>
cudaError_t launch_win_bwd(const BwdLaunchArgs& a, const WinBwdParams& p) {
  cudaError_t e = cudaSuccess;
  constexpr int kRows = 256 / (D / 8) * PASSES;
  const long long prep = static_cast<long long>(p.B) * p.H * p.nq_pad;
  const long long prep_blocks = (prep + kRows - 1) / kRows + (VARLEN && p.order ? 1 : 0);
  if (prep_blocks > 0) fa_win_prep_kernel<D, VARLEN, SPLIT, PASSES><<<static_cast<unsigned>(prep_blocks), 256, 0, a.stream>>>(p);
  auto* kern = &fa_win_bwd_kernel<D, kWinBwdStages<D>, VARLEN, SPLIT>;
  constexpr int smem = BwdSmem<D, kWinBwdStages<D>>::kAlloc;
  static std::atomic<unsigned long long> done{0};
  e = set_smem_once(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  // Each kernel is set up while the one before it ends, and waits for its end before it
  // reads what that one wrote.  The key-block kernel clears dK and dV rows that nothing
  // sees without that wait, so without a prep kernel before it it starts in order.
  if (a.grid.x > 0) {
    if (prep_blocks > 0)
      e = launch_dependent(kern, a.grid, kThreads, smem, a.stream, a.tm_q, a.tm_k, a.tm_v, a.tm_do, p);
    else
      kern<<<a.grid, kThreads, smem, a.stream>>>(a.tm_q, a.tm_k, a.tm_v, a.tm_do, p);
    if (e != cudaSuccess) return e;
  }
  const long long sum_rows = static_cast<long long>(p.B) * p.Hk * (p.split > 1 ? p.num_kb : p.num_skb) * kBwdBK;
  const long long sum_blocks = (sum_rows + 7) / 8, blocks = sum_blocks + (prep + kRows - 1) / kRows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (blocks > 0) {
    e = launch_dependent(&fa_win_finish_kernel<D, VARLEN, SPLIT, PASSES>, dim3(static_cast<unsigned>(blocks)), 256, 0,
                         a.stream, p, static_cast<uint32_t>(sum_blocks));
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int D, bool VARLEN>
cudaError_t dispatch_win_bwd(const BwdLaunchArgs& a, const WinBwdParams& p) {
  // The rows of a packed batch are walked up to the longest length: blocks of more rows
  // where three in four are of no sequence (4000 tokens and 40 x 100, 16 heads on 4 of
  // d 128: 439 -> 169 us).
  if (VARLEN && p.split == 1 && static_cast<long long>(p.B) * p.nq_pad > 4 * (p.total_q + 128LL * p.B))
    return launch_win_bwd<D, VARLEN, false, VARLEN ? kBwdBQ / (256 / (D / 8)) : 1>(a, p);
  return p.split > 1 ? launch_win_bwd<D, VARLEN, true, 1>(a, p) : launch_win_bwd<D, VARLEN, false, 1>(a, p);
}

// Checks shared by the forward and the backward entry.
int check_sizes(int B, int Nq, int Nk, int H, int Hk, int d, float scale, int window, int sinks, const int* cu_q,
                const int* cu_k, int total_q, int total_k) {
  if (B < 0 || Nq < 0 || Nk < 0 || H < 0 || Hk < 0) return FA_ERR_INVALID_ARG;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if ((cu_q == nullptr) != (cu_k == nullptr)) return FA_ERR_INVALID_ARG;
  if (cu_q && (total_q < 0 || total_k < 0)) return FA_ERR_INVALID_ARG;
  if (misaligned(cu_q, 4) || misaligned(cu_k, 4)) return FA_ERR_ALIGN;
  if (H > 65535 || B > 65535) return FA_ERR_INVALID_ARG;
  const long long lim = 0x7fffffffLL;
  if (Nq > lim - 2 * kBR || Nk > lim - 2 * kBR) return FA_ERR_INVALID_ARG;  // rounding up to tiles stays in 32 bits
  if (static_cast<long long>(B) * Nq > lim || static_cast<long long>(B) * Nk > lim ||
      static_cast<long long>(B) * H * Nq > lim)
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

struct BwdSizes {
  int nq_pad, num_kb, num_skb, chunk_qb, num_chunks, split;
  long long sink_units, units;
  size_t dq_bytes, part_floats, part2_floats;
  size_t order_bytes;  // of the list of units, behind all else
  size_t bytes() const { return dq_bytes + 4 * (part_floats + part2_floats) + order_bytes; }
};

// Parts of a unit: the fewest steps on the busiest of 152 SMs (this part's number,
// so that the workspace depends on the sizes alone), where a unit's beginning and end
// cost about kUnitSteps, the kernel that sums the parts kSumSteps, and the bytes of
// 64 parts one step (2.9 us; 128 KB written and read a part of d 128).
// Two sequences of 1024, 8 heads on 2 of d 64, no window: 74.9 us whole, 34.5 in parts.
constexpr int kPlanSms = 152, kMaxSplit = 8, kUnitSteps = 1, kSumSteps = 2, kStepParts = 64;
int bwd_split(long long units, long long steps) {
  int best = 1;
  long long least = 0;
  for (int n = 1; n <= kMaxSplit && n <= steps; ++n) {
    const long long rounds = (units * n + kPlanSms - 1) / kPlanSms;
    const long long cost = rounds * ((steps + n - 1) / n + kUnitSteps) + (n > 1 ? kSumSteps + units * n / kStepParts : 0);
    if (n > 1 && cost >= least) continue;
    best = n;
    least = cost;
  }
  return best;
}

// A chunk of a sink block walks as many query blocks as the other units do
// (floor((window + 126) / 128) + 1), at least 4 so that short windows do not pay
// for many small chunks.
BwdSizes bwd_sizes(int B, int Nq, int Nk, int H, int Hk, int d, int window, int sinks) {
  BwdSizes z;
  const int blocks = (Nq + kBwdBQ - 1) / kBwdBQ;
  z.nq_pad = blocks * kBwdBQ;
  z.num_kb = (Nk + kBwdBK - 1) / kBwdBK;
  z.num_skb = (std::min(sinks, Nk) + kBwdBK - 1) / kBwdBK;
  z.chunk_qb = std::max(4, (std::min(window, std::max(Nk, 1)) + 126) / kBwdBQ + 1);
  z.num_chunks = (blocks + z.chunk_qb - 1) / z.chunk_qb;
  z.dq_bytes = static_cast<size_t>(B) * H * z.nq_pad * (static_cast<size_t>(d) + 2) * 4;
  z.sink_units = static_cast<long long>(B) * Hk * z.num_skb * z.num_chunks;
  z.units = z.sink_units + static_cast<long long>(B) * Hk * (z.num_kb - z.num_skb);
  z.split = bwd_split(z.units, static_cast<long long>(Hk > 0 ? H / Hk : 1) * std::min(blocks, z.chunk_qb));
  const size_t rows = static_cast<size_t>(z.split) * B * Hk * kBwdBK * 2 * d;  // of a key block
  z.part_floats = rows * z.num_chunks * z.num_skb;
  z.part2_floats = z.split > 1 ? rows * (z.num_kb - z.num_skb) : 0;
  z.order_bytes = z.units * z.split <= kOrderMax ? 4 * (static_cast<size_t>(z.units) * z.split + 1) : 0;
  return z;
}

}  // namespace

size_t window_parts_bytes(int num_sms, int d) {
  return static_cast<size_t>(num_sms) * (16 + 2 * kBR * kQT * (static_cast<size_t>(d) + 1) * 4);
}

void window_parts(WinParams& p, void* at, int num_sms) {
  p.cut = static_cast<int2*>(at);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(at) + 16 * static_cast<size_t>(num_sms));
  p.part_o = p.part_lse + static_cast<size_t>(num_sms) * 2 * kBR * kQT;
}

int launch_window(WinLaunchArgs& a, const void* q, const void* k, const void* v, int Hk, int d, bool kpad) {
  WinParams& p = a.p;
  const bool varlen = p.cu_q != nullptr;
  const bool kpacked = varlen && !kpad;
  const int nq = varlen ? p.total_q : p.Nq, nk = std::max(kpacked ? p.total_k : p.Nk, 1);
  int e;
  if ((e = encode_rows(&a.tm_q, q, varlen, p.B, nq, p.H, d, kBR)) != FA_OK) return e;
  if ((e = encode_rows(&a.tm_o, p.o, varlen, p.B, nq, p.H, d, 32)) != FA_OK) return e;
  if ((e = encode_rows(&a.tm_k, k, kpacked, p.B, nk, Hk, d, 128)) != FA_OK) return e;
  if ((e = encode_rows(&a.tm_v, v, kpacked, p.B, nk, Hk, d, 128)) != FA_OK) return e;
  p.group = p.H / Hk;
  // One query tile a unit where the SMs take all of them at once (1000 queries, 8 heads
  // of d 64, window 128: 12.2 -> 9.3 us; with more tiles than SMs two a unit take half
  // again as long as one).
  const long long tiles = static_cast<long long>(p.B) * p.H * ((p.Nq + kBR - 1) / kBR);
  p.tiles = !kpad && tiles <= a.num_sms ? 1 : kQT;
  p.pair = p.tiles == kQT && p.group % 2 == 0;
  p.unit_rows = p.pair ? kBR : kBR * p.tiles;
  p.unit_heads = p.pair ? p.H / 2 : p.H;
  p.num_mblocks = (p.Nq + p.unit_rows - 1) / p.unit_rows;
  const long long units = static_cast<long long>(p.B) * p.unit_heads * p.num_mblocks;
  if (units > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  p.num_units = static_cast<int>(units);
  // A window longer than the keys changes nothing and is cut to them, so that
  // the kernel's index arithmetic stays in 32 bits.
  p.window = std::min(p.window, std::max(p.Nk, 1));
  p.sinks = std::min(p.sinks, p.Nk);
  p.whole = kpad && units >= kWholeUnits * a.num_sms;
  p.by_block = !varlen && !kpad && p.window >= p.Nk / 2;
  p.scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
  // A row's first tile may show it a single key (the window's start, few sinks),
  // so its reference maximum is often far below its true one.  Nothing is lost
  // by that: weights are bf16 and sums fp32, whose relative precision does not
  // depend on the reference, and 2^40 is far from overflow; a threshold of 2^8
  // would send most rows' second tile through the slow path.
  p.rescale_threshold = 40.f;
  const cudaError_t ce = d == 128 ? dispatch_win<128>(a, varlen, kpad) : dispatch_win<64>(a, varlen, kpad);
  return ce == cudaSuccess ? FA_OK : host_cuda_fail(ce);
}

}  // namespace fa

extern "C" {

int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Nq, int Nk, int H, int Hk,
                  int d, float scale, int window, int sinks, const int* cu_seqlens_q, const int* cu_seqlens_k,
                  int total_q, int total_k, void* stream) {
  int rc = fa::check_sizes(B, Nq, Nk, H, Hk, d, scale, window, sinks, cu_seqlens_q, cu_seqlens_k, total_q, total_k);
  if (rc != FA_OK) return rc;
  const bool varlen = cu_seqlens_q != nullptr;
  if (B == 0 || Nq == 0 || H == 0 || (varlen && total_q == 0)) return FA_OK;
  if (!q || !o || !lse || ((!varlen || total_k > 0) && (!k || !v))) return FA_ERR_INVALID_ARG;
  if (!varlen && Nk == 0) return FA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, v, static_cast<const void*>(o)})
    if (fa::misaligned(ptr, 16)) return FA_ERR_ALIGN;
  if (fa::misaligned(lse, 4)) return FA_ERR_ALIGN;
  fa::HostDevice dev;
  if ((rc = fa::host_device(&dev)) != FA_OK) return rc;
  fa::WinLaunchArgs a;
  std::memset(&a, 0, sizeof(a));
  fa::WinParams& p = a.p;
  p.B = B;
  p.Nq = Nq;
  p.Nk = Nk;
  p.H = H;
  p.window = window;
  p.sinks = sinks;
  p.total_q = total_q;
  p.total_k = total_k;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.lse = lse;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.scale = scale;
  p.timeout_ns = dev.timeout_ns;
  p.status = dev.status;
  a.num_sms = dev.num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  // No keys at all (packed): the maps need an address, nothing is read from it.
  const bool none = varlen && total_k == 0;
  return fa::launch_window(a, q, none ? q : k, none ? q : v, Hk, d, false);
}

long long fa_bwd_window_workspace_bytes(int B, int Nq, int Nk, int H, int Hk, int d, int window, int sinks) {
  const int rc = fa::check_sizes(B, Nq, Nk, H, Hk, d, 1.f, window, sinks, nullptr, nullptr, 0, 0);
  if (rc != FA_OK) return rc;
  const fa::BwdSizes z = fa::bwd_sizes(B, Nq, Nk, H, Hk, d, window, sinks);
  return static_cast<long long>(z.bytes());
}

int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                  void* dq, void* dk, void* dv, int B, int Nq, int Nk, int H, int Hk, int d, float scale, int window,
                  int sinks, const int* cu_seqlens_q, const int* cu_seqlens_k, int total_q, int total_k,
                  void* workspace, long long workspace_bytes, void* stream) {
  int rc = fa::check_sizes(B, Nq, Nk, H, Hk, d, scale, window, sinks, cu_seqlens_q, cu_seqlens_k, total_q, total_k);
  if (rc != FA_OK) return rc;
  const bool varlen = cu_seqlens_q != nullptr;
  const int rows_q = varlen ? total_q : Nq, rows_k = varlen ? total_k : Nk;
  if (B == 0 || H == 0 || (rows_q == 0 && rows_k == 0)) return FA_OK;
  if (!varlen && Nk == 0) return FA_ERR_INVALID_ARG;  // queries without keys, as in the forward
  if (rows_k > 0 && (!k || !v || !dk || !dv)) return FA_ERR_INVALID_ARG;
  if (rows_q > 0 && (!q || !o || !dout || !lse || !dq)) return FA_ERR_INVALID_ARG;
  const fa::BwdSizes z = fa::bwd_sizes(B, Nq, Nk, H, Hk, d, window, sinks);
  if (static_cast<long long>(B) * H * z.nq_pad > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  if (z.bytes() > 0 &&
      (!workspace || workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < z.bytes()))
    return FA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k, v, o, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv), static_cast<const void*>(workspace)})
    if (fa::misaligned(ptr, 16)) return FA_ERR_ALIGN;
  if (fa::misaligned(lse, 4)) return FA_ERR_ALIGN;
  fa::HostDevice dev;
  if ((rc = fa::host_device(&dev)) != FA_OK) return rc;
  fa::BwdLaunchArgs a;
  std::memset(&a, 0, sizeof(a));
  fa::WinBwdParams p;
  std::memset(static_cast<void*>(&p), 0, sizeof(p));
  p.B = B;
  p.Nq = Nq;
  p.Nk = Nk;
  p.H = H;
  p.Hk = Hk;
  p.group = H / Hk;
  p.causal = 1;
  p.nq_pad = z.nq_pad;
  p.num_kb = z.num_kb;
  p.num_skb = z.num_skb;
  p.chunk_qb = z.chunk_qb;
  p.num_chunks = z.num_chunks;
  if (z.units * z.split > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  p.split = z.split;
  p.num_sink_units = static_cast<int>(z.sink_units * z.split);
  p.num_units = static_cast<int>(z.units * z.split);
  p.window = std::min(window, std::max(Nk, 1));
  p.sinks = std::min(sinks, Nk);
  p.total_q = total_q;
  p.total_k = total_k;
  p.o = static_cast<const __nv_bfloat16*>(o);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.lse = lse;
  const size_t rows_pad = static_cast<size_t>(B) * H * z.nq_pad;
  p.dq_acc = static_cast<float*>(workspace);
  p.lse2 = p.dq_acc + rows_pad * d;
  p.delta = p.lse2 + rows_pad;
  p.part = p.delta + rows_pad;
  p.part2 = p.part + z.part_floats;
  p.order = varlen && z.order_bytes > 0 ? reinterpret_cast<int*>(p.part2 + z.part2_floats) : nullptr;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.scale = scale;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.timeout_ns = dev.timeout_ns;
  p.status = dev.status;
  // Maps need a valid address and extent even where nothing is read.
  const void* qp = rows_q > 0 ? q : k;
  const void* dop = rows_q > 0 ? dout : k;
  const void* kp = rows_k > 0 ? k : q;
  const void* vp = rows_k > 0 ? v : q;
  const int hq = rows_q > 0 ? H : Hk, hk = rows_k > 0 ? Hk : H;
  const int nq = rows_q > 0 ? rows_q : 1, nk = rows_k > 0 ? rows_k : 1;
  if ((rc = fa::encode_rows(&a.tm_q, qp, varlen, B, nq, hq, d, fa::kBwdBQ)) != FA_OK) return rc;
  if ((rc = fa::encode_rows(&a.tm_do, dop, varlen, B, nq, hq, d, fa::kBwdBQ)) != FA_OK) return rc;
  if ((rc = fa::encode_rows(&a.tm_k, kp, varlen, B, nk, hk, d, fa::kBwdBK)) != FA_OK) return rc;
  if ((rc = fa::encode_rows(&a.tm_v, vp, varlen, B, nk, hk, d, fa::kBwdBK)) != FA_OK) return rc;
  a.grid = dim3(static_cast<unsigned>(std::min(p.num_units, dev.num_sms)));
  a.stream = static_cast<cudaStream_t>(stream);
  cudaError_t ce;
  if (d == 128)
    ce = varlen ? fa::dispatch_win_bwd<128, true>(a, p) : fa::dispatch_win_bwd<128, false>(a, p);
  else
    ce = varlen ? fa::dispatch_win_bwd<64, true>(a, p) : fa::dispatch_win_bwd<64, false>(a, p);
  return ce == cudaSuccess ? FA_OK : fa::host_cuda_fail(ce);
}

}  // extern "C"
