// fa_kv_attn.cu -- attention over the paged e4m3 cache (fa_fwd_kvcache): few query
// rows by the kernel of fa_kv_attn.cuh, long query chunks by dequantising the
// visible pages to bf16 (exact) and running the window kernel on them.
#include "fa_kv_attn.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa.h"
#include "fa_window.h"

namespace fa {
namespace {

// Query rows per key/value head (queries times heads of a group) up to which the
// kernel for few rows runs, a unit of 8 or 16 rows at a time (the codes of later row
// groups come from L2): 5.6 ns a group and 128 keys of a key/value head (64 x 8192
// keys, 8 heads of d 128), where the bf16 copy and 128-row tiles take 54 ns, most of
// them for the copy and for tiles that a few queries leave empty.
constexpr int kFewRows = 128;

struct KvPlan {
  bool few;
  int rows;             // few rows: query rows per unit
  int ctas;             // few rows: CTAs (at most three an SM; fewer when there are fewer steps)
  int cluster;          // few rows: CTAs of a unit in the cluster form, 0: equal ranges
  int k_pad;            // chunk form: key rows per sequence of the bf16 copy
  size_t ws_bytes;
};

// The cluster form's launch.
template <int D, int NT>
cudaLaunchConfig_t cluster_config(cudaLaunchAttribute& a, int cluster, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kKvThreads);
  c.dynamicSmemBytes = KvSmem<D, NT>::kAlloc;
  c.stream = stream;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = cluster;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return c;
}

// Clusters of `c` CTAs that the device holds at once (fewer than its CTAs allow: a
// cluster stays within one group of SMs; 64 clusters of 7 fit by number, but ran in
// two rounds, 18.7 us where clusters of 4 took 10.0).  Asked once for each size.
template <int D, int NT>
int max_clusters(int c) {
  static std::atomic<int> known[64][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][c].load(std::memory_order_relaxed);
  if (n == 0) {
    auto* kern = &fa_kv_attn_kernel<D, NT, true>;
    static std::atomic<unsigned long long> done{0};
    if (set_smem_once(reinterpret_cast<const void*>(kern), KvSmem<D, NT>::kAlloc, done) != cudaSuccess) return 0;
    cudaLaunchAttribute a;
    const cudaLaunchConfig_t config = cluster_config<D, NT>(a, c, c, nullptr);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &config) != cudaSuccess) {
      cudaGetLastError();  // the equal ranges run instead
      n = 0;
    }
    n = n > 0 ? n : -1;
    known[dev][c].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Steps of a CTA up to which the cluster form runs, where its units fit the SMs at once
// (one token, 16 heads on 4 of d 128: 4000 keys, 4 steps, 11.1 us against 11.3 in equal
// ranges; 8000 keys, 8 steps, 14.9 against 13.2).
constexpr int kClusterSteps = 4;

// Depends on the sizes alone.
KvPlan kv_plan(int B, int max_q, int max_k, int H, int Hk, int d, int causal, int window, int sinks, int num_sms) {
  KvPlan z{};
  const long long rows = static_cast<long long>(max_q) * (Hk > 0 ? H / Hk : 1);
  z.few = rows <= kFewRows;
  if (!z.few) {
    z.k_pad = (max_k + kKvTile - 1) / kKvTile * kKvTile;
    z.ws_bytes = 2 * static_cast<size_t>(B) * z.k_pad * Hk * d * 2 + window_parts_bytes(num_sms, d);
    return z;
  }
  long long steps = (static_cast<long long>(max_k) + kKvTile - 1) / kKvTile;
  if (causal && window > 0) {
    const long long win = (static_cast<long long>(window) + max_q + kKvTile - 2) / kKvTile + 1;
    steps = std::min(steps, win + (static_cast<long long>(sinks) + kKvTile - 1) / kKvTile);
  }
  z.rows = rows <= 8 ? 8 : 16;
  const long long resident = (z.rows == 8 || d == 64 ? 3 : kKvCtas<128, 2>) * num_sms;
  const long long units = B * static_cast<long long>(Hk) * ((rows + z.rows - 1) / z.rows);
  long long c = std::max<long long>(1, std::min({8LL, steps, units > 0 ? resident / units : 1}));
  auto fits = [&](int n) -> bool {
    return units <= (z.rows == 8 ? (d == 128 ? max_clusters<128, 1>(n) : max_clusters<64, 1>(n))
                                 : (d == 128 ? max_clusters<128, 2>(n) : max_clusters<64, 2>(n)));
  };
  while (c >= 1 && steps <= kClusterSteps * c && !fits(static_cast<int>(c))) --c;
  if (c >= 1 && steps <= kClusterSteps * c) {
    z.cluster = static_cast<int>(c);
    z.ctas = static_cast<int>(c * units);
    return z;
  }
  z.ctas = static_cast<int>(std::max<long long>(1, std::min(units * std::max<long long>(steps, 1), resident)));
  z.ws_bytes = static_cast<size_t>(z.ctas) * (16 + 2 * z.rows * (static_cast<size_t>(d) + 1) * 4);
  return z;
}

// Codes as a map: rows of d bytes, boxes of one page (at most 128 rows).
int encode_cache(CUtensorMap* m, const void* codes, long long rows, int d, int page) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(page)};
  return host_encode(m, codes, 2, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                     d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D, int NT>
cudaError_t launch_one(const CUtensorMap& tk, const CUtensorMap& tv, const KvAttnParams& p, int ctas, cudaStream_t stream) {
  auto* kern = &fa_kv_attn_kernel<D, NT, true>;
  constexpr int smem = KvSmem<D, NT>::kAlloc;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute a;
  const cudaLaunchConfig_t c = cluster_config<D, NT>(a, p.cluster, ctas, stream);
  return cudaLaunchKernelEx(&c, kern, tk, tv, p);
}

template <int D, int NT>
cudaError_t launch_few(const CUtensorMap& tk, const CUtensorMap& tv, const KvAttnParams& p, int ctas, cudaStream_t stream) {
  if (p.cluster > 0) return launch_one<D, NT>(tk, tv, p, ctas, stream);
  auto* kern = &fa_kv_attn_kernel<D, NT, false>;
  constexpr int smem = KvSmem<D, NT>::kAlloc;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kKvThreads, smem, stream>>>(tk, tv, p);
  const cudaError_t le = cudaGetLastError();
  if (le != cudaSuccess) return le;
  const dim3 grid(ctas, std::min(8 * NT, p.max_q * p.G));
  return launch_dependent(&fa_kv_join_kernel<D, 8 * NT>, grid, 128, 0, stream, p);
}

// ------------------------------------------------------------- long query chunks
// bf16 copy [B, k_pad, Hk, d] of the key tiles that some query sees, zeros behind
// the sequence's end up to the tile's: with power-of-two scales the copy is exact,
// so the products that follow see the values the codes stand for.  One block per
// (64 tokens, sequence, K or V); bound by its bytes (1 read, 2 written a value: 75 MB for
// three sequences of 8192 keys, 4 heads of d 128, 13 us).
struct DequantParams {
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  const int *cu, *lens, *table;
  __nv_bfloat16 *k, *v;
  int B, max_q, max_k, total_q, Hk, width, page, num_pages, k_pad, causal, window, sinks;
  int* status;
};

template <int D>
__global__ void __launch_bounds__(256) fa_kv_dequant_kernel(const DequantParams p) {
  grid_dependents_launch();  // the window kernel may be set up; it waits for this grid's end
  const int b = blockIdx.y;
  const int t0 = blockIdx.x * 64;
  const bool is_k = blockIdx.z == 0;
  const int len = p.lens[b];
  const int row0 = p.cu ? p.cu[b] : b * p.max_q;
  const int n_q = p.cu ? p.cu[b + 1] - row0 : p.max_q;
  if (len < 0 || len > p.max_k || len > static_cast<long long>(p.width) * p.page || n_q < 0 || n_q > p.max_q || row0 < 0 ||
      row0 > p.total_q - n_q) {
    if (threadIdx.x == 0) record_error(p.status, kErrBadSeqlens, 0);
    return;
  }
  if (n_q == 0) return;
  const KvRange r = kv_range(p.causal ? len - n_q : len - 1, len - 1, p.window, p.sinks);
  const int tile = t0 / kKvTile * kKvTile;
  // Whole tiles: the kernel that follows reads them whole.
  if (!kv_needed(r, tile, kKvTile)) return;
  constexpr int kLanes = D / 16;
  const uint8_t* const codes = is_k ? p.k8 : p.v8;
  const float* const scales = is_k ? p.k_scale : p.v_scale;
  __nv_bfloat16* const out = is_k ? p.k : p.v;
  // A thread's tokens and, four heads at a time, its loads are in flight together.
  constexpr int kTok = 256 / kLanes, kPass = 64 / kTok;
  const int ch = threadIdx.x % kLanes;
  int id[kPass];
#pragma unroll
  for (int n = 0; n < kPass; ++n) {
    const int t = t0 + n * kTok + threadIdx.x / kLanes;
    id[n] = t < len ? p.table[static_cast<size_t>(b) * p.width + t / p.page] : -1;
    if (t < len && !kv_page_ok(id[n], p.num_pages)) {
      if (ch == 0) record_error(p.status, kErrBadPage, 0);
      id[n] = -1;
    }
  }
  for (int hk0 = 0; hk0 < p.Hk; hk0 += 4) {
    uint4 raw[kPass][4];
    float s[kPass][4];
#pragma unroll
    for (int n = 0; n < kPass; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const bool in = id[n] >= 0 && hk0 + g < p.Hk;
        const int t = t0 + n * kTok + threadIdx.x / kLanes;
        const size_t ph = in ? static_cast<size_t>(id[n]) * p.Hk + hk0 + g : 0;
        s[n][g] = in ? scales[ph] : 0.f;
        raw[n][g] = in ? *reinterpret_cast<const uint4*>(codes + (ph * p.page + t % p.page) * D + 16 * ch)
                       : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int n = 0; n < kPass; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (hk0 + g >= p.Hk) continue;
        const uint32_t v[4] = {raw[n][g].x, raw[n][g].y, raw[n][g].z, raw[n][g].w};
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t lo, hi;
          e4m3x4_to_f16(v[k], lo, hi);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          w[2 * k] = ptx::pack_bf16x2(a.x * s[n][g], a.y * s[n][g]);
          w[2 * k + 1] = ptx::pack_bf16x2(c.x * s[n][g], c.y * s[n][g]);
        }
        const int t = t0 + n * kTok + threadIdx.x / kLanes;
        __nv_bfloat16* const dst = out + ((static_cast<size_t>(b) * p.k_pad + t) * p.Hk + hk0 + g) * D + 16 * ch;
        ptx::st_global_v4(dst, w[0], w[1], w[2], w[3]);
        ptx::st_global_v4(dst + 8, w[4], w[5], w[6], w[7]);
      }
  }
}

int check_sizes(int B, int total_q, int max_q, int max_k, int H, int Hk, int d, int page, int num_pages, int width,
                int causal, int window, int sinks) {
  if (B < 0 || total_q < 0 || max_q < 0 || max_k < 0 || H < 0 || Hk < 0 || num_pages < 0 || width < 0)
    return FA_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || (window > 0 && !causal)) return FA_ERR_INVALID_ARG;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (H > 65535 || B > 65535) return FA_ERR_INVALID_ARG;
  const long long lim = 0x7fffffffLL;
  if (static_cast<long long>(B) * H * max_q > lim || static_cast<long long>(num_pages) * Hk * page > lim ||
      static_cast<long long>(B) * (max_k + 127LL) > lim || max_k > lim - kKvTile || max_q > lim - 2 * 128)
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

long long fa_kvcache_workspace_bytes(int B, int max_seqlen_q, int max_seqlen_k, int H, int Hk, int d, int causal,
                                     int window, int sinks) {
  int rc = fa::check_sizes(B, 0, max_seqlen_q, max_seqlen_k, H, Hk, d, 16, 0, 0, causal, window, sinks);
  if (rc != FA_OK) return rc;
  fa::HostDevice dev;
  if ((rc = fa::host_device(&dev)) != FA_OK) return rc;
  return static_cast<long long>(
      fa::kv_plan(B, max_seqlen_q, max_seqlen_k, H, Hk, d, causal, window, sinks, dev.num_sms).ws_bytes);
}

int fa_fwd_kvcache(const void* q, const void* k8, const void* v8, const float* k_scale, const float* v_scale,
                   const int* block_table, const int* seq_lens, const int* cu_seqlens_q, void* o, float* lse, int B,
                   int total_q, int max_seqlen_q, int max_seqlen_k, int H, int Hk, int d, int page, int num_pages,
                   int table_width, float scale, int causal, int window, int sinks, void* workspace,
                   long long workspace_bytes, void* stream) {
  int rc = fa::check_sizes(B, total_q, max_seqlen_q, max_seqlen_k, H, Hk, d, page, num_pages, table_width, causal,
                           window, sinks);
  if (rc != FA_OK) return rc;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!cu_seqlens_q && static_cast<long long>(B) * max_seqlen_q != total_q) return FA_ERR_INVALID_ARG;
  if (B == 0 || total_q == 0 || max_seqlen_q == 0 || H == 0) return FA_OK;
  if (!q || !o || !lse || !seq_lens) return FA_ERR_INVALID_ARG;
  if (num_pages > 0 && (!k8 || !v8 || !k_scale || !v_scale)) return FA_ERR_INVALID_ARG;
  if (table_width > 0 && !block_table) return FA_ERR_INVALID_ARG;
  for (const void* ptr : {q, k8, v8, static_cast<const void*>(o), static_cast<const void*>(workspace)})
    if (fa::misaligned(ptr, 16)) return FA_ERR_ALIGN;
  for (const void* ptr : {static_cast<const void*>(k_scale), static_cast<const void*>(v_scale),
                          static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(cu_seqlens_q), static_cast<const void*>(lse)})
    if (fa::misaligned(ptr, 4)) return FA_ERR_ALIGN;
  fa::HostDevice dev;
  if ((rc = fa::host_device(&dev)) != FA_OK) return rc;
  const fa::KvPlan z = fa::kv_plan(B, max_seqlen_q, max_seqlen_k, H, Hk, d, causal, window, sinks, dev.num_sms);
  if (z.ws_bytes > 0 && (!workspace || workspace_bytes < 0 || static_cast<size_t>(workspace_bytes) < z.ws_bytes))
    return FA_ERR_INVALID_ARG;
  // No window is a window over every key.
  const int win = causal && window > 0 ? std::min(window, std::max(max_seqlen_k, 1)) : 0;
  const int snk = win > 0 ? std::min(sinks, max_seqlen_k) : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (z.few) {
    fa::KvAttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.cu = cu_seqlens_q;
    p.lens = seq_lens;
    p.table = block_table;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.B = B;
    p.max_q = max_seqlen_q;
    p.max_k = max_seqlen_k;
    p.total_q = total_q;
    p.H = H;
    p.Hk = Hk;
    p.G = H / Hk;
    p.width = table_width;
    p.page = page;
    p.num_pages = num_pages;
    p.causal = causal != 0;
    p.window = win;
    p.sinks = snk;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    p.cluster = z.cluster;
    p.row_groups = static_cast<int>((static_cast<long long>(max_seqlen_q) * p.G + z.rows - 1) / z.rows);
    p.cut = static_cast<int4*>(workspace);
    p.part_lse = reinterpret_cast<float*>(p.cut + z.ctas);
    p.part_o = p.part_lse + static_cast<size_t>(z.ctas) * 2 * z.rows;
    p.timeout_ns = dev.timeout_ns;
    p.status = dev.status;
    CUtensorMap tk, tv;
    // Without pages nothing is read; the maps need a valid address all the same.
    const long long rows = std::max<long long>(static_cast<long long>(num_pages) * Hk * page, page);
    if ((rc = fa::encode_cache(&tk, num_pages > 0 ? k8 : q, rows, d, page)) != FA_OK) return rc;
    if ((rc = fa::encode_cache(&tv, num_pages > 0 ? v8 : q, rows, d, page)) != FA_OK) return rc;
    if (d == 128)
      e = z.rows == 8 ? fa::launch_few<128, 1>(tk, tv, p, z.ctas, st) : fa::launch_few<128, 2>(tk, tv, p, z.ctas, st);
    else
      e = z.rows == 8 ? fa::launch_few<64, 1>(tk, tv, p, z.ctas, st) : fa::launch_few<64, 2>(tk, tv, p, z.ctas, st);
    return e == cudaSuccess ? FA_OK : fa::host_cuda_fail(e);
  }
  fa::DequantParams dq{};
  dq.k8 = static_cast<const uint8_t*>(k8);
  dq.v8 = static_cast<const uint8_t*>(v8);
  dq.k_scale = k_scale;
  dq.v_scale = v_scale;
  dq.cu = cu_seqlens_q;
  dq.lens = seq_lens;
  dq.table = block_table;
  dq.k = static_cast<__nv_bfloat16*>(workspace);
  dq.v = dq.k + static_cast<size_t>(B) * z.k_pad * Hk * d;
  dq.B = B;
  dq.max_q = max_seqlen_q;
  dq.max_k = max_seqlen_k;
  dq.total_q = total_q;
  dq.Hk = Hk;
  dq.width = table_width;
  dq.page = page;
  dq.num_pages = num_pages;
  dq.k_pad = z.k_pad;
  dq.causal = causal != 0;
  dq.window = win;
  dq.sinks = snk;
  dq.status = dev.status;
  {
    const dim3 grid(std::max(z.k_pad / 64, 1), B, 2);  // without keys it still checks the lengths
    if (d == 128)
      fa::fa_kv_dequant_kernel<128><<<grid, 256, 0, st>>>(dq);
    else
      fa::fa_kv_dequant_kernel<64><<<grid, 256, 0, st>>>(dq);
    if ((e = cudaGetLastError()) != cudaSuccess) return fa::host_cuda_fail(e);
  }
  fa::WinLaunchArgs a;
  std::memset(&a, 0, sizeof(a));
  fa::WinParams& p = a.p;
  p.B = B;
  p.Nq = max_seqlen_q;
  p.Nk = z.k_pad;
  p.H = H;
  p.window = win > 0 ? win : std::max(z.k_pad, 1);
  p.sinks = snk;
  p.full = causal == 0;
  p.total_q = total_q;
  p.cu_q = cu_seqlens_q;
  p.cu_k = seq_lens;
  p.lse = lse;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.scale = scale;
  p.timeout_ns = dev.timeout_ns;
  p.status = dev.status;
  fa::window_parts(p, dq.v + static_cast<size_t>(B) * z.k_pad * Hk * d, dev.num_sms);
  a.num_sms = dev.num_sms;
  a.stream = st;
  return fa::launch_window(a, q, z.k_pad > 0 ? static_cast<const void*>(dq.k) : q,
                           z.k_pad > 0 ? static_cast<const void*>(dq.v) : q, Hk, d, true);
}

}  // extern "C"
