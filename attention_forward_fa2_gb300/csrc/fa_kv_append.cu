// fa_kv_append.cu -- new keys and values into a paged e4m3 cache, keys (and
// queries) rotated to their positions on the way (fa_kvcache_append).
//
// For pair c < rot / 2 of a token at position p, with (a, b) the c-th pair of
// elements (halves: c and c + rot / 2; neighbours: 2c and 2c + 1):
//     y_a = x_a cos(p, c) - x_b sin(p, c),   y_b = x_b cos(p, c) + x_a sin(p, c)
// in fp32 (products and sums rounded separately); queries are rounded once to
// bf16, keys once to e4m3 under the scale of their page and head
//     s = 2^e, e the smallest with max |y| <= 448 * 2^e over the page's new tokens,
// or the page's present scale where that is larger and the page was begun
// before.  When a begun page's scale grows, its older codes are rounded to the
// new scale: a shift of the exponent, exact but for values that become subnormal.
// Infinities saturate and NaN stays NaN; neither counts for the maximum.
//
// Bound by its bytes (3 d bytes per key/value row, 4 d per query row) for long
// prompts, by latency for single tokens.  Four prompts of 4096 tokens, 32 heads on 8 of
// d 128: 78 us, 4840 GB/s, 60 % of the issue slots (the rotation and the two passes over
// the registers); four single tokens 2.4 us.  A work item is one page of one head of
// K or V: a 16-lane (d = 128) or 8-lane (d = 64) group holds a row, 16 bytes of
// bf16 a lane, all rows of the item stay in registers between the maximum and
// the rounding, so the input is read once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fa.h"
#include "fa_kvcache.h"
#include "fa_launch.h"

namespace fa {
namespace {

struct AppendParams {
  const __nv_bfloat16 *k, *v, *q;            // token rows, `*_stride` elements apart; heads d apart
  long long k_stride, v_stride, q_stride;
  __nv_bfloat16* q_out;                      // [total, H, d]
  const int *cu, *lens, *table;              // cu null: max_new tokens per sequence
  const float *cos, *sin;                    // [max_pos, rot / 2]
  uint8_t *k8, *v8;
  float *k_scale, *v_scale;
  int B, total, max_new, H, Hk, width, page, num_pages, max_pos, rot;
  int touch;                                 // pages that one sequence's new tokens can lie in
  int kv_blocks, q_blocks;                   // blocks per sequence
  int* status;
};

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// cos / sin of the 8 elements of chunk c of a row at position pos.
struct Turn {
  float c[8], s[8];
};
template <bool INTER>
__device__ __forceinline__ void load_turn(const AppendParams& p, int pos, int c, Turn& t) {
  const int half = p.rot >> 1;
  if constexpr (INTER) {
    const float4 cc = *reinterpret_cast<const float4*>(p.cos + static_cast<size_t>(pos) * half + 4 * c);
    const float4 ss = *reinterpret_cast<const float4*>(p.sin + static_cast<size_t>(pos) * half + 4 * c);
    const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t.c[2 * e] = t.c[2 * e + 1] = cv[e];
      t.s[2 * e] = t.s[2 * e + 1] = sv[e];
    }
  } else {
    const int at = 8 * c < half ? 8 * c : 8 * c - half;
    const float4* cp = reinterpret_cast<const float4*>(p.cos + static_cast<size_t>(pos) * half + at);
    const float4* sp = reinterpret_cast<const float4*>(p.sin + static_cast<size_t>(pos) * half + at);
    const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
    t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
    t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
    t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
    t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  }
}

// Rotates chunk c (8 elements) of a row; the lanes of a row's group call together.
template <bool INTER>
__device__ __forceinline__ void rotate8(const AppendParams& p, int c, const uint4& raw, const Turn& t, float (&x)[8]) {
  if constexpr (INTER) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float a = x[e], b = x[e + 1];
      x[e] = __fsub_rn(__fmul_rn(a, t.c[e]), __fmul_rn(b, t.s[e]));
      x[e + 1] = __fadd_rn(__fmul_rn(b, t.c[e]), __fmul_rn(a, t.s[e]));
    }
  } else {
    // The other element of each pair lies rot / 16 chunks away, in another lane.
    const int hc = p.rot >> 4;
    const bool first = c < hc;
    const int lane = threadIdx.x & 31;
    const int src = c >= 2 * hc ? lane : first ? lane + hc : lane - hc;
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, raw.x, src);
    o.y = __shfl_sync(0xffffffffu, raw.y, src);
    o.z = __shfl_sync(0xffffffffu, raw.z, src);
    o.w = __shfl_sync(0xffffffffu, raw.w, src);
    float y[8];
    unpack8(o, y);
    if (c >= 2 * hc) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xc = __fmul_rn(x[e], t.c[e]), ys = __fmul_rn(y[e], t.s[e]);
      x[e] = first ? __fsub_rn(xc, ys) : __fadd_rn(xc, ys);
    }
  }
}

// Bits of the largest finite magnitude of 8 values and `m`.
__device__ __forceinline__ uint32_t amax8(const float (&x)[8], uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
    if (b < 0x7f800000u) m = max(m, b);
  }
  return m;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  return ptx::pack_e4m3x2(a, b) | (ptx::pack_e4m3x2(c, d) << 16);
}

// Two e4m3 codes to floats.
__device__ __forceinline__ void unpack_e4m3x2(uint32_t codes, float& lo, float& hi) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(codes & 0xffffu));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// THREADS = 32: an item is a warp's (few new tokens); 256: a block's.
// ITERS rows per group of lanes; THREADS / (D / 8) * ITERS rows hold a page's.
// HEADS heads of a page are one item: their loads are in flight together, and the
// angles of a row are loaded once for all of them.
template <int D, int THREADS, int ITERS, int HEADS, bool INTER>
__global__ void __launch_bounds__(256, THREADS > 32 ? 3 : ITERS > 1 ? 2 : 4) fa_kv_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;            // lanes of a row
  constexpr int kRows = THREADS / kLanes;  // rows per iteration of an item
  __shared__ uint32_t s_max[8][HEADS];
  const int b = blockIdx.x / (p.kv_blocks + p.q_blocks);
  const int r = blockIdx.x % (p.kv_blocks + p.q_blocks);
  const int c = threadIdx.x % kLanes;
  const int old_len = p.lens[b];
  const int row0 = p.cu ? p.cu[b] : b * p.max_new;
  const int n = p.cu ? p.cu[b + 1] - row0 : p.max_new;
  if (!kv_append_fits(old_len, row0, n, p.max_new, p.total, p.width, p.page, p.rot > 0 ? p.max_pos : -1)) {
    if (r == 0 && threadIdx.x == 0) record_error(p.status, kErrBadSeqlens, 0);
    return;
  }
  if (r >= p.kv_blocks) {
    // ------------------------- queries: QHEADS heads of a token per group of lanes
    constexpr int kQHeads = THREADS > 32 ? 8 : 4;
    constexpr int kGroups = 256 / kLanes;
    const int sets = (p.H + kQHeads - 1) / kQHeads;
    const long long item = static_cast<long long>(r - p.kv_blocks) * kGroups + threadIdx.x / kLanes;
    const bool in = item < static_cast<long long>(n) * sets;
    const int i = in ? static_cast<int>(item / sets) : 0;
    const int h0 = in ? kQHeads * static_cast<int>(item % sets) : 0;
    const __nv_bfloat16* src = p.q + static_cast<size_t>(row0 + i) * p.q_stride + static_cast<size_t>(h0) * D + 8 * c;
    uint4 raw[kQHeads];
#pragma unroll
    for (int e = 0; e < kQHeads; ++e)
      raw[e] = in && h0 + e < p.H ? *reinterpret_cast<const uint4*>(src + e * D) : make_uint4(0, 0, 0, 0);
    Turn t;
    const bool turns = in && 8 * c < p.rot;
    if (turns) load_turn<INTER>(p, old_len + i, c, t);
    __nv_bfloat16* dst = p.q_out + (static_cast<size_t>(row0 + i) * p.H + h0) * D + 8 * c;
#pragma unroll
    for (int e = 0; e < kQHeads; ++e) {
      float x[8];
      unpack8(raw[e], x);
      if (!INTER || turns) rotate8<INTER>(p, c, raw[e], t, x);
      if (in && h0 + e < p.H) {
        if (turns)
          ptx::st_global_v4(dst + e * D, ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                            ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
        else
          ptx::st_global_v4(dst + e * D, raw[e].x, raw[e].y, raw[e].z, raw[e].w);
      }
    }
    return;
  }
  // ------------------------------------------------------------ a page of one head of K or V
  const int item = r * (256 / THREADS) + (THREADS == 32 ? threadIdx.x >> 5 : 0);
  const int head_groups = (p.Hk + HEADS - 1) / HEADS;
  if (item >= p.touch * head_groups * 2) return;  // whole warps (THREADS = 32) or the whole block
  const bool is_k = (item & 1) == 0;
  const int h0 = (item >> 1) % head_groups * HEADS;
  const int pg = old_len / p.page + (item >> 1) / head_groups;  // page of the sequence
  // Slots [s0, s1) of the page take new tokens.
  const int s0 = max(old_len - pg * p.page, 0);
  const int s1 = min(old_len + n - pg * p.page, p.page);
  if (s1 <= s0) return;
  const int id = p.table[static_cast<size_t>(b) * p.width + pg];
  if (!kv_page_ok(id, p.num_pages)) {
    if (threadIdx.x % THREADS == 0) record_error(p.status, kErrBadPage, 0);
    return;
  }
  const size_t ph0 = static_cast<size_t>(id) * p.Hk + h0;
  float* const scales = (is_k ? p.k_scale : p.v_scale) + ph0;
  uint8_t* const codes = (is_k ? p.k8 : p.v8) + ph0 * p.page * D;
  const int tid = threadIdx.x % THREADS;
  const __nv_bfloat16* const x0 = is_k ? p.k : p.v;
  const long long stride = is_k ? p.k_stride : p.v_stride;
  const bool turn_item = is_k && p.rot > 0;
  float old_scale[HEADS];
#pragma unroll
  for (int g = 0; g < HEADS; ++g) old_scale[g] = s0 > 0 && h0 + g < p.Hk ? scales[g] : 0.f;
  // The rows stay in registers as they were read (rotated keys would take twice the
  // registers); keys are rotated once for the maximum and once for the codes.
  uint4 raw[HEADS][ITERS];
  uint32_t amax[HEADS];
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int slot = s0 + it * kRows + tid / kLanes;
    const int i = slot < s1 ? pg * p.page + slot - old_len : 0;  // index among the new tokens
    const __nv_bfloat16* const src = x0 + static_cast<size_t>(row0 + i) * stride + h0 * D + 8 * c;
#pragma unroll
    for (int g = 0; g < HEADS; ++g)
      raw[g][it] = slot < s1 && h0 + g < p.Hk ? *reinterpret_cast<const uint4*>(src + g * D) : make_uint4(0, 0, 0, 0);
  }
  // Calls f(g, it, values) for every row, in fp32 and rotated.
  auto each = [&](auto&& f) {
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
      const int slot = s0 + it * kRows + tid / kLanes;
      const bool turns = turn_item && slot < s1 && 8 * c < p.rot;
      Turn t;
      if (turns) load_turn<INTER>(p, pg * p.page + slot, c, t);
#pragma unroll
      for (int g = 0; g < HEADS; ++g) {
        float y[8];
        unpack8(raw[g][it], y);
        if (turn_item) {
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = y[e];
          if (!INTER || turns) rotate8<INTER>(p, c, raw[g][it], t, z);
          if (turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = z[e];
          }
        }
        f(g, slot, y);
      }
    }
  };
#pragma unroll
  for (int g = 0; g < HEADS; ++g) amax[g] = 0u;
  each([&](int g, int, const float(&y)[8]) { amax[g] = amax8(y, amax[g]); });
#pragma unroll
  for (int g = 0; g < HEADS; ++g) amax[g] = __reduce_max_sync(0xffffffffu, amax[g]);
  if constexpr (THREADS > 32) {
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int g = 0; g < HEADS; ++g) s_max[threadIdx.x >> 5][g] = amax[g];
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < HEADS; ++g)
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) amax[g] = max(amax[g], s_max[w][g]);
  }
  float inv[HEADS];
#pragma unroll
  for (int g = 0; g < HEADS; ++g) {
    const float need = __uint_as_float(static_cast<uint32_t>(kv_scale_exp(amax[g]) + 127) << 23);
    const float scale = fmaxf(old_scale[g], need);
    inv[g] = 1.f / scale;  // exact
    if (h0 + g >= p.Hk) continue;
    if (s0 > 0 && scale > old_scale[g]) {
      const float ratio = old_scale[g] * inv[g];
      for (int e = tid; e < s0 * (D / 16); e += THREADS) {
        uint4* const ptr = reinterpret_cast<uint4*>(codes + static_cast<size_t>(g) * p.page * D) + e;
        const uint4 w = *ptr;
        uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a, d0, d1, d2;
          unpack_e4m3x2(v[k], a, d0);
          unpack_e4m3x2(v[k] >> 16, d1, d2);
          v[k] = pack4(a * ratio, d0 * ratio, d1 * ratio, d2 * ratio);
        }
        *ptr = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    if (tid == 0) scales[g] = scale;
  }
  each([&](int g, int slot, const float(&y)[8]) {
    if (slot < s1 && h0 + g < p.Hk)
      *reinterpret_cast<uint2*>(codes + (static_cast<size_t>(g) * p.page + slot) * D + 8 * c) =
          make_uint2(pack4(y[0] * inv[g], y[1] * inv[g], y[2] * inv[g], y[3] * inv[g]),
                     pack4(y[4] * inv[g], y[5] * inv[g], y[6] * inv[g], y[7] * inv[g]));
  });
}

template <int D, int THREADS, int ITERS, int HEADS>
void launch(AppendParams& p, bool inter, cudaStream_t stream) {
  const int items = p.touch * ((p.Hk + HEADS - 1) / HEADS) * 2;
  p.kv_blocks = THREADS == 32 ? (items + 7) / 8 : items;
  constexpr int kQHeads = THREADS > 32 ? 8 : 4;
  const long long groups = static_cast<long long>(p.max_new) * ((p.H + kQHeads - 1) / kQHeads);
  p.q_blocks = p.q ? static_cast<int>((groups + 256 / (D / 8) - 1) / (256 / (D / 8))) : 0;
  const unsigned grid = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.kv_blocks + p.q_blocks);
  if (inter)
    fa_kv_append_kernel<D, THREADS, ITERS, HEADS, true><<<grid, 256, 0, stream>>>(p);
  else
    fa_kv_append_kernel<D, THREADS, ITERS, HEADS, false><<<grid, 256, 0, stream>>>(p);
}

// Few new tokens (up to 2 or 8 rows of d = 128, 4 or 16 of d = 64): an item per warp and
// head, so that a batch of single tokens spreads over the SMs.  More: a block per
// page and up to four heads, whose loads cover one another's latency.
template <int D>
void dispatch(AppendParams& p, bool inter, cudaStream_t stream) {
  constexpr int kRows = 256 / (D / 8);
  const int rows = std::min(p.page, p.max_new);
  if (rows <= kRows / 8)
    launch<D, 32, 1, 1>(p, inter, stream);
  else if (rows <= 4 * (kRows / 8))
    launch<D, 32, 4, 1>(p, inter, stream);
  else if (rows <= kRows)
    launch<D, 256, 1, 4>(p, inter, stream);
  else if (rows <= 2 * kRows)
    launch<D, 256, 2, 4>(p, inter, stream);
  else if (rows <= 4 * kRows)
    launch<D, 256, 4, 2>(p, inter, stream);
  else
    launch<D, 256, 8, 1>(p, inter, stream);  // page 128 at d = 128
}

}  // namespace
}  // namespace fa

extern "C" int fa_kvcache_append(const void* k, const void* v, long long k_stride, long long v_stride, const void* q,
                                 long long q_stride, void* q_out, const float* cos, const float* sin, int max_pos,
                                 int rot, int interleaved, void* k8, void* v8, float* k_scale, float* v_scale,
                                 const int* block_table, const int* cache_lens, const int* cu_seqlens, int B, int total,
                                 int max_new, int H, int Hk, int d, int page, int num_pages, int table_width,
                                 void* stream) {
  if (B < 0 || total < 0 || max_new < 0 || H < 0 || Hk < 0 || num_pages < 0 || table_width < 0 || max_pos < 0)
    return FA_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return FA_ERR_INVALID_ARG;
  if (rot < 0 || rot > d || rot % 16 != 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (!cu_seqlens && static_cast<long long>(B) * max_new != total) return FA_ERR_INVALID_ARG;
  if (B == 0 || total == 0 || max_new == 0 || (Hk == 0 && (H == 0 || !q))) return FA_OK;
  if ((q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (Hk > 0 && (!k || !v || !k8 || !v8 || !k_scale || !v_scale || !block_table)) return FA_ERR_INVALID_ARG;
  if (!cache_lens || (rot > 0 && (!cos || !sin))) return FA_ERR_INVALID_ARG;
  if (H > 65535 || Hk > 65535 || B > 65535) return FA_ERR_INVALID_ARG;
  const long long kv_row = static_cast<long long>(Hk) * d, q_row = static_cast<long long>(H) * d;
  if (total > 1 && Hk > 0 && (k_stride < kv_row || v_stride < kv_row)) return FA_ERR_INVALID_ARG;
  if (total > 1 && q && q_stride < q_row) return FA_ERR_INVALID_ARG;
  if (q && H > 0 && q_out == q && total > 1 && q_stride != q_row) return FA_ERR_INVALID_ARG;
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || (q && q_stride % 8 != 0)) return FA_ERR_ALIGN;
  for (const void* ptr : {k, v, q, static_cast<const void*>(q_out), static_cast<const void*>(k8),
                          static_cast<const void*>(v8), static_cast<const void*>(cos), static_cast<const void*>(sin)})
    if (fa::misaligned(ptr, 16)) return FA_ERR_ALIGN;
  for (const void* ptr : {static_cast<const void*>(k_scale), static_cast<const void*>(v_scale),
                          static_cast<const void*>(block_table), static_cast<const void*>(cache_lens),
                          static_cast<const void*>(cu_seqlens)})
    if (fa::misaligned(ptr, 4)) return FA_ERR_ALIGN;
  const long long touch = (static_cast<long long>(page) - 1 + max_new + page - 1) / page;
  const long long blocks = B * (touch * Hk * 2 + (static_cast<long long>(max_new) * ((H + 3) / 4) + 15) / 16);
  if (blocks > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  fa::HostDevice dev;
  const int rc = fa::host_device(&dev);
  if (rc != FA_OK) return rc;
  fa::AppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q = H > 0 ? static_cast<const __nv_bfloat16*>(q) : nullptr;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_stride = q_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.cu = cu_seqlens;
  p.lens = cache_lens;
  p.table = block_table;
  p.cos = cos;
  p.sin = sin;
  p.k8 = static_cast<uint8_t*>(k8);
  p.v8 = static_cast<uint8_t*>(v8);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.B = B;
  p.total = total;
  p.max_new = max_new;
  p.H = H;
  p.Hk = Hk;
  p.width = table_width;
  p.page = page;
  p.num_pages = num_pages;
  p.max_pos = max_pos;
  p.rot = rot;
  p.touch = static_cast<int>(touch);
  p.status = dev.status;
  if (d == 128)
    fa::dispatch<128>(p, interleaved != 0, static_cast<cudaStream_t>(stream));
  else
    fa::dispatch<64>(p, interleaved != 0, static_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : fa::host_cuda_fail(e);
}
