// fa_kvcache.h -- the paged e4m3 key/value cache: its index rules, shared by the
// append and the attention kernels, and the launch interface between the two
// translation units.
//
// Layout: codes [num_pages, Hk, page, d] (a page of one head is contiguous), one
// fp32 scale per (page, head) of K and of V, a power of two: a code c stands for
// the value c * scale.  A power of two costs nothing in relative precision (e4m3
// is a floating-point format; only its subnormals start up to one step sooner)
// and makes every change of a page's scale, and every dequantised bf16 value,
// exact.  Sequence b's token t lies in page table[b][t / page], slot t % page.
#pragma once
#include <cstdint>

#ifndef FA_HD
#define FA_HD __host__ __device__ __forceinline__
#endif

namespace fa {

constexpr int kErrBadPage = -9;
constexpr int kKvTile = 128;         // tokens per step of the attention kernels
constexpr int kKvMinExp = -64;       // smallest scale 2^-64 (a page of zeros)

FA_HD bool kv_page_ok(int id, int num_pages) { return id >= 0 && id < num_pages; }

// n new tokens (rows row0 .. of the packed input of `total` rows) behind old_len
// cached ones: within the input, the table's `width` pages and, when rotating,
// the tables' max_pos positions (max_pos < 0: no rotation).
FA_HD bool kv_append_fits(long long old_len, long long row0, long long n, long long max_new, long long total,
                          long long width, long long page, long long max_pos) {
  return old_len >= 0 && row0 >= 0 && n >= 0 && n <= max_new && row0 + n <= total && old_len + n <= width * page &&
         (max_pos < 0 || old_len + n <= max_pos);
}

// Exponent e of the page scale for the largest finite magnitude, given as the
// bits of a non-negative float: the smallest e >= kKvMinExp with amax <= 448 * 2^e
// (448 = 1.75 * 2^8).
FA_HD int kv_scale_exp(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kKvMinExp ? kKvMinExp : e;
}

// Keys that a group of query rows at positions p_min .. p_max sees: [0, sinks) and
// [lo, p_max] (window <= 0: all of [0, p_max]).  The steps of the attention
// kernels: step j < ns is key tile j, step j >= ns key tile j + gap.
struct KvRange {
  int end;     // keys [0, end) are the sequence's up to p_max
  int lo;      // first key of the windows
  int sinks;
  int ns, gap, steps;
};
FA_HD KvRange kv_range(int p_min, int p_max, int window, int sinks) {
  KvRange r;
  r.end = p_max + 1;
  r.lo = window > 0 && p_min >= window ? p_min - window + 1 : 0;
  r.sinks = sinks;
  r.ns = r.gap = r.steps = 0;
  if (r.end <= 0) return r;
  const int first = r.lo / kKvTile, last = p_max / kKvTile;
  const int sink_tiles = (sinks + kKvTile - 1) / kKvTile;
  r.ns = sink_tiles < first ? sink_tiles : first;
  r.gap = first - r.ns;
  r.steps = r.ns + last - first + 1;
  return r;
}
// Whether some row of the group sees a key of [a, a + n).
FA_HD bool kv_needed(const KvRange& r, int a, int n) { return a < r.end && (a + n > r.lo || a < r.sinks); }

}  // namespace fa
