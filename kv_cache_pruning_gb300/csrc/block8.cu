// kvp_compact_block8, kvp_append_block8, kvp_append_block8_devpos and
// kvp_read_block8: writing and reading a paged cache held in 8 bits with one
// scale per page (16 tokens of one (b, h)) for K and one for V.
//
// The bulk write of a short prompt is one launch (below); any other runs three
// passes (after zeroing the counts, unless they are few), each launched early
// behind the one before it. The count pass counts the present entries of every
// 128-entry segment and (b, h) and leaves a bit for each score. The list pass, one
// warp per segment, writes the remapping list, the expire values and the page
// table, and names each page's owner. The page pass gives one warp a page: it
// gathers the page's 16 K and V rows through the list (all row loads of a lane in
// flight before the first is used), takes the two largest magnitudes, and writes
// codes and scales, so every row is read once and every code written once. Pages
// are dealt out by their ids over a persistent grid, which keeps the warps even
// whatever the counts are.
//
// The page pass is bound by memory (a row's 4 D bytes in, 2 D out) with the
// conversions close behind. Measured on a GB300, 16 x 8192 x 8 heads of 128,
// 26 % kept, E4M3 / 65,521 x 64 heads, half kept, int8 (whole calls): 65 / 440 us
// with the list read page by page, 55 / 337 with owners and positions read ahead,
// 54 / 329 with cached instead of streaming loads, 51 / 274 with magnitudes on
// packed pairs and int8 rounded by the multiply-add, 48 / 271 with the passes
// launched early, 46 / 266 with the list pass in 32-bit arithmetic, 45 / 266 with
// the count pass's bits for the list pass (scores only). Not kept: K and V in
// separate warps (55 / 343), a third CTA per SM (52 / 306), pages in position order
// over all heads (no faster reads, a dearer list), listing and quantising in one
// pass (61 / 364: its warps idle while they list), and counting by clusters of CTAs,
// which needs no zeroed counts (47 / 266; 3 to 10 us slower at 131,072 x 8 and
// 70,000 x 64 positions).
#include "block8.cuh"
#include "compact_prep.cuh"

namespace kvp {
namespace {

// Workspace: the preparation passes' words, then the number of pages in use,
// then each page's owner: its (b, h), and its index in that (b, h) with the
// number of its rows in the low 5 bits (an index is below 2^27).
size_t prep_bytes(int64_t BH, int NS) { return (compact_ws_bytes(BH, NS) + 15) & ~static_cast<size_t>(15); }
// Then, for the scored mask, a bit for each position: its score reaches the threshold.
size_t owner_bytes(int n_pages_cap) {
  return (static_cast<size_t>(n_pages_cap) * sizeof(uint2) + 15) & ~static_cast<size_t>(15);
}
size_t block8_ws_bytes(int64_t BH, int NS, int n_pages_cap) {
  return prep_bytes(BH, NS) + 16 + owner_bytes(n_pages_cap) + static_cast<size_t>(BH) * NS * sizeof(uint4);
}

// ------------------------------------------------------------------ count pass
// Zeroes the counts. The launches after it start early, but read nothing before their pdl_wait: what lies in an SM's
// first-level cache may be older than the call's inputs until then.
__global__ void __launch_bounds__(1024) zero_counts_kernel(int BH, int32_t* count) {
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < BH; i += 1024) count[i] = 0;
}

// A CTA's entries of a (b, h): to its place among the sums that the list pass's CTAs all add up (the CTA's blockIdx.y of
// [.., BH]), or, where those would be too many, to the (b, h)'s count, which a launch of its own has zeroed. Measured on a
// GB300 (us a write, on the device in brackets; heads of 128, 0.4 kept; sums / zeroed counts): 1 x 1,500 positions of 8 heads
// 16.2 (7.4) / 19.6 (7.9), 4 x 4,096 of 8 14.5 (12.2) / 17.9 (12.3), 8 x 2,048 of 16 25.2 (24.4) / 27.5 (24.7); more (b, h)s:
// 16 x 4,096 of 8 35.8 (34.9) / 37.8 (34.6), 64 x 1,100 of 5 31.4 (30.6) / 32.6 (28.9); more sums of each: 1 x 8,192 of 8
// 16.1 (9.9) / 19.7 (9.6), 1 x 131,072 of 8 85 (84) / 65 (61).
constexpr int kMostSums = 512;     // in all
constexpr int kMostSumsEach = 8;   // of a (b, h)
KVP_DEV void add_count(int32_t* part, int32_t* count, int BH, int bh, int kept) {
  if (part != nullptr) part[static_cast<int64_t>(blockIdx.y) * BH + bh] = kept;
  else if (kept) atomicAdd(&count[bh], kept);
}

// Present entries of each 128-entry segment, and of each (b, h) in kWarpsPerCta of them. A warp takes a segment of one (b, h):
// flags lie along its positions. Of scores it leaves a bit each (the score reaches the threshold) for the list pass.
constexpr int kWords = kSeg / 32;
template <bool kScores>
__global__ void __launch_bounds__(kWarpsPerCta * 32) count_segments_kernel(MaskedSrc src, int now, int NS, uint4* high,
                                                                           int32_t* seg_cnt, int32_t* part,
                                                                           int32_t* count) {
  __shared__ int cta_kept[kWarpsPerCta];
  pdl_launch_dependents();
  pdl_wait();
  const int bh = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sg = blockIdx.y * kWarpsPerCta + warp;
  const auto sv = src.view(bh);
  const int lo = sg * kSeg, hi = min(lo + kSeg, sv.length());
  int kept = 0;
  uint32_t word[kWords];
#pragma unroll
  for (int u = 0; u < kWords; ++u) {
    const int t = lo + u * 32 + lane;
    int64_t row;
    if constexpr (kScores) {
      const int32_t e = sg < NS && t < hi ? sv.expire_row(t, row) : now;
      kept += sv.keep(e, now);
      word[u] = __ballot_sync(0xffffffffu, e == kNever);
    } else {
      if (sg < NS && t < hi) kept += sv.keep(sv.expire_row(t, row), now);
    }
  }
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (lane == 0) {
    cta_kept[warp] = kept;
    if (sg < NS) {
      const int64_t at = static_cast<int64_t>(bh) * NS + sg;
      seg_cnt[at] = kept;
      if constexpr (kScores) high[at] = make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWarpsPerCta; ++w) t += cta_kept[w];
    add_count(part, count, gridDim.x, bh, t);
  }
}

// The same of scores, which lie along the heads of one position, when there are many: a warp takes 32 positions of up to
// 32 heads, a head a lane, so that whole lines are read. Measured on a GB300 (us a write on the device, heads of 128, 0.4
// kept, segments / heads side by side): 4 x 20,000 positions of 12 heads 56.1 / 58.8, of 16 73.4 / 73.3, of 24 105.6 /
// 104.1; 64 x 1,200 of 16 82.9 / 81.7; 70,000 of 64 242 / 230; 512 x 64 of 32 190 / 179; 16 x 8,192 of 8 61.1 / 64.9.
constexpr int kManyHeads = 16;
__global__ void __launch_bounds__(kWarpsPerCta * kWords * 32) count_scores_kernel(MaskedSrc src, int now, int NS,
                                                                                 int BH, uint32_t* high, int32_t* seg_cnt,
                                                                                 int32_t* part, int32_t* count) {
  __shared__ int kept_s[kWarpsPerCta * kWords][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % kWords;
  const int chunks = (src.H + 31) / 32, b = blockIdx.x / chunks, h = (blockIdx.x - b * chunks) * 32 + lane;
  const int bh = b * src.H + h, sg = blockIdx.y * kWarpsPerCta + warp / kWords, t0 = sg * kSeg + w * 32;
  const bool live = h < src.H && sg < NS;
  int kept = 0;
  if (live) {
    const float* sc = src.scores + (static_cast<int64_t>(b) * src.n + t0) * src.H + h;
    const float th = src.tau[bh];
    const int n = min(src.n - t0, 32);
    float x[32];
#pragma unroll
    for (int u = 0; u < 32; ++u) x[u] = u < n ? sc[static_cast<int64_t>(u) * src.H] : 0.f;
    uint32_t word = 0;
#pragma unroll
    for (int u = 0; u < 32; ++u) {
      const int32_t e = expire_kvzap(x[u], th, t0 + u, src.window);
      word |= (e == kNever ? 1u : 0u) << u;
      kept += u < n && now < e;
    }
    high[(static_cast<int64_t>(bh) * NS + sg) * kWords + w] = word;
  }
  kept_s[warp][lane] = kept;
  __syncthreads();
  if (w == 0) {  // the segment's words
#pragma unroll
    for (int i = 1; i < kWords; ++i) kept += kept_s[warp + i][lane];
    if (live) seg_cnt[static_cast<int64_t>(bh) * NS + sg] = kept;
    kept_s[warp][lane] = kept;
  }
  __syncthreads();
  if (warp == 0 && h < src.H) {
#pragma unroll
    for (int i = 1; i < kWarpsPerCta; ++i) kept += kept_s[i * kWords][lane];
    add_count(part, count, BH, bh, kept);
  }
}

// ------------------------------------------------------------------ list pass
template <bool kFused, bool kScores>
__global__ void __launch_bounds__(kWarpsPerCta * 32) list_kernel(
    MaskedSrc src, int now, int NS, int table_share, int reserve, int max_pages, int n_pages_cap, int BH, CompactWs ws,
    const int32_t* part, int32_t* count, int32_t* status, int32_t* expire_pool, int32_t* page_table, int32_t* remap,
    int32_t* n_used, uint2* owner, const uint4* high) {
  pdl_launch_dependents();
  pdl_wait();
  const int bh = blockIdx.x;  // pairs vary fastest: CTAs resident together read the same positions of all heads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sg = blockIdx.y * kWarpsPerCta + warp;
  const bool live = sg < NS;
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;

  // loads that do not depend on one another, all issued first
  const auto sv = src.view(bh);
  const int n = sv.length();
  const int lo = sg * kSeg, hi = min(lo + kSeg, n);
  int32_t exps[kWords];
  if constexpr (kScores) {
    const uint4 x = live ? high[static_cast<int64_t>(bh) * NS + sg] : make_uint4(0, 0, 0, 0);
    const uint32_t word[kWords] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < kWords; ++u) exps[u] = (word[u] >> lane) & 1u ? kNever : lo + u * 32 + lane + src.window;
  } else {
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const int t = lo + u * 32 + lane;
      int64_t row;
      exps[u] = live && t < hi ? sv.expire_row(t, row) : 0;
    }
  }
  int slot0 = 0;
  if (live)
    for (int c0 = 0; c0 < sg; c0 += 32)
      slot0 += c0 + lane < sg ? ws.seg_cnt[static_cast<int64_t>(bh) * NS + c0 + lane] : 0;
  int base, cnt;
  if constexpr (kFused) {
    // (page sums stay below 2^31: checked on the host)
    __shared__ int3 red_s[kWarpsPerCta];
    __shared__ int cnt_s;
    int before = 0, total = 0, most = 0;
    for (int i = threadIdx.x; i < BH; i += kWarpsPerCta * 32) {
      int c = 0;
      if (part != nullptr) {
#pragma unroll 8
        for (int y = 0; y < static_cast<int>(gridDim.y); ++y) c += part[y * BH + i];
        if (i == bh && blockIdx.y == 0) count[bh] = c;
      } else {
        c = count[i];
      }
      if (i == bh) cnt_s = c;
      const int pg = (c + reserve + kPage - 1) / kPage;
      before += i < bh ? pg : 0;
      total += pg;
      most = max(most, pg);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    total = __reduce_add_sync(0xffffffffu, total);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) red_s[warp] = make_int3(before, total, most);
    __syncthreads();
    before = total = most = 0;
#pragma unroll
    for (int w = 0; w < kWarpsPerCta; ++w) {
      before += red_s[w].x;
      total += red_s[w].y;
      most = max(most, red_s[w].z);
    }
    const bool ok = most <= max_pages && total <= n_pages_cap;
    if (first_cta && threadIdx.x == 0) {
      *n_used = ok ? total : 0;
      if (!ok) record_error(status, KVP_ERR_CAPACITY);
    }
    if (!ok) return;
    base = before;
    cnt = cnt_s;
  } else {
    const bool ok = ws.ok[0] != 0;
    if (first_cta && threadIdx.x == 0)
      *n_used = ok ? ws.base[BH - 1] + (count[BH - 1] + reserve + kPage - 1) / kPage : 0;
    if (!ok) return;
    base = ws.base[bh];
    cnt = count[bh];
  }
  if (!live) return;
  slot0 = __reduce_add_sync(0xffffffffu, slot0);
  const int pages = (cnt + reserve + kPage - 1) / kPage;
  int32_t* remap_bh = remap + static_cast<int64_t>(bh) * max_pages * kPage;
  // this segment's share of the page-table row, the owners and the remap tail: table_share pages and their slots. A table
  // wider than the prompt is cleared to its end all the same. Measured on a GB300 (us on the device, heads of 128, half
  // kept; tables of the prompt's pages / of 8,192): 1 x 100 positions of 8 heads 4.8 / 14.6 (short_kernel), 4 x 1,100 of 8
  // 8.5 / 12.7, 64 x 128 of 8 11.8 / 63.7 (a warp clears 512 KB; all of it is 268 MB, 40 us at the copy rate), 16 x 8,192
  // of 8 59.9 / 69.6 (67 MB, 10 us).
  const int p_lo = static_cast<int>(min(static_cast<int64_t>(sg) * table_share, static_cast<int64_t>(max_pages)));
  const int p_hi = p_lo + min(table_share, max_pages - p_lo);
  for (int p = p_lo + lane; p < p_hi; p += 32) {
    page_table[static_cast<int64_t>(bh) * max_pages + p] = p < pages ? base + p : -1;
    if (p < pages) owner[base + p] = make_uint2(bh, static_cast<uint32_t>(p) << 5 | min(max(cnt - p * kPage, 0), kPage));
  }
  for (int64_t j = max(p_lo * kPage, cnt) + lane; j < p_hi * kPage; j += 32) remap_bh[j] = -1;

  int nk = 0;
#pragma unroll
  for (int u = 0; u < kWords; ++u) {
    const int t = lo + u * 32 + lane;
    const int32_t e = exps[u];
    const bool keep = t < hi && sv.keep(e, now);
    const unsigned bal = __ballot_sync(0xffffffffu, keep);
    if (keep) {
      const int j = slot0 + nk + __popc(bal & ((1u << lane) - 1u));
      expire_pool[static_cast<int64_t>(base + (j >> 4)) * kPage + (j & 15)] = e;
      remap_bh[j] = t;
    }
    nk += __popc(bal);
  }
}

// ------------------------------------------------------------------ page pass
constexpr int kPageWarps = 8;  // warps per CTA of the page and read passes
constexpr int kPageCtas = 2;   // CTAs per SM of the page pass: 16 warps, each with a page's rows (8 KB at 128) in flight

// The largest magnitude among a warp's words (NI uint4 a lane), as bf16 bits; kFinite: among the finite ones.
template <int NI, bool kFinite>
KVP_DEV uint32_t largest(const uint4 (&w)[NI]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) a = __vmaxu2(a, kFinite ? finite_abs2(x[c]) : x[c] & 0x7FFF7FFFu);
  }
  return __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
}

// A page's K and V rows in a warp's registers, 16 bytes of a row a lane.
template <int D>
struct PageRows {
  static constexpr int LPR = D / 8;      // lanes a row takes
  static constexpr int RPI = 32 / LPR;   // rows a warp instruction takes
  static constexpr int NI = kPage / RPI;
  uint4 k[NI], v[NI];
  // rows r < n at base + position * st, lane r holding row r's position; the others zero
  KVP_DEV void load(const uint16_t* kb, const uint16_t* vb, int64_t st, int32_t position, int n, int lane) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + lane / LPR;
      const int64_t at = __shfl_sync(0xffffffffu, position, r) * st + lane % LPR * 8;
      k[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (r < n) {
        k[i] = *reinterpret_cast<const uint4*>(kb + at);
        v[i] = *reinterpret_cast<const uint4*>(vb + at);
      }
    }
  }
  // codes and scales to page pg, and expire 0 to its rows from n on
  template <int FMT>
  KVP_DEV void store(int64_t pg, int n, uint8_t* kq_pool, uint8_t* vq_pool, float2* scale_pool, int32_t* expire_pool,
                     int lane) const {
    // the largest magnitudes, as bf16 bits; only a page that holds infinities or NaNs looks at them one by one
    uint32_t ka = largest<NI, false>(k), va = largest<NI, false>(v);
    const bool odd = ka >= 0x7F80u || va >= 0x7F80u;
    if (odd) {
      ka = largest<NI, true>(k);
      va = largest<NI, true>(v);
    }
    const uint32_t ks = scale_bits_for<FMT>(ka), vs = scale_bits_for<FMT>(va);
    const float ki = inverse_of_scale(ks), vi = inverse_of_scale(vs);
    const int64_t row0 = pg * kPage;
    uint8_t* kd = kq_pool + (row0 + lane / LPR) * D + lane % LPR * 8;
    uint8_t* vd = vq_pool + (row0 + lane / LPR) * D + lane % LPR * 8;
    if (!odd) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        *reinterpret_cast<uint2*>(kd + i * RPI * D) = encode8_finite<FMT>(k[i], ki);
        *reinterpret_cast<uint2*>(vd + i * RPI * D) = encode8_finite<FMT>(v[i], vi);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        *reinterpret_cast<uint2*>(kd + i * RPI * D) = encode8<FMT>(k[i], ki);
        *reinterpret_cast<uint2*>(vd + i * RPI * D) = encode8<FMT>(v[i], vi);
      }
    }
    if (lane == 0) scale_pool[pg] = make_float2(__uint_as_float(ks), __uint_as_float(vs));
    if (lane >= n && lane < kPage) expire_pool[row0 + lane] = 0;
  }
};

template <int D, int FMT>
__global__ void __launch_bounds__(kPageWarps * 32, kPageCtas) page_kernel(
    const uint16_t* k, const uint16_t* v, int64_t sb, int64_t st, int64_t sh, int H, const int32_t* n_used,
    const uint2* owner, int max_pages, const int32_t* remap, uint8_t* kq_pool, uint8_t* vq_pool, float2* scale_pool,
    int32_t* expire_pool) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int total = *n_used, step = gridDim.x * kPageWarps;
  // a page's owner is read two pages ahead and its rows' positions one page ahead, so that only the rows are waited for
  const int first = blockIdx.x * kPageWarps + (threadIdx.x >> 5);
  auto owner_of = [&](int64_t pg) { return pg < total ? owner[pg] : make_uint2(0, 0); };
  auto position_of = [&](uint2 ow) {  // lane r: the position of row r
    return lane < static_cast<int>(ow.y & 31u)
               ? remap[(static_cast<int64_t>(ow.x) * max_pages + (ow.y >> 5)) * kPage + lane]
               : 0;
  };
  uint2 ow = owner_of(first), ow_next = owner_of(static_cast<int64_t>(first) + step);
  int32_t mine = position_of(ow);
  for (int64_t pg = first; pg < total; pg += step) {
    const int b = static_cast<int>(ow.x) / H, h = static_cast<int>(ow.x) - b * H;
    const int n = static_cast<int>(ow.y & 31u);
    const int64_t off = b * sb + h * sh;
    PageRows<D> rows;
    rows.load(k + off, v + off, st, mine, n, lane);
    ow = ow_next;
    mine = position_of(ow);
    ow_next = owner_of(pg + 2 * static_cast<int64_t>(step));
    rows.template store<FMT>(pg, n, kq_pool, vq_pool, scale_pool, expire_pool, lane);
  }
}

// ------------------------------------------------------------------ short prompts
// The whole write in one launch, a CTA for each (b, h): it counts every (b, h)'s present entries itself (which is
// why all their positions together are few), lists its own and quantises its pages. Such calls are bound by the host's
// launches: in us a call (on the device alone), one launch / four, measured on a GB300 with heads of 128, half kept:
// 2 x 317 positions 12.0 (6.2) / 19.1 (7.1), 8 x 512 11.7 (7.5) / 19.1 (8.0), 32 x 256 10.4 (6.5) / 17.8 (8.0), 8 x 1000
// 11.8 (11.2) / 19.3 (8.2), 128 x 128 10.8 (10.3) / 17.7 (8.7), 64 x 250 13.2 (13.2) / 17.8 (9.2); above kShortRounds
// rounds of counting it loses: 512 x 30 63 / 18.
constexpr int kShortWarps = 16;
constexpr int kShortPositions = 1024;   // of a (b, h): its pages are one CTA's work
constexpr int kShortRounds = 8;         // of counting, 8 loads a lane each

// Present entries among a lane's positions lane, lane + 32, .. below n: their scores (or flags) loaded eight at a time.
template <class Load, class Expire>
KVP_DEV int present_among(int n, int lane, int now, Load load, Expire expire) {
  int kept = 0;
  for (int t0 = lane; t0 < n; t0 += 256) {
    decltype(load(0)) x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = t0 + 32 * u < n ? load(t0 + 32 * u) : decltype(load(0)){};
#pragma unroll
    for (int u = 0; u < 8; ++u) kept += t0 + 32 * u < n && now < expire(x[u], t0 + 32 * u);
  }
  return kept;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kShortWarps * 32, 1) short_kernel(MaskedSrc src, int now, int reserve, int max_pages,
                                                                    int n_pages_cap, int BH, uint8_t* kq_pool,
                                                                    uint8_t* vq_pool, float2* scale_pool,
                                                                    int32_t* expire_pool, int32_t* page_table,
                                                                    int32_t* remap, int32_t* count, int32_t* status) {
  constexpr int kThreads = kShortWarps * 32, kChunks = kShortPositions / 32;
  __shared__ int32_t count_s[kFusedBH];
  __shared__ int32_t list_s[kShortPositions];
  __shared__ int32_t chunk_s[kChunks];
  __shared__ int3 red_s[kShortWarps];
  pdl_wait();
  const int bh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = src.n;
  // ---- every (b, h)'s count, a warp each
  for (int i = warp; i < BH; i += kShortWarps) {
    const auto sv = src.view(i);
    int kept = src.mode == KVP_MASK_KVZAP
                   ? present_among(n, lane, now, [&](int t) { return sv.sc[static_cast<int64_t>(t) * sv.H]; },
                                   [&](float x, int t) { return expire_kvzap(x, sv.th, t, sv.window); })
                   : present_among(n, lane, now, [&](int t) { return sv.fl[t]; },
                                   [&](int x, int t) { return expire_dms(x, t, sv.delay, sv.window); });
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 0) count_s[i] = kept;
  }
  __syncthreads();
  // ---- this (b, h)'s first page and the budget (page sums stay below 2^31: checked on the host)
  int before = 0, total = 0, most = 0;
  for (int i = tid; i < BH; i += kThreads) {
    const int pg = (count_s[i] + reserve + kPage - 1) / kPage;
    before += i < bh ? pg : 0;
    total += pg;
    most = max(most, pg);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) red_s[warp] = make_int3(before, total, most);
  // ---- its present entries, by chunks of 32 positions: first how many, then where
  const auto sv = src.view(bh);
  constexpr int kMine = kChunks / kShortWarps;
  int32_t e[kMine];
  unsigned bal[kMine];
#pragma unroll
  for (int c = 0; c < kMine; ++c) {
    const int t = (warp * kMine + c) * 32 + lane;
    int64_t row;
    e[c] = t < n ? sv.expire_row(t, row) : 0;
    bal[c] = __ballot_sync(0xffffffffu, t < n && sv.keep(e[c], now));
    if (lane == 0) chunk_s[warp * kMine + c] = __popc(bal[c]);
  }
  __syncthreads();
  before = total = most = 0;
#pragma unroll
  for (int w = 0; w < kShortWarps; ++w) {
    before += red_s[w].x;
    total += red_s[w].y;
    most = max(most, red_s[w].z);
  }
  const int cnt = count_s[bh];
  if (tid == 0) count[bh] = cnt;
  if (most > max_pages || total > n_pages_cap) {
    if (bh == 0 && tid == 0) record_error(status, KVP_ERR_CAPACITY);
    return;
  }
  const int base = before, pages = (cnt + reserve + kPage - 1) / kPage;
  int32_t* remap_bh = remap + static_cast<int64_t>(bh) * max_pages * kPage;
#pragma unroll
  for (int c = 0; c < kMine; ++c) {
    const int chunk = warp * kMine + c;
    const int slot0 = __reduce_add_sync(0xffffffffu, lane < chunk ? chunk_s[lane] : 0);
    if ((bal[c] >> lane) & 1u) {
      const int j = slot0 + __popc(bal[c] & ((1u << lane) - 1u));
      list_s[j] = chunk * 32 + lane;
      remap_bh[j] = chunk * 32 + lane;
      expire_pool[static_cast<int64_t>(base + (j >> 4)) * kPage + (j & 15)] = e[c];
    }
  }
  for (int p = tid; p < max_pages; p += kThreads)
    page_table[static_cast<int64_t>(bh) * max_pages + p] = p < pages ? base + p : -1;
  for (int64_t j = cnt + tid; j < static_cast<int64_t>(max_pages) * kPage; j += kThreads) remap_bh[j] = -1;
  __syncthreads();
  // ---- its pages, a warp each
  const int b = bh / src.H, h = bh - b * src.H;
  const int64_t off = b * src.sb + h * src.sh;
  for (int p = warp; p < pages; p += kShortWarps) {
    const int m = min(max(cnt - p * kPage, 0), kPage);
    PageRows<D> rows;
    rows.load(src.k + off, src.v + off, src.st, lane < m ? list_s[p * kPage + lane] : 0, m, lane);
    rows.template store<FMT>(base + p, m, kq_pool, vq_pool, scale_pool, expire_pool, lane);
  }
}

// ------------------------------------------------------------------ append
constexpr int kAppendWarps = 4;

// One row (x, EPL bf16 values a lane, element 0 in the low half of x.x) into
// row r of a page whose scale is `old` (0 when r is 0): returns the page's scale.
template <int D, int FMT>
KVP_DEV uint32_t append_row(uint2 x, uint8_t* page, int r, uint32_t old, int lane) {
  constexpr int EPL = D / 32;
  uint32_t a = finite_abs2(x.x);
  if constexpr (EPL == 4) a = __vmaxu2(a, finite_abs2(x.y));
  a = __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
  const uint32_t mine = scale_bits_for<FMT>(a);
  const uint32_t now = max(old, mine);  // positive floats order like their bits
  if (now > old) {  // the rows before this one take the larger scale (those of scale 0, infinities among them, become 0)
    const float ratio = __fdiv_rn(__uint_as_float(old), __uint_as_float(now));
    for (int i = lane; i < r * D / 16; i += 32) {
      uint4 w = reinterpret_cast<uint4*>(page)[i];
      w.x = rescale4<FMT>(w.x, ratio);
      w.y = rescale4<FMT>(w.y, ratio);
      w.z = rescale4<FMT>(w.z, ratio);
      w.w = rescale4<FMT>(w.w, ratio);
      reinterpret_cast<uint4*>(page)[i] = w;
    }
  }
  const float inv = inverse_of_scale(now);
  uint8_t* dst = page + r * D + lane * EPL;
  const uint32_t c0 = encode2<FMT>(__fmul_rn(bf16_lo(x.x), inv), __fmul_rn(bf16_hi(x.x), inv));
  if constexpr (EPL == 4) {
    const uint32_t c1 = encode2<FMT>(__fmul_rn(bf16_lo(x.y), inv), __fmul_rn(bf16_hi(x.y), inv));
    *reinterpret_cast<uint32_t*>(dst) = c0 | (c1 << 16);
  } else {
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(c0);
  }
  return now;
}

template <int EPL>
KVP_DEV uint2 load_row_part(const uint16_t* row, int lane) {
  if constexpr (EPL == 4) return reinterpret_cast<const uint2*>(row)[lane];
  return make_uint2(reinterpret_cast<const uint32_t*>(row)[lane], 0u);
}

// One warp per (b, h).
template <int D, int FMT>
__global__ void __launch_bounds__(kAppendWarps * 32) append_block8_kernel(
    int mode, int BH, int H, int pos_arg, const int32_t* pos_dev, const uint16_t* k_new,
    const uint16_t* v_new, int64_t k_sb, int64_t k_sh, int64_t v_sb, int64_t v_sh,
    const float* score, const float* tau, const int32_t* flag, int window,
    int delay, uint8_t* kq_pool, uint8_t* vq_pool, float2* scale_pool,
    int32_t* expire_pool, int n_pages_cap, const int32_t* page_table, int max_pages,
    int32_t* remap, int32_t* count, int32_t* status) {
  constexpr int EPL = D / 32;
  pdl_wait();
  const int bh = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (bh >= BH) return;
  const int b = bh / H, h = bh - b * H;
  const int pos = pos_dev != nullptr ? *pos_dev : pos_arg;
  const int j = count[bh];
  const uint2 kx = load_row_part<EPL>(k_new + b * k_sb + h * k_sh, lane);
  const uint2 vx = load_row_part<EPL>(v_new + b * v_sb + h * v_sh, lane);
  if (pos < 0 || static_cast<int64_t>(pos) + window + delay >= kNever) {
    if (lane == 0) record_error(status, KVP_ERR_INVALID);
    return;
  }
  const int32_t e = (mode == KVP_MASK_KVZAP) ? expire_kvzap(score[bh], tau[bh], pos, window)
                                             : expire_dms(flag[bh], pos, delay, window);
  if (j < 0) {
    if (lane == 0) record_error(status, KVP_ERR_BOUNDS);
    return;
  }
  const int p = j >> 4, r = j & 15;
  const int page = (p < max_pages) ? page_table[static_cast<int64_t>(bh) * max_pages + p] : -1;
  if (page < 0) {
    if (lane == 0) record_error(status, KVP_ERR_CAPACITY);
    return;
  }
  if (page >= n_pages_cap) {
    if (lane == 0) record_error(status, KVP_ERR_BOUNDS);
    return;
  }
  const int64_t row0 = static_cast<int64_t>(page) * kPage;
  // a page's first row starts its scale anew, whatever the page held before
  const float2 old = r > 0 ? scale_pool[page] : make_float2(0.f, 0.f);
  const uint32_t ks = append_row<D, FMT>(kx, kq_pool + row0 * D, r, __float_as_uint(old.x), lane);
  const uint32_t vs = append_row<D, FMT>(vx, vq_pool + row0 * D, r, __float_as_uint(old.y), lane);
  if (lane == 0) {
    scale_pool[page] = make_float2(__uint_as_float(ks), __uint_as_float(vs));
    expire_pool[row0 + r] = e;
    remap[static_cast<int64_t>(bh) * max_pages * kPage + j] = pos;
    count[bh] = j + 1;
  }
}

// ------------------------------------------------------------------ read
template <int FMT>
KVP_DEV uint32_t value2(uint32_t two, float scale) {
  const float2 x = decode2<FMT>(two);
  const __nv_bfloat162 y = __floats2bfloat162_rn(__fmul_rn(x.x, scale), __fmul_rn(x.y, scale));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// One warp per page of a (b, h): 8 codes a lane, LPR lanes a row, so that a warp's stores are whole lines (with 16 codes
// and two 16-byte stores a lane the first-level cache was 82 % busy with half-used sectors: 69 us at 16 x 4096 x 8 heads).
template <int D, int FMT>
__global__ void __launch_bounds__(kPageWarps * 32) read_block8_kernel(
    int H, int64_t n_items, int pages_each, const uint8_t* kq_pool, const uint8_t* vq_pool,
    const float2* scale_pool, int n_pages_cap, const int32_t* page_table, int max_pages,
    const int32_t* count, int first, int n_slots, uint16_t* k_out,
    uint16_t* v_out, int64_t sb, int64_t st, int64_t sh, int32_t* status) {
  constexpr int LPR = D / 8;
  constexpr int RPI = 32 / LPR;
  constexpr int NI = kPage / RPI;
  pdl_wait();
  const int lane = threadIdx.x & 31, piece = lane % LPR, sub = lane / LPR;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kPageWarps + (threadIdx.x >> 5);
  if (item >= n_items) return;
  const int bh = static_cast<int>(item / pages_each);
  const int p = first / kPage + static_cast<int>(item % pages_each);
  const int b = bh / H, h = bh - b * H;
  const int64_t cap = static_cast<int64_t>(max_pages) * kPage;
  const int64_t cnt = min(max(static_cast<int64_t>(count[bh]), int64_t{0}), cap);
  const int64_t slot0 = static_cast<int64_t>(p) * kPage;
  int n = static_cast<int>(min(max(cnt - slot0, int64_t{0}), int64_t{kPage}));  // rows the cache holds here
  int page = 0;
  if (n > 0) {
    page = page_table[static_cast<int64_t>(bh) * max_pages + p];
    if (page < 0 || page >= n_pages_cap) {
      if (lane == 0) record_error(status, KVP_ERR_BOUNDS);
      n = 0;
    }
  }
  const float2 s = n > 0 ? scale_pool[page] : make_float2(0.f, 0.f);
  uint2 kw[NI], vw[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = i * RPI + sub;
    const int64_t at = (static_cast<int64_t>(page) * kPage + r) * D + piece * 8;
    kw[i] = vw[i] = make_uint2(0, 0);
    if (r < n) {
      kw[i] = *reinterpret_cast<const uint2*>(kq_pool + at);
      vw[i] = *reinterpret_cast<const uint2*>(vq_pool + at);
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t slot = slot0 + i * RPI + sub - first;
    if (slot < 0 || slot >= n_slots) continue;
    const int64_t at = b * sb + slot * st + h * sh + piece * 8;
    auto put = [&](uint16_t* dst, uint2 c, float f) {
      *reinterpret_cast<uint4*>(dst + at) =
          make_uint4(value2<FMT>(c.x, f), value2<FMT>(c.x >> 16, f), value2<FMT>(c.y, f), value2<FMT>(c.y >> 16, f));
    };
    put(k_out, kw[i], s.x);
    put(v_out, vw[i], s.y);
  }
}

// The buffers that every call on this cache takes.
kvp_status check_block8(int fmt, int batch, int n_kv_heads, int head_dim, const void* kq_pool, const void* vq_pool,
                        const void* scale_pool, int n_pages_cap, const void* page_table, int max_pages,
                        const void* count, const void* status) {
  if (fmt != KVP_BLOCK8_E4M3 && fmt != KVP_BLOCK8_INT8) return KVP_ERR_INVALID;
  if (batch <= 0 || n_kv_heads <= 0 || n_pages_cap < 0 || max_pages < 0) return KVP_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128) return KVP_ERR_UNSUPPORTED;
  if (kq_pool == nullptr || vq_pool == nullptr || scale_pool == nullptr || page_table == nullptr || count == nullptr ||
      status == nullptr)
    return KVP_ERR_INVALID;
  if (!aligned16(kq_pool) || !aligned16(vq_pool) || !aligned16(scale_pool)) return KVP_ERR_ALIGN;
  if (static_cast<int64_t>(max_pages) * kPage > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * n_kv_heads > kMaxCompactBH) return KVP_ERR_UNSUPPORTED;
  return KVP_OK;
}

template <int D, int FMT>
kvp_status launch_compact(const MaskedSrc& src, int BH, int NS, int now, int reserve, uint8_t* kq_pool,
                          uint8_t* vq_pool, float* scale_pool, int32_t* expire_pool, int n_pages_cap,
                          int32_t* page_table, int max_pages, int32_t* remap, int32_t* count, void* workspace,
                          int32_t* status, cudaStream_t st) {
  if (BH <= kFusedBH && src.n <= kShortPositions &&
      (BH + kShortWarps - 1) / kShortWarps * ((src.n + 255) / 256) <= kShortRounds) {
    return launch_pdl(short_kernel<D, FMT>, dim3(BH), dim3(kShortWarps * 32), 0, st, src, now, reserve, max_pages,
                      n_pages_cap, BH, kq_pool, vq_pool, reinterpret_cast<float2*>(scale_pool), expire_pool, page_table,
                      remap, count, status) == cudaSuccess
               ? KVP_OK
               : KVP_ERR_CUDA;
  }
  const CompactWs ws = carve(workspace, BH, NS);
  int32_t* n_used = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + prep_bytes(BH, NS));
  uint2* owner = reinterpret_cast<uint2*>(n_used + 4);
  int device = 0;
  const int sms = current_sms(&device);
  if (sms == 0) return KVP_ERR_CUDA;
  const int segs = (NS + kWarpsPerCta - 1) / kWarpsPerCta;
  const bool fused = BH <= kFusedBH;
  int32_t* part = segs <= kMostSumsEach && BH * segs <= kMostSums ? ws.seg_off : nullptr;
  if (part == nullptr && launch_after(zero_counts_kernel, dim3(1), dim3(1024), st, BH, count) != cudaSuccess)
    return KVP_ERR_CUDA;
  uint4* high = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(owner) + owner_bytes(n_pages_cap));
  const bool scores = src.mode == KVP_MASK_KVZAP;
  const dim3 warps(kWarpsPerCta * 32);
  const cudaError_t counted =
      scores && src.H >= kManyHeads
          ? launch_pdl(count_scores_kernel, dim3(BH / src.H * ((src.H + 31) / 32), segs), dim3(kWarpsPerCta * kWords * 32), 0,
                       st, src, now, NS, BH, reinterpret_cast<uint32_t*>(high), ws.seg_cnt, part, count)
          : launch_pdl(scores ? count_segments_kernel<true> : count_segments_kernel<false>, dim3(BH, segs), warps, 0, st, src,
                       now, NS, high, ws.seg_cnt, part, count);
  if (counted != cudaSuccess) return KVP_ERR_CUDA;
  if (!fused && launch_after(base_kernel, dim3(1), dim3(1024), st, BH, reserve, max_pages, n_pages_cap, ws,
                             static_cast<const int32_t*>(count), status) != cudaSuccess)
    return KVP_ERR_CUDA;
  const auto list = fused ? (scores ? list_kernel<true, true> : list_kernel<true, false>)
                          : (scores ? list_kernel<false, true> : list_kernel<false, false>);
  if (launch_pdl(list, dim3(BH, segs), warps, 0, st, src, now, NS, (max_pages + NS - 1) / NS, reserve, max_pages,
                 n_pages_cap, BH, ws, static_cast<const int32_t*>(part), count, status, expire_pool, page_table, remap,
                 n_used, owner, static_cast<const uint4*>(high)) != cudaSuccess)
    return KVP_ERR_CUDA;
  // at most one page for each 16 positions and reserved slots: small calls take a small grid
  const int64_t most = static_cast<int64_t>(BH) * ((static_cast<int64_t>(src.n) + reserve + kPage - 1) / kPage);
  const int64_t need = (most < n_pages_cap ? most : n_pages_cap) / kPageWarps + 1;
  const int grid = static_cast<int>(need < sms * kPageCtas ? need : sms * kPageCtas);
  if (launch_pdl(page_kernel<D, FMT>, dim3(grid), dim3(kPageWarps * 32), 0, st, src.k, src.v, src.sb, src.st, src.sh,
                 src.H, static_cast<const int32_t*>(n_used), static_cast<const uint2*>(owner), max_pages,
                 static_cast<const int32_t*>(remap), kq_pool, vq_pool, reinterpret_cast<float2*>(scale_pool),
                 expire_pool) != cudaSuccess)
    return KVP_ERR_CUDA;
  return KVP_OK;
}

kvp_status append_block8_impl(int fmt, int mode, int batch, int n_kv_heads, int head_dim, int pos,
                              const int32_t* pos_dev, const void* k_new, const void* v_new, int64_t k_stride_b,
                              int64_t k_stride_h, int64_t v_stride_b, int64_t v_stride_h, const float* score,
                              const float* tau, const int32_t* flag_step, int window, int delay, void* kq_pool,
                              void* vq_pool, float* scale_pool, int32_t* expire_pool, int n_pages_cap,
                              const int32_t* page_table, int max_pages, int32_t* remap, int32_t* count,
                              int32_t* status, void* stream) {
  if (pos < 0 || window < 0 || delay < 0) return KVP_ERR_INVALID;
  const kvp_status s = check_block8(fmt, batch, n_kv_heads, head_dim, kq_pool, vq_pool, scale_pool, n_pages_cap,
                                    page_table, max_pages, count, status);
  if (s != KVP_OK) return s;
  if ((reinterpret_cast<uintptr_t>(pos_dev) & 3u) != 0) return KVP_ERR_ALIGN;
  if (mode == KVP_MASK_KVZAP) {
    if (score == nullptr || tau == nullptr || flag_step != nullptr) return KVP_ERR_INVALID;
  } else if (mode == KVP_MASK_DMS) {
    if (flag_step == nullptr || score != nullptr || tau != nullptr) return KVP_ERR_INVALID;
  } else {
    return KVP_ERR_INVALID;
  }
  if (k_new == nullptr || v_new == nullptr || expire_pool == nullptr || remap == nullptr) return KVP_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new)) return KVP_ERR_ALIGN;
  if (k_stride_b < 0 || k_stride_h < 0 || v_stride_b < 0 || v_stride_h < 0) return KVP_ERR_INVALID;
  if (k_stride_b % 8 || k_stride_h % 8 || v_stride_b % 8 || v_stride_h % 8) return KVP_ERR_ALIGN;
  if (static_cast<int64_t>(pos) + window + delay >= kNever) return KVP_ERR_INVALID;
  const int BH = batch * n_kv_heads;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((BH + kAppendWarps - 1) / kAppendWarps), dim3(kAppendWarps * 32), 0,
                      static_cast<cudaStream_t>(stream), mode, BH, n_kv_heads, pos, pos_dev,
                      static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new), k_stride_b, k_stride_h,
                      v_stride_b, v_stride_h, score, tau, flag_step, window, delay, static_cast<uint8_t*>(kq_pool),
                      static_cast<uint8_t*>(vq_pool), reinterpret_cast<float2*>(scale_pool), expire_pool, n_pages_cap,
                      page_table, max_pages, remap, count, status) == cudaSuccess
               ? KVP_OK
               : KVP_ERR_CUDA;
  };
  if (fmt == KVP_BLOCK8_E4M3)
    return head_dim == 128 ? go(append_block8_kernel<128, KVP_BLOCK8_E4M3>) : go(append_block8_kernel<64, KVP_BLOCK8_E4M3>);
  return head_dim == 128 ? go(append_block8_kernel<128, KVP_BLOCK8_INT8>) : go(append_block8_kernel<64, KVP_BLOCK8_INT8>);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" size_t kvp_compact_block8_workspace_bytes(int batch, int n_kv_heads, int n_pos, int n_pages_cap) {
  if (batch <= 0 || n_kv_heads <= 0 || n_pos < 0 || n_pages_cap < 0) return 0;
  return block8_ws_bytes(static_cast<int64_t>(batch) * n_kv_heads, n_segments(n_pos), n_pages_cap);
}

extern "C" kvp_status kvp_compact_block8(int fmt, int mode, int batch, int n_kv_heads, int head_dim, int n_pos,
                                         const void* k_src, const void* v_src, int64_t stride_b, int64_t stride_t,
                                         int64_t stride_h, const float* scores, const float* tau,
                                         const int32_t* flag_step, int window, int delay, int now, int reserve,
                                         void* kq_pool, void* vq_pool, float* scale_pool, int32_t* expire_pool,
                                         int n_pages_cap, int32_t* page_table, int max_pages, int32_t* remap,
                                         int32_t* count, void* workspace, size_t workspace_bytes, int32_t* status,
                                         void* stream) {
  if (n_pos < 0 || window < 0 || delay < 0 || reserve < 0) return KVP_ERR_INVALID;
  const kvp_status s = check_block8(fmt, batch, n_kv_heads, head_dim, kq_pool, vq_pool, scale_pool, n_pages_cap,
                                    page_table, max_pages, count, status);
  if (s != KVP_OK) return s;
  if (expire_pool == nullptr || remap == nullptr) return KVP_ERR_INVALID;
  // the per-position inputs may be NULL when there are no positions; tau is read per (b, h)
  if (mode == KVP_MASK_KVZAP) {
    if (flag_step != nullptr || tau == nullptr || (n_pos > 0 && scores == nullptr)) return KVP_ERR_INVALID;
  } else if (mode == KVP_MASK_DMS) {
    if (scores != nullptr || tau != nullptr || (n_pos > 0 && flag_step == nullptr)) return KVP_ERR_INVALID;
  } else {
    return KVP_ERR_INVALID;
  }
  if (static_cast<int64_t>(n_pos) + window + delay >= kNever) return KVP_ERR_INVALID;
  if (static_cast<int64_t>(n_pos) + reserve > 0x7fffffff - kPage) return KVP_ERR_UNSUPPORTED;
  if (n_pos > 0 && (k_src == nullptr || v_src == nullptr)) return KVP_ERR_INVALID;
  if (!aligned16(k_src) || !aligned16(v_src) || stride_b % 8 || stride_t % 8 || stride_h % 8) return KVP_ERR_ALIGN;
  if (stride_b < 0 || stride_t < 0 || stride_h < 0) return KVP_ERR_INVALID;
  const int BH = batch * n_kv_heads;
  const int NS = n_segments(n_pos);
  if ((NS + kWarpsPerCta - 1) / kWarpsPerCta > 65535) return KVP_ERR_UNSUPPORTED;  // the grid's second dimension
  // page ids are 32-bit: with every position kept they have to be countable, or the budget check could wrap
  if (BH * ((static_cast<int64_t>(n_pos) + reserve + kPage - 1) / kPage) > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < block8_ws_bytes(BH, NS, n_pages_cap)) return KVP_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVP_ERR_ALIGN;
  const MaskedSrc src{static_cast<const uint16_t*>(k_src),
                      static_cast<const uint16_t*>(v_src),
                      stride_b,
                      stride_t,
                      stride_h,
                      mode,
                      scores,
                      tau,
                      flag_step,
                      window,
                      delay,
                      n_kv_heads,
                      n_pos};
  auto go = [&](auto run) {
    return run(src, BH, NS, now, reserve, static_cast<uint8_t*>(kq_pool), static_cast<uint8_t*>(vq_pool), scale_pool,
               expire_pool, n_pages_cap, page_table, max_pages, remap, count, workspace, status,
               static_cast<cudaStream_t>(stream));
  };
  if (fmt == KVP_BLOCK8_E4M3)
    return head_dim == 128 ? go(launch_compact<128, KVP_BLOCK8_E4M3>) : go(launch_compact<64, KVP_BLOCK8_E4M3>);
  return head_dim == 128 ? go(launch_compact<128, KVP_BLOCK8_INT8>) : go(launch_compact<64, KVP_BLOCK8_INT8>);
}

extern "C" kvp_status kvp_append_block8(int fmt, int mode, int batch, int n_kv_heads, int head_dim, int pos,
                                        const void* k_new, const void* v_new, int64_t k_stride_b, int64_t k_stride_h,
                                        int64_t v_stride_b, int64_t v_stride_h, const float* score, const float* tau,
                                        const int32_t* flag_step, int window, int delay, void* kq_pool, void* vq_pool,
                                        float* scale_pool, int32_t* expire_pool, int n_pages_cap,
                                        const int32_t* page_table, int max_pages, int32_t* remap, int32_t* count,
                                        int32_t* status, void* stream) {
  return append_block8_impl(fmt, mode, batch, n_kv_heads, head_dim, pos, nullptr, k_new, v_new, k_stride_b, k_stride_h,
                            v_stride_b, v_stride_h, score, tau, flag_step, window, delay, kq_pool, vq_pool, scale_pool,
                            expire_pool, n_pages_cap, page_table, max_pages, remap, count, status, stream);
}

extern "C" kvp_status kvp_append_block8_devpos(int fmt, int mode, int batch, int n_kv_heads, int head_dim,
                                               const int32_t* pos_dev, const void* k_new, const void* v_new,
                                               int64_t k_stride_b, int64_t k_stride_h, int64_t v_stride_b,
                                               int64_t v_stride_h, const float* score, const float* tau,
                                               const int32_t* flag_step, int window, int delay, void* kq_pool,
                                               void* vq_pool, float* scale_pool, int32_t* expire_pool, int n_pages_cap,
                                               const int32_t* page_table, int max_pages, int32_t* remap,
                                               int32_t* count, int32_t* status, void* stream) {
  if (pos_dev == nullptr) return KVP_ERR_INVALID;
  return append_block8_impl(fmt, mode, batch, n_kv_heads, head_dim, 0, pos_dev, k_new, v_new, k_stride_b, k_stride_h,
                            v_stride_b, v_stride_h, score, tau, flag_step, window, delay, kq_pool, vq_pool, scale_pool,
                            expire_pool, n_pages_cap, page_table, max_pages, remap, count, status, stream);
}

extern "C" kvp_status kvp_read_block8(int fmt, int batch, int n_kv_heads, int head_dim, const void* kq_pool,
                                      const void* vq_pool, const float* scale_pool, int n_pages_cap,
                                      const int32_t* page_table, int max_pages, const int32_t* count, int first_slot,
                                      int n_slots, void* k_out, void* v_out, int64_t stride_b, int64_t stride_t,
                                      int64_t stride_h, int32_t* status, void* stream) {
  if (first_slot < 0 || n_slots < 0) return KVP_ERR_INVALID;
  const kvp_status s = check_block8(fmt, batch, n_kv_heads, head_dim, kq_pool, vq_pool, scale_pool, n_pages_cap,
                                    page_table, max_pages, count, status);
  if (s != KVP_OK) return s;
  if (static_cast<int64_t>(first_slot) + n_slots > 0x7fffffff - kPage) return KVP_ERR_UNSUPPORTED;
  if (n_slots == 0) return KVP_OK;
  if (k_out == nullptr || v_out == nullptr) return KVP_ERR_INVALID;
  if (!aligned16(k_out) || !aligned16(v_out) || stride_b % 8 || stride_t % 8 || stride_h % 8) return KVP_ERR_ALIGN;
  if (!rows_apart({{{stride_b, batch}, {stride_t, n_slots}, {stride_h, n_kv_heads}}}, head_dim)) return KVP_ERR_INVALID;
  const int pages_each = (first_slot + n_slots - 1) / kPage - first_slot / kPage + 1;
  const int64_t items = static_cast<int64_t>(batch) * n_kv_heads * pages_each;
  const int64_t ctas = (items + kPageWarps - 1) / kPageWarps;
  if (ctas > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kPageWarps * 32), 0,
                      static_cast<cudaStream_t>(stream), n_kv_heads, items, pages_each,
                      static_cast<const uint8_t*>(kq_pool), static_cast<const uint8_t*>(vq_pool),
                      reinterpret_cast<const float2*>(scale_pool), n_pages_cap, page_table, max_pages, count, first_slot,
                      n_slots, static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out), stride_b, stride_t, stride_h,
                      status) == cudaSuccess
               ? KVP_OK
               : KVP_ERR_CUDA;
  };
  if (fmt == KVP_BLOCK8_E4M3)
    return head_dim == 128 ? go(read_block8_kernel<128, KVP_BLOCK8_E4M3>) : go(read_block8_kernel<64, KVP_BLOCK8_E4M3>);
  return head_dim == 128 ? go(read_block8_kernel<128, KVP_BLOCK8_INT8>) : go(read_block8_kernel<64, KVP_BLOCK8_INT8>);
}
