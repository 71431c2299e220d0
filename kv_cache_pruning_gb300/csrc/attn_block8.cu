// kvp_decode_attn_block8: single-query GQA attention over a paged cache held
// in 8 bits with one power-of-two scale per page for K and one for V.
//
//   out[b, j] = sum_i softmax_i(scale q[b, j] . k_i) v_i,  k = ks c_k, v = vs c_v
//
// A page's scales leave the sums: its logits are ks times the products of q
// with the codes, its share of the output is vs times the weighted sum of the
// codes. So the codes themselves are the tensor-core operands, as fp16 (exact
// for both formats), and nothing is dequantised to memory.
//
// One warp takes a page at a time, in two products of mma.sync m16n8k16:
//   S = K q^T    16 tokens x 8 query heads, K's codes as the A operand
//   O += V^T P   16 channels x 8 query heads, V's codes transposed as A
// Both products may run over their summed index in any order, and the output's
// channels may sit in any row, so the operands' layouts are chosen such that
// every lane's fragment is made of 16-byte runs of a page's rows: codes go
// from global memory straight to registers, with no shared memory, and V's
// transposition is two byte permutes per pair of tokens. The weights cross
// from the first product's result to the second's operand by two movmatrix.
// tcgen05 does not fit here: its smallest tile has 64 or 128 rows of one
// operand in shared memory, of which a page and 8 heads fill a fraction.
//
// Precision: q is scaled by a power of two per head and turned into fp16
// exactly (but for elements 2^-28 of the largest). The weights
// (at most 2^15; the largest of a row is 2^12 or more, 1 or more at logits whose
// steps in fp32 are 8 and more) enter the second product
// as an fp16 pair hi + lo: 22 bits, and never further off than 2^-25, 2^-37 of
// the row's sum (2^-25 at such logits). With at most 4 heads per kv head the pair fills the 8 columns of one product
// (hi in columns 0..3, lo in 4..7), with 5 to 8 it takes two. A page's product
// starts from zero and is added to the fp32 accumulators with the V scale by
// fused multiply-adds. They hold 2^-23 of the weighted sums, which are up to 2^15
// a slot larger than the values: no sum of values whose magnitudes add up to less
// than 2^135 overflows, and the smallest scale, 2^-126, still is a number (a power of
// two, so that nothing else changes).
//
// The running reference is lazy: it is 12 below the largest base-2 logit when it
// moves (rounded up, so that logits of any size stay within 12 above it), and
// moves only when a logit is more than 15 above it (a vote per page), so most
// pages need no shuffles and no rescaling. A logit is compared with the
// reference by their difference, which is exact where it matters: a sum of the
// reference and 15 rounds by more than that at logits of 2^25, where a weight
// would leave fp16's range.
//
// Work split: all pages of all (b, h) form one list (b-major, h-minor, page
// order), cut evenly over the CTAs and, within a CTA, over its warps. Partial
// results of a (b, h) that several warps share are merged in shared memory;
// those that several CTAs share go to the workspace, and the last CTA to
// arrive merges them. Nothing ever waits on another CTA.
#include <atomic>

#include "block8.cuh"

namespace kvp {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxBH = 4096;     // (b, h) pairs whose page prefix fits in shared memory
constexpr int kMaxCtas = 512;    // grid bound used to size the workspace
constexpr float kBelow = 12.f;   // the reference's distance from the largest base-2 logit when it moves
constexpr float kAbove = 15.f;   // how far a logit may be above it: weights 2^(x - m) are at most 2^15 in fp16
constexpr float kDown = 1.f / 8388608.f;  // the accumulators' share of the weighted sums, 2^-23
constexpr int kFewPieces = 8;    // CTAs whose partial results of one (b, h) are merged in one round trip
// Pages by which the longest (b, h) may pass an even share to have a CTA of its own: its further pages against a merge
// between CTAs. Measured on a GB300 with (b, h)s of equal length and 4 queries each (us on the device, a CTA of their own /
// dealt out evenly), at 72, 96 and 120 pages more than an even share: E4M3 of 128, 8 (b, h) 9.7 / 11.4, 11.5 / 11.6, 12.9 /
// 11.4, 64 (b, h) 14.7 / 16.1, 17.7 / 18.1, 20.2 / 19.3, 128 (b, h) 42.6 / 46.2, 54.3 / 58.0, 66.7 / 69.7; int8 of 128, 8
// (b, h) 10.7 / 11.7, 12.9 / 12.0, 14.6 / 11.8, 64 (b, h) 16.0 / 16.7, 19.8 / 18.6, 22.7 / 20.1; E4M3 of 64, 8 (b, h) 7.5 /
// 9.8, 8.8 / 10.2, 9.8 / 10.1, 64 (b, h) 11.4 / 13.2, 13.8 / 14.5, 15.6 / 15.4; int8 of 64, 64 (b, h) 11.8 / 13.5, 14.4 /
// 14.9, 16.4 / 15.7. With 8 and 64 (b, h) the two are level at 80 (int8 of 128) to 140 (E4M3 of 64); with 128, which HBM
// bounds, at 108 (E4M3 of 64), 155 (int8 of 128) and past 200 (E4M3 of 128), so that right above 96 they lose a little.
constexpr int kOwnExtra = 96;
constexpr int kCtaPages = 2 * kWarps;  // fewest pages of an even share: more CTAs would have more to merge
constexpr int kAhead = 1;        // pages whose lines are brought into L2 before their loads
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  const uint16_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float2* scale_pool;
  const int32_t* expire_pool;
  const int32_t* page_table;
  const int32_t* count;
  const int32_t* now_dev;
  int BH, G, max_pages, n_pages_cap, now;
  int64_t table_lines, q_lines;  // 128-byte lines of the page table and the queries worth bringing into L2 early
  float qscale;        // scale * log2(e)
  float* out;          // [B, Hq, D]
  float* lse;          // [B, Hq] or null
  int32_t* arrived;    // [BH] counters, zero at entry and exit
  float* part_acc;     // [2 * grid, G, D]
  float* part_ml;      // [2 * grid, G, 2]
  int32_t* status;
};

KVP_DEV uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
KVP_DEV void prefetch_l2(const void* a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); }
// d = A B with a zero accumulator.
KVP_DEV void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The four codes of a word as two fp16 pairs (codes 0, 1 and 2, 3). int8: the
// byte with its sign bit flipped becomes 1024 + (c + 128) as fp16 (0x64 in the
// high byte), less 1152.
template <int FMT>
KVP_DEV void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == KVP_BLOCK8_E4M3) {
    lo = cvt_e4m3x2_to_f16x2(w);
    hi = cvt_e4m3x2_to_f16x2(w >> 16);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

KVP_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A warp's share of one (b, h): fp32 accumulators, reference and sum of its
// lane's two heads (2t, 2t + 1; t = lane % 4). Lane (g, t) holds channels
// g * D/8 .. + D/8 of both heads: acc[i] = {channel 2i head 2t, channel 2i
// head 2t+1, channel 2i+1 head 2t, channel 2i+1 head 2t+1}.
template <int D>
struct State {
  float acc[D / 16][4];
  float m[2], l[2];
  KVP_DEV void clear() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }
};

// The words of a page that a lane holds. K: row g's (and g + 8's) 16-byte runs
// t * 16 and, at D = 128, 64 + t * 16. V: the run g * D/8 of the rows 2t,
// 2t + 1, 2t + 8, 2t + 9.
template <int D>
struct KWords {
  uint32_t w[2][D / 16];
};
template <int D>
struct VWords {
  uint32_t w[4][D / 32];
};

template <int D>
KVP_DEV void load_k(KWords<D>& x, const uint8_t* page, int g, int t) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint4 y = *reinterpret_cast<const uint4*>(page + (g + 8 * r) * D + c * 64 + t * 16);
      x.w[r][4 * c] = y.x;
      x.w[r][4 * c + 1] = y.y;
      x.w[r][4 * c + 2] = y.z;
      x.w[r][4 * c + 3] = y.w;
    }
}
template <int D>
KVP_DEV void load_v(VWords<D>& x, const uint8_t* page, int g, int t) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint8_t* row = page + (2 * t + (r & 1) + 8 * (r >> 1)) * D + g * (D / 8);
    if constexpr (D == 128) {
      const uint4 y = *reinterpret_cast<const uint4*>(row);
      x.w[r][0] = y.x;
      x.w[r][1] = y.y;
      x.w[r][2] = y.z;
      x.w[r][3] = y.w;
    } else {
      const uint2 y = *reinterpret_cast<const uint2*>(row);
      x.w[r][0] = y.x;
      x.w[r][1] = y.y;
    }
  }
}

// Shared memory: page prefix, then each warp's two partial results (the (b, h)
// its range starts in, and the one it ends in), then what a merge over CTAs
// takes: (reference, sum) of each head and CTA, and a row of partial sums for
// each thread.
template <int D>
__host__ __device__ constexpr int part_floats(int G) {
  return (G * (D + 2) + 3) & ~3;
}
__host__ __device__ constexpr size_t prefix_bytes(int BH) { return static_cast<size_t>(BH + 4) / 4 * 16; }
template <int D>
__host__ __device__ constexpr size_t smem_bytes(int BH, int G) {
  return prefix_bytes(BH) + static_cast<size_t>(kWarps) * 2 * part_floats<D>(G) * 4 +
         static_cast<size_t>(G) * kMaxCtas * 8 + kThreads * 16;
}

// What takes a row's accumulators to its output, from its sum of weights (0 for a row without slots).
KVP_DEV float out_factor(float l) { return l == 0.f ? 0.f : (1.f / kDown) / l; }

// A row's log-sum-exp from its reference and sum (0 for a row without slots; NaN passes through).
KVP_DEV void write_lse(const Params& p, int64_t row, float m, float l) {
  if (p.lse != nullptr) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// kDup: at most 4 heads per kv head, hi and lo weights in one product.
template <int D, int FMT, bool kDup>
__global__ void __launch_bounds__(kThreads, 1) attn_block8_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ int4 warp_stat[kWarps];     // pages of a warp's (b, h)s: sum, most, fewest
  __shared__ int part_unit[kWarps * 2];
  __shared__ float wts[8][2 * kWarps];   // a merge's weights: head, partial result
  __shared__ float2 merged_ml[8];
  __shared__ int last_s[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int G = p.G;
  const int pf = part_floats<D>(G);
  int* prefix = reinterpret_cast<int*>(sm);
  float* parts = reinterpret_cast<float*>(sm + prefix_bytes(p.BH));
  float2* cta_ml = reinterpret_cast<float2*>(parts + kWarps * 2 * pf);
  float4* rows = reinterpret_cast<float4*>(cta_ml + G * kMaxCtas);
  // the page table's and the queries' lines on their way to L2 while the counts are read and summed up
  {
    const int64_t line = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
    if (line < p.table_lines) prefetch_l2(reinterpret_cast<const uint8_t*>(p.page_table) + line * 128);
    else if (line - p.table_lines < p.q_lines) prefetch_l2(reinterpret_cast<const uint8_t*>(p.q) + (line - p.table_lines) * 128);
  }
  pdl_wait();
  const int now = p.now_dev != nullptr ? *p.now_dev : p.now;

  // ---- pages before each (b, h)
  const int cap = p.max_pages * kPage;
  const int each = (p.BH + kThreads - 1) / kThreads;
  auto pages_of = [&](int u) { return (min(max(p.count[u], 0), cap) + kPage - 1) / kPage; };
  int sum = 0, most = 0, least = 1;
  for (int i = tid * each; i < min(p.BH, (tid + 1) * each); ++i) {
    const int pages = pages_of(i);
    sum += pages;
    most = max(most, pages);
    least = min(least, pages);
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 31) warp_stat[warp] = make_int4(incl, most, least, 0);
  if (tid < kWarps * 2) part_unit[tid] = -1;
  __syncthreads();
  const int4 st = lane < kWarps ? warp_stat[lane] : make_int4(0, 0, 1, 0);
  const int total = __reduce_add_sync(0xffffffffu, st.x);
  int at_page = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? st.x : 0);
  most = __reduce_max_sync(0xffffffffu, st.y);
  least = __reduce_min_sync(0xffffffffu, st.z);
  // A CTA for each (b, h), where there are enough of them and no (b, h) is much longer than an even share: nothing to
  // merge between CTAs. Otherwise all pages are dealt out evenly.
  const bool own = p.BH <= static_cast<int>(gridDim.x) &&
                   most - total / static_cast<int>(gridDim.x) <= kOwnExtra;
  int ctas;
  if (own) {
    ctas = p.BH;
    if (tid == 0 && static_cast<int>(blockIdx.x) < p.BH) {
      prefix[blockIdx.x] = 0;
      prefix[blockIdx.x + 1] = pages_of(blockIdx.x);
    }
  } else {
    for (int i = tid * each; i < min(p.BH, (tid + 1) * each); ++i) {
      prefix[i] = at_page;
      at_page += pages_of(i);
    }
    if (tid == 0) prefix[p.BH] = total;
    ctas = min(static_cast<int>(gridDim.x), (total + kCtaPages - 1) / kCtaPages);
  }
  __syncthreads();

  // rows of (b, h) without pages
  for (int u = blockIdx.x; least == 0 && u < p.BH; u += gridDim.x) {
    if (prefix[u + 1] > prefix[u]) continue;
    for (int i = tid; i < G * D; i += kThreads) p.out[static_cast<int64_t>(u) * G * D + i] = 0.f;
    if (p.lse != nullptr && tid < G) p.lse[static_cast<int64_t>(u) * G + tid] = -INFINITY;
  }

  // ---- this CTA's and this warp's pages
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  // CTA c takes pages cta_begin(c) .. cta_begin(c + 1) - 1: `share` each, the first `extra` CTAs one more
  const int share = own ? 0 : total / ctas, extra = own ? 0 : total - share * ctas;
  auto cta_begin = [&](int c) { return c * share + min(c, extra); };
  const int c_lo = own ? 0 : cta_begin(blockIdx.x), c_hi = own ? prefix[blockIdx.x + 1] : cta_begin(blockIdx.x + 1);
  const int lo = c_lo + warp * ((c_hi - c_lo) / kWarps) + min(warp, (c_hi - c_lo) % kWarps);
  const int hi = c_lo + (warp + 1) * ((c_hi - c_lo) / kWarps) + min(warp + 1, (c_hi - c_lo) % kWarps);
  // the (b, h) of a page of the list: the last one whose pages start at or before it and that has any
  auto unit_of = [&](int page) {
    int a = 0, b = p.BH;
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (prefix[mid] <= page) a = mid; else b = mid;
    }
    return a;
  };

  if (lo < hi) {
    int at = lo;
    int u = own ? static_cast<int>(blockIdx.x) : unit_of(lo);
    while (at < hi) {
      while (prefix[u + 1] <= at) ++u;
      const int u_lo = prefix[u], u_hi = prefix[u + 1];
      const int end = min(hi, u_hi);
      const int cnt = min(max(p.count[u], 0), cap);
      // ---- this (b, h)'s queries, requested first: lane (g, t) takes head g's (kDup: g % 4's) channels of its words
      uint4 x[D / 32];
      {
        const int head = kDup ? (g & 3) : g;
        const uint16_t* row = p.q + (static_cast<int64_t>(u) * G + head) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          x[i] = make_uint4(0, 0, 0, 0);
          if (head < G) x[i] = *reinterpret_cast<const uint4*>(row + (i >> 1) * 64 + t * 16 + (i & 1) * 8);
        }
      }
      const int32_t* table = p.page_table + static_cast<int64_t>(u) * p.max_pages + (at - u_lo);
      const int n = end - at;            // pages of this (b, h) in the warp's range

      // ---- page ids, 32 at a time in the lanes, two blocks of them
      int ids0 = lane < n ? table[lane] : -1, ids1 = 32 + lane < n ? table[32 + lane] : -1, block = 0;
      auto id_of = [&](int i) {
        const int k = i - block;
        const int id = k < 32 ? __shfl_sync(0xffffffffu, ids0, k & 31) : __shfl_sync(0xffffffffu, ids1, k & 31);
        return id < p.n_pages_cap ? id : -1;
      };
      // A page's loads. One page ahead its K words and scales are requested as soon as the page before is
      // through the first product, its V words as soon as it is through the second; kAhead pages ahead its
      // lines are brought into L2 (one line a lane), which leaves the register loads an L2 latency to cover.
      KWords<D> kw;
      VWords<D> vw;
      float2 sc_next = make_float2(0.f, 0.f);
      int32_t e0_next = INT32_MIN, e1_next = INT32_MIN;
      auto request_k = [&](int id) {
        if (id >= 0) {
          load_k<D>(kw, p.k_pool + static_cast<int64_t>(id) * kPage * D, g, t);
          sc_next = p.scale_pool[id];
          e0_next = p.expire_pool[static_cast<int64_t>(id) * kPage + g];
          e1_next = p.expire_pool[static_cast<int64_t>(id) * kPage + g + 8];
        } else {  // a page that is not there: all of its slots absent
          if (lane == 0) record_error(p.status, KVP_ERR_BOUNDS);
          e0_next = e1_next = INT32_MIN;
        }
      };
      auto request_v = [&](int id) {
        if (id >= 0) load_v<D>(vw, p.v_pool + static_cast<int64_t>(id) * kPage * D, g, t);
      };
      auto bring = [&](int i) {
        if (i >= n) return;
        const int id = id_of(i);
        constexpr int kLines = D * kPage / 128;
        if (id >= 0 && lane < 2 * kLines) {
          const uint8_t* a = (lane < kLines ? p.k_pool : p.v_pool) + static_cast<int64_t>(id) * kPage * D +
                             (lane % kLines) * 128;
          prefetch_l2(a);
        }
      };
      {
        const int id = id_of(0);
        request_k(id);
        request_v(id);
      }
#pragma unroll
      for (int i = 1; i <= kAhead; ++i) bring(i);

      // ---- the queries as B fragments
      uint32_t qf[D / 16][2];
      float qs[2];   // logits' factors of the lane's heads 2t, 2t + 1
      {
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          big = __vmaxu2(big, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                       __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
        uint32_t a = max(big & 0xFFFFu, big >> 16);
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
        // the head's largest element to 2^14 .. 2^15 (a row that is not finite keeps its infinities and NaNs)
        const int e = min(max(static_cast<int>(a >> 7), 16), 254);   // biased exponent
        const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          // words 4 (i >> 1) + 2 (i & 1) and the next: 4 channels each
          qf[2 * i][0] = pack_half2(bf16_lo(x[i].x) * up, bf16_hi(x[i].x) * up);
          qf[2 * i][1] = pack_half2(bf16_lo(x[i].y) * up, bf16_hi(x[i].y) * up);
          qf[2 * i + 1][0] = pack_half2(bf16_lo(x[i].z) * up, bf16_hi(x[i].z) * up);
          qf[2 * i + 1][1] = pack_half2(bf16_lo(x[i].w) * up, bf16_hi(x[i].w) * up);
        }
        const float f = p.qscale / up;
        qs[0] = __shfl_sync(0xffffffffu, f, 4 * (2 * t));
        qs[1] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + 1));
      }

      State<D> s;
      s.clear();
      for (int i = 0; i < n; ++i) {
        const int slot = (at - u_lo + i) * kPage;
        const bool in0 = slot + g < cnt && e0_next > now, in1 = slot + g + 8 < cnt && e1_next > now;
        const float2 sc = sc_next;
        // two sums, so that the products wait for one another half as often
        float x[4] = {0.f, 0.f, 0.f, 0.f}, x2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t a0, a1, a2, a3;
          codes_to_f16<FMT>(kw.w[0][j], a0, a2);
          codes_to_f16<FMT>(kw.w[1][j], a1, a3);
          mma_f16_16816(j & 1 ? x2 : x, a0, a1, a2, a3, qf[j][0], qf[j][1]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] += x2[c];
        const int id_next = i + 1 < n ? id_of(i + 1) : -1;
        if (i + 1 < n) request_k(id_next);
        const float f0 = qs[0] * sc.x, f1 = qs[1] * sc.x, fv = sc.y * kDown;
        x[0] = in0 ? x[0] * f0 : -INFINITY;
        x[1] = in0 ? x[1] * f1 : -INFINITY;
        x[2] = in1 ? x[2] * f0 : -INFINITY;
        x[3] = in1 ? x[3] * f1 : -INFINITY;
        // a reference that has fallen behind (or none yet, -inf) moves up to 12 below the page's maximum
        const float top0 = fmaxf(x[0], x[2]), top1 = fmaxf(x[1], x[3]);
        if (__any_sync(0xffffffffu, top0 - s.m[0] > kAbove || top1 - s.m[1] > kAbove)) {
          float m0 = top0, m1 = top1;
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
          }
          m0 = fmaxf(__fsub_ru(m0, kBelow), s.m[0]);
          m1 = fmaxf(__fsub_ru(m1, kBelow), s.m[1]);
          const float r0 = m0 == s.m[0] ? 1.f : ex2_approx(s.m[0] - m0), r1 = m1 == s.m[1] ? 1.f : ex2_approx(s.m[1] - m1);
          s.m[0] = m0;
          s.m[1] = m1;
          s.l[0] *= r0;
          s.l[1] *= r1;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            s.acc[j][0] *= r0;
            s.acc[j][1] *= r1;
            s.acc[j][2] *= r0;
            s.acc[j][3] *= r1;
          }
        }
        // a head whose reference is still -inf has only -inf logits: weight 0, not NaN
        const float c0 = s.m[0] == -INFINITY ? 0.f : s.m[0], c1 = s.m[1] == -INFINITY ? 0.f : s.m[1];
        const float w0 = ex2_approx(x[0] - c0), w1 = ex2_approx(x[1] - c1);
        const float w2 = ex2_approx(x[2] - c0), w3 = ex2_approx(x[3] - c1);
        s.l[0] += w0 + w2;
        s.l[1] += w1 + w3;
        const uint32_t h0 = pack_half2(w0, w1), h1 = pack_half2(w2, w3);
        const float2 q0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
        const float2 q1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        const uint32_t e0 = pack_half2(w0 - q0.x, w1 - q0.y), e1 = pack_half2(w2 - q1.x, w3 - q1.y);
        uint32_t b0, b1, d0 = 0, d1 = 0;
        if constexpr (kDup) {
          b0 = movmatrix_trans(t < 2 ? h0 : e0);
          b1 = movmatrix_trans(t < 2 ? h1 : e1);
        } else {
          b0 = movmatrix_trans(h0);
          b1 = movmatrix_trans(h1);
          d0 = movmatrix_trans(e0);
          d1 = movmatrix_trans(e1);
        }
        // a masked token's codes may be anything (an E4M3 NaN times a zero weight is NaN): its words become zero
        const unsigned live0 = __ballot_sync(0xffffffffu, in0), live1 = __ballot_sync(0xffffffffu, in1);
        if ((live0 & live1) != 0xffffffffu) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // row 2t + (r & 1) + 8 (r >> 1): its flag is lane 4 * row's
            const bool on = ((r >> 1 ? live1 : live0) >> (4 * (2 * t + (r & 1)))) & 1u;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vw.w[r][w] = on ? vw.w[r][w] : 0u;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // byte pairs (token 2t, token 2t + 1) of channels 4w, 4w + 1 | 4w + 2, 4w + 3, and of tokens 2t + 8, 2t + 9
          const uint32_t ab0 = __byte_perm(vw.w[0][w], vw.w[1][w], 0x5140), ab1 = __byte_perm(vw.w[0][w], vw.w[1][w], 0x7362);
          const uint32_t cd0 = __byte_perm(vw.w[2][w], vw.w[3][w], 0x5140), cd1 = __byte_perm(vw.w[2][w], vw.w[3][w], 0x7362);
          uint32_t a0, a1, a2, a3;
          float y[4];
          codes_to_f16<FMT>(ab0, a0, a1);
          codes_to_f16<FMT>(cd0, a2, a3);
          mma_f16_zero(y, a0, a1, a2, a3, b0, b1);
          if constexpr (!kDup) mma_f16_16816(y, a0, a1, a2, a3, d0, d1);
#pragma unroll
          for (int c = 0; c < 4; ++c) s.acc[2 * w][c] = fmaf(y[c], fv, s.acc[2 * w][c]);
          codes_to_f16<FMT>(ab1, a0, a1);
          codes_to_f16<FMT>(cd1, a2, a3);
          mma_f16_zero(y, a0, a1, a2, a3, b0, b1);
          if constexpr (!kDup) mma_f16_16816(y, a0, a1, a2, a3, d0, d1);
#pragma unroll
          for (int c = 0; c < 4; ++c) s.acc[2 * w + 1][c] = fmaf(y[c], fv, s.acc[2 * w + 1][c]);
        }
        if (i + 1 < n) {
          request_v(id_next);
          bring(i + 1 + kAhead);
          if (i + 1 - block == 32) {  // the first block of ids is used up
            ids0 = ids1;
            block += 32;
            ids1 = block + 32 + lane < n ? table[block + 32 + lane] : -1;
          }
        }
      }

      // ---- the warp's share of this (b, h) is done
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        s.l[0] += __shfl_xor_sync(0xffffffffu, s.l[0], o);
        s.l[1] += __shfl_xor_sync(0xffffffffu, s.l[1], o);
      }
      if constexpr (kDup) {  // lanes t and t + 2 hold the hi and the lo products of the same heads
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) s.acc[j][c] += __shfl_xor_sync(0xffffffffu, s.acc[j][c], 2);
      }
      const bool whole = at == u_lo && end == u_hi;
      // partial 0: the (b, h) the range starts in, unless it starts there too and ends elsewhere
      const int which = at == lo && !(at == u_lo) ? 0 : (end == u_hi ? 0 : 1);
      float* part = parts + (warp * 2 + which) * pf;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int head = 2 * t + hh;
        if (head < G && (!kDup || t < 2)) {
          float* dst = whole ? p.out + (static_cast<int64_t>(u) * G + head) * D : part + head * D;
          const float inv = whole ? out_factor(s.l[hh]) : 1.f;
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            reinterpret_cast<float4*>(dst + g * (D / 8))[j] =
                make_float4(s.acc[2 * j][hh] * inv, s.acc[2 * j][2 + hh] * inv, s.acc[2 * j + 1][hh] * inv,
                            s.acc[2 * j + 1][2 + hh] * inv);
          if (g == 0) {
            if (whole) {
              write_lse(p, static_cast<int64_t>(u) * G + head, s.m[hh], s.l[hh]);
            } else {
              part[G * D + 2 * head] = s.m[hh];
              part[G * D + 2 * head + 1] = s.l[hh];
            }
          }
        }
      }
      if (!whole && lane == 0) part_unit[warp * 2 + which] = u;
      at = end;
    }
  }
  __syncthreads();

  // ---- merge the CTA's partial results, one (b, h) after another: entry e of part_unit is lane e's
  const int my_unit = part_unit[lane];
  const unsigned same = __match_any_sync(0xffffffffu, my_unit);
  unsigned leaders = __ballot_sync(0xffffffffu, my_unit >= 0 && (same & ((1u << lane) - 1u)) == 0);
  int shared0 = -1, shared1 = -1;  // the (b, h)s that other CTAs share: at most the CTA's first (slot 0) and last (slot 1)
  while (leaders != 0) {
    const int lead = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const int u = __shfl_sync(0xffffffffu, my_unit, lead);
    const unsigned entries = __shfl_sync(0xffffffffu, same, lead);
    const int u_lo = prefix[u], u_hi = prefix[u + 1];
    const bool whole = u_lo >= c_lo && u_hi <= c_hi;
    if (warp < G) {  // one warp a head: the partial results' weights
      const bool in = (entries >> lane) & 1u;
      const float2 ml = in ? *reinterpret_cast<const float2*>(parts + lane * pf + G * D + 2 * warp)
                           : make_float2(-INFINITY, 0.f);
      float m = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float w = ml.x == m ? 1.f : ex2_approx(ml.x - m);
      float l = in ? w * ml.y : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      wts[warp][lane] = w;
      if (lane == 0) merged_ml[warp] = make_float2(m, l);
    }
    __syncthreads();
    const int side = u_lo <= c_lo ? 0 : 1;
    const int64_t slot = blockIdx.x * 2 + side;
    if (!whole && side == 0) shared0 = u;
    if (!whole && side == 1) shared1 = u;
    for (int i = tid; i < G * D / 4; i += kThreads) {
      const int head = i / (D / 4);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      unsigned left = entries;
      while (left != 0) {  // four at a time, so that their reads overlap
        int e[4];
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          e[k] = left != 0 ? __ffs(left) - 1 : lead;
          w[k] = left != 0 ? wts[head][e[k]] : 0.f;
          left &= left - 1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 x = reinterpret_cast<const float4*>(parts + e[k] * pf)[i];
          a.x = fmaf(w[k], x.x, a.x);
          a.y = fmaf(w[k], x.y, a.y);
          a.z = fmaf(w[k], x.z, a.z);
          a.w = fmaf(w[k], x.w, a.w);
        }
      }
      const float2 ml = merged_ml[head];
      if (whole) {
        const float inv = out_factor(ml.y);
        reinterpret_cast<float4*>(p.out + static_cast<int64_t>(u) * G * D)[i] =
            make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        if (i % (D / 4) == 0) write_lse(p, static_cast<int64_t>(u) * G + head, ml.x, ml.y);
      } else {
        reinterpret_cast<float4*>(p.part_acc + slot * G * D)[i] = a;
        if (i % (D / 4) == 0) reinterpret_cast<float2*>(p.part_ml)[slot * G + head] = ml;
      }
    }
    __syncthreads();  // the weights are read before the next (b, h) writes its own
  }
  if (shared0 < 0 && shared1 < 0) return;

  // ---- shared with other CTAs: the last one to arrive merges
  auto cta_of = [&](int page) {
    const int longer = extra * (share + 1);  // pages of the CTAs with one more
    return page < longer ? page / (share + 1) : extra + (page - longer) / share;
  };
  // the barrier above saw the CTA's partial results written; each thread's fence publishes them before it counts
  if (tid < 2) {
    const int u = tid == 0 ? shared0 : shared1;
    last_s[tid] = 0;
    if (u >= 0) {
      const int pieces = cta_of(prefix[u + 1] - 1) - cta_of(prefix[u]) + 1;
      fence_acq_rel_gpu();
      last_s[tid] = atomicAdd(&p.arrived[u], 1) == pieces - 1;
      if (last_s[tid]) fence_acq_rel_gpu();
    }
  }
  __syncthreads();
  for (int side = 0; side < 2; ++side) {
    if (!last_s[side]) continue;
    const int u = side == 0 ? shared0 : shared1;
    const int u_lo = prefix[u], first_cta = cta_of(u_lo), pieces = cta_of(prefix[u + 1] - 1) - first_cta + 1;
    // a CTA's partial result lies in its slot 0 if the (b, h) has begun where the CTA's pages begin, else in slot 1
    auto slot_of = [&](int c) { return static_cast<int64_t>(first_cta + c) * 2 + (c > 0 || u_lo <= cta_begin(first_cta) ? 0 : 1); };
    if (pieces <= kFewPieces) {  // everything a thread needs in one round trip
      for (int i = tid; i < G * D / 4; i += kThreads) {
        const int head = i / (D / 4);
        float2 ml[kFewPieces];
        float4 x[kFewPieces];
#pragma unroll
        for (int c = 0; c < kFewPieces; ++c) {
          ml[c] = make_float2(-INFINITY, 0.f);
          x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < pieces) {
            ml[c] = load8_l2(p.part_ml + (slot_of(c) * G + head) * 2);
            x[c] = load16_l2(p.part_acc + slot_of(c) * G * D + 4 * i);
          }
        }
        float m = ml[0].x, l = 0.f;
#pragma unroll
        for (int c = 1; c < kFewPieces; ++c) m = fmaxf(m, ml[c].x);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kFewPieces; ++c) {
          const float w = ml[c].x == m ? 1.f : ex2_approx(ml[c].x - m);
          l = fmaf(w, ml[c].y, l);
          a.x = fmaf(w, x[c].x, a.x);
          a.y = fmaf(w, x[c].y, a.y);
          a.z = fmaf(w, x[c].z, a.z);
          a.w = fmaf(w, x[c].w, a.w);
        }
        const float inv = out_factor(l);
        reinterpret_cast<float4*>(p.out + static_cast<int64_t>(u) * G * D)[i] =
            make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        if (i % (D / 4) == 0) write_lse(p, static_cast<int64_t>(u) * G + head, m, l);
      }
      if (tid == 0) p.arrived[u] = 0;
      continue;
    }
    if (warp < G) {
      float m = -INFINITY;
      for (int c = lane; c < pieces; c += 32) {
        const float2 ml = load8_l2(p.part_ml + (slot_of(c) * G + warp) * 2);
        cta_ml[warp * kMaxCtas + c] = ml;
        m = fmaxf(m, ml.x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float l = 0.f;
      for (int c = lane; c < pieces; c += 32) {
        float2& ml = cta_ml[warp * kMaxCtas + c];
        const float w = ml.x == m ? 1.f : ex2_approx(ml.x - m);
        l = fmaf(w, ml.y, l);
        ml.x = w;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) merged_ml[warp] = make_float2(m, l);
    }
    __syncthreads();
    // the threads in groups of G * D / 4, each group taking every `groups`-th CTA's partial result
    const int items = G * D / 4, groups = kThreads / items;
    const int i = tid % items, grp = tid / items, head = i / (D / 4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp < groups) {
#pragma unroll 4
      for (int c = grp; c < pieces; c += groups) {
        const float w = cta_ml[head * kMaxCtas + c].x;
        const float4 x = load16_l2(p.part_acc + slot_of(c) * G * D + 4 * i);
        a.x = fmaf(w, x.x, a.x);
        a.y = fmaf(w, x.y, a.y);
        a.z = fmaf(w, x.z, a.z);
        a.w = fmaf(w, x.w, a.w);
      }
    }
    rows[tid] = a;
    __syncthreads();
    if (grp == 0) {
      for (int k = 1; k < groups; ++k) {
        const float4 x = rows[k * items + i];
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
      }
      const float2 ml = merged_ml[head];
      const float inv = out_factor(ml.y);
      reinterpret_cast<float4*>(p.out + static_cast<int64_t>(u) * G * D)[i] =
          make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      if (i % (D / 4) == 0) write_lse(p, static_cast<int64_t>(u) * G + head, ml.x, ml.y);
    }
    if (tid == 0) p.arrived[u] = 0;
    __syncthreads();
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The arrival counters of the most (b, h)s come first whatever a call's own number is, so that no call's partial results
// lie where another call's counters have to be zero.
constexpr size_t kCountersBytes = static_cast<size_t>(kMaxBH) * 4;
size_t attn_ws_bytes(int G, int D) {
  return kCountersBytes + static_cast<size_t>(2) * kMaxCtas * G * (D + 2) * sizeof(float);
}

template <int D, int FMT, bool kDup>
kvp_status launch(const Params& p, int device, int grid, cudaStream_t st) {
  // the shared-memory limit is a property of the kernel on each device: set once there, for the largest call
  static std::atomic<uint64_t> ready{0};
  if (device > 63 || !((ready.load(std::memory_order_relaxed) >> device) & 1u)) {
    if (cudaFuncSetAttribute(attn_block8_kernel<D, FMT, kDup>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes<D>(kMaxBH, kDup ? 4 : 8))) != cudaSuccess) {
      (void)cudaGetLastError();
      return KVP_ERR_CUDA;
    }
    if (device <= 63) ready.fetch_or(uint64_t{1} << device, std::memory_order_relaxed);
  }
  return launch_pdl(attn_block8_kernel<D, FMT, kDup>, dim3(grid), dim3(kThreads), smem_bytes<D>(p.BH, p.G), st, p) ==
                 cudaSuccess
             ? KVP_OK
             : KVP_ERR_CUDA;
}

kvp_status attn_block8_impl(int fmt, int batch, int n_q_heads, int n_kv_heads, int head_dim, const void* q,
                            const void* kq_pool, const void* vq_pool, const float* scale_pool,
                            const int32_t* expire_pool, int n_pages_cap, const int32_t* page_table, int max_pages,
                            const int32_t* count, int now, const int32_t* now_dev, float scale, float* out, float* lse,
                            int grid_limit, void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  if (fmt != KVP_BLOCK8_E4M3 && fmt != KVP_BLOCK8_INT8) return KVP_ERR_INVALID;
  if (batch <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || max_pages < 0 || n_pages_cap < 0 || grid_limit < 0)
    return KVP_ERR_INVALID;
  if (!(scale >= 0.f) || scale > 3.402823466e38f) return KVP_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128) return KVP_ERR_UNSUPPORTED;
  if (n_q_heads % n_kv_heads != 0) return KVP_ERR_UNSUPPORTED;
  const int G = n_q_heads / n_kv_heads;
  const int64_t BH = static_cast<int64_t>(batch) * n_kv_heads;
  if (G > 8 || BH > kMaxBH) return KVP_ERR_UNSUPPORTED;
  if (BH * max_pages > 0x7fffffff || static_cast<int64_t>(max_pages) * kPage > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  if (q == nullptr || kq_pool == nullptr || vq_pool == nullptr || scale_pool == nullptr || expire_pool == nullptr ||
      page_table == nullptr || count == nullptr || out == nullptr)
    return KVP_ERR_INVALID;
  if (!al16(q) || !al16(kq_pool) || !al16(vq_pool) || !al16(scale_pool) || !al16(out)) return KVP_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(now_dev) & 3u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return KVP_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < attn_ws_bytes(G, head_dim)) return KVP_ERR_WORKSPACE;
  if (!al16(workspace)) return KVP_ERR_ALIGN;
  int device = 0;
  const int sms = current_sms(&device);
  if (sms == 0) return KVP_ERR_CUDA;
  int grid = sms < kMaxCtas ? sms : kMaxCtas;
  if (grid_limit > 0 && grid_limit < grid) grid = grid_limit;
  // no more CTAs than a full page table keeps busy
  const int64_t busy = (BH * max_pages + kCtaPages - 1) / kCtaPages;
  if (grid > BH && grid > busy) grid = static_cast<int>(busy > BH ? busy : BH);
  Params p;
  p.q = static_cast<const uint16_t*>(q);
  p.k_pool = static_cast<const uint8_t*>(kq_pool);
  p.v_pool = static_cast<const uint8_t*>(vq_pool);
  p.scale_pool = reinterpret_cast<const float2*>(scale_pool);
  p.expire_pool = expire_pool;
  p.page_table = page_table;
  p.count = count;
  p.now_dev = now_dev;
  p.BH = static_cast<int>(BH);
  p.G = G;
  p.max_pages = max_pages;
  p.n_pages_cap = n_pages_cap;
  p.now = now;
  p.qscale = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(head_dim))) * kLog2e;
  p.out = out;
  p.lse = lse;
  p.arrived = static_cast<int32_t*>(workspace);
  p.part_acc = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCountersBytes);
  p.part_ml = p.part_acc + static_cast<size_t>(2) * kMaxCtas * G * head_dim;
  p.status = status;
  // bringing lines into L2 early pays while one instruction of each thread does it; a table with more lines than
  // that is larger than its used part is likely to be
  const int64_t threads = static_cast<int64_t>(grid) * kThreads;
  p.table_lines = (BH * max_pages * 4 + 127) / 128;
  p.q_lines = (BH * G * head_dim * 2 + 127) / 128;
  if (p.table_lines + p.q_lines > threads) p.table_lines = 0;
  if (p.q_lines > threads) p.q_lines = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool dup = G <= 4;
#define KVP_ATTN8(D, F) (dup ? launch<D, F, true>(p, device, grid, st) : launch<D, F, false>(p, device, grid, st))
  if (fmt == KVP_BLOCK8_E4M3) return head_dim == 128 ? KVP_ATTN8(128, KVP_BLOCK8_E4M3) : KVP_ATTN8(64, KVP_BLOCK8_E4M3);
  return head_dim == 128 ? KVP_ATTN8(128, KVP_BLOCK8_INT8) : KVP_ATTN8(64, KVP_BLOCK8_INT8);
#undef KVP_ATTN8
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" size_t kvp_decode_attn_block8_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim) {
  if (batch <= 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  const int64_t BH = static_cast<int64_t>(batch) * n_kv_heads;
  if (n_q_heads / n_kv_heads > 8 || BH > kMaxBH) return 0;
  return attn_ws_bytes(n_q_heads / n_kv_heads, head_dim);
}

extern "C" kvp_status kvp_decode_attn_block8(int fmt, int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                             const void* q, const void* kq_pool, const void* vq_pool,
                                             const float* scale_pool, const int32_t* expire_pool, int n_pages_cap,
                                             const int32_t* page_table, int max_pages, const int32_t* count, int now,
                                             float scale, float* out, float* lse, int grid_limit, void* workspace,
                                             size_t workspace_bytes, int32_t* status, void* stream) {
  return attn_block8_impl(fmt, batch, n_q_heads, n_kv_heads, head_dim, q, kq_pool, vq_pool, scale_pool, expire_pool,
                          n_pages_cap, page_table, max_pages, count, now, nullptr, scale, out, lse, grid_limit,
                          workspace, workspace_bytes, status, stream);
}

extern "C" kvp_status kvp_decode_attn_block8_devpos(int fmt, int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                                    const void* q, const void* kq_pool, const void* vq_pool,
                                                    const float* scale_pool, const int32_t* expire_pool,
                                                    int n_pages_cap, const int32_t* page_table, int max_pages,
                                                    const int32_t* count, const int32_t* now_dev, float scale,
                                                    float* out, float* lse, int grid_limit, void* workspace,
                                                    size_t workspace_bytes, int32_t* status, void* stream) {
  if (now_dev == nullptr) return KVP_ERR_INVALID;
  return attn_block8_impl(fmt, batch, n_q_heads, n_kv_heads, head_dim, q, kq_pool, vq_pool, scale_pool, expire_pool,
                          n_pages_cap, page_table, max_pages, count, 0, now_dev, scale, out, lse, grid_limit, workspace,
                          workspace_bytes, status, stream);
}
