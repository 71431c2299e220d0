// kvp_qk_norm_rope: the norm of each query and key head's row and the position
// rotation of its first rot_dim values, in one pass over q and k; and
// kvp_rope_turns, its table of angles per position.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// Bound by memory (2 bytes in, 2 out a value). D / 16 lanes take a head's row,
// 16 values each in two 16-byte runs that lie half a rotation apart, so that
// both members of every pair are in one lane (for interleaved pairs any run
// does) and a lane's loads and stores stay 16 bytes wide; a row's norm is three
// (two at D = 64) shuffles. A warp takes one token's heads, or a share of them
// when there are few tokens, with the token's cosines and sines in registers.
//
// Measured on a GB300, 65,521 tokens x 40 heads of 128: 271 us at first, 239 with fewer
// registers a thread, 231 with the norm's weights folded into the cosines and sines and
// streaming loads, 210 (0.94 of measured HBM) with the weights in shared memory
// instead, which leaves the registers of 32 warps an SM without spills to speak of.
// Not kept: the next step's rows requested before this one's arithmetic (264), one
// step or three in flight instead of two (239, 241); scaling rows whose squares leave
// fp32's range by a power of two, behind a vote a row (214, 218 interleaved; 131,072 x
// 5 heads 82.5 against 80.4), after the other rows (215, 84.5), or in a function of its
// own (218, 82.6).
//
// An angle is a 64-bit product: turns[i] = inv_freq[i] / (2 pi) as a 64-bit
// fraction of a turn, times the position modulo one turn (the integer wraps
// exactly there), whose top 32 bits go to sincospif. No far position loses
// digits, and no argument reduction is needed.
#include <cmath>

#include "block8.cuh"

namespace kvp {
namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 2;  // rows a lane has in flight
constexpr int kCtas = 4;    // CTAs per SM: 32 warps with 2 KB in flight each (three: 218 us at 65,521 x 40 heads, five 243, they spill)
// Steps (of 32 / LPH rows) a token's heads may take for the kernel for few heads. Measured on a GB300, 131,072 tokens,
// heads side by side / tokens side by side: 2 heads of 128 151 / 59 us, 5 154 / 81, 8 113 / 92, 12 170 / 146, 16 226 /
// 195, 24 260 / 281; 24 heads of 64 174 / 136; 65,536 x 72 heads of 64 195 / 274; 65,521 x 40 of 128 210 / 255.
constexpr int kFewSteps = 5;

struct RotateParams {
  const uint16_t* x[2];   // q, k
  uint16_t* y[2];
  int64_t xt[2], xh[2], yt[2], yh[2];
  const float* w[2];
  const int32_t* pos;
  const uint64_t* turns;
  int heads[2];
  int64_t n_items;
  int parts;              // warps that a token's (a group of tokens') heads are dealt to
  int parts_q;            // rotate_tokens_kernel: those of them that take q's heads
  int64_t n_tok;
  int rot;
  float eps;
};

KVP_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
KVP_DEV void unpack_row(const uint4& a, const uint4& b, float (&f)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

// cos and sin of turns[pair] * pos
KVP_DEV void angle(const uint64_t* turns, int pair, uint64_t pos, float& c, float& s) {
  sincospif(static_cast<float>(static_cast<int32_t>((turns[pair] * pos) >> 32)) * (1.f / 2147483648.f), &s, &c);
}

// One row's 16 values of a lane (runs a, b): norm over the row's D / 16 lanes (if any), rotation, and to dst + run0 * 8
// and dst + run1 * 8. The cosines and sines of the lane's 8 pairs (e and e + 8, or kPairs: 2 e and 2 e + 1) are in
// registers, the norm's weights in shared memory (w4[c * D / 16]: the lane's values 4 c .. 4 c + 3): with them in
// registers too, folded into the cosines and sines, an SM has room for fewer warps (235 us against 210 at 65,521 x 40).
template <int D, bool kPairs>
KVP_DEV void turn_row(const uint4& a, const uint4& b, bool norm, float eps, bool rotates, const float (&cs)[8],
                        const float (&sn)[8], const float4* w4, bool store, uint16_t* dst, int run0, int run1) {
  float f[16];
  unpack_row(a, b, f);
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum = fmaf(f[e], f[e], sum);
#pragma unroll
    for (int o = 1; o < D / 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = rsqrtf(sum * (1.f / D) + eps);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 w = w4[c * (D / 16)];
      f[4 * c] *= r * w.x;
      f[4 * c + 1] *= r * w.y;
      f[4 * c + 2] *= r * w.z;
      f[4 * c + 3] *= r * w.w;
    }
  }
  if (rotates) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = kPairs ? 2 * e : e, k = kPairs ? 2 * e + 1 : e + 8;
      const float m = f[i], n = f[k];
      f[i] = m * cs[e] - n * sn[e];
      f[k] = n * cs[e] + m * sn[e];
    }
  }
  if (store) {
    uint4* out = reinterpret_cast<uint4*>(dst);
    __stcs(out + run0, make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
    __stcs(out + run1, make_uint4(pack_bf16(f[8], f[9]), pack_bf16(f[10], f[11]), pack_bf16(f[12], f[13]),
                                  pack_bf16(f[14], f[15])));
  }
}

// The runs of 8 values that lane j of a row's LPH lanes takes: pairs of rotated runs first, then what is left of the row
// in the same manner. Returns whether they are rotated ones.
template <int LPH>
KVP_DEV bool runs_of(int j, int rot, int& run0, int& run1) {
  const int nh = rot / 16;
  run0 = j < nh ? j : nh + j;
  run1 = run0 + (j < nh ? nh : LPH - nh);
  return j < nh;
}

// The norm weights of q and of k, by lane: w_s[(which * 4 + c) * LPH + j] holds values 4 c .. 4 c + 3 of lane j's runs.
template <int LPH>
KVP_DEV void load_weights(const RotateParams& p, float4* w_s) {
  for (int i = threadIdx.x; i < 2 * 4 * LPH; i += kWarps * 32) {
    const float* w = p.w[i / (4 * LPH)];
    int run0, run1;
    runs_of<LPH>(i % LPH, p.rot, run0, run1);
    const int c = i / LPH % 4;
    if (w != nullptr) w_s[i] = *reinterpret_cast<const float4*>(w + (c < 2 ? run0 : run1) * 8 + (c & 1) * 4);
  }
  __syncthreads();
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32, kCtas) rotate_kernel(const RotateParams p) {
  constexpr int LPH = D / 16;       // lanes a head takes
  constexpr int HPI = 32 / LPH;     // heads a warp takes at once
  __shared__ float4 w_s[2 * 4 * LPH];
  pdl_wait();
  load_weights<LPH>(p, w_s);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= p.n_items) return;
  const int lane = threadIdx.x & 31, j = lane % LPH, sub = lane / LPH;
  const int64_t tok = item / p.parts;
  const int part = static_cast<int>(item - tok * p.parts);

  int run0, run1;
  const bool turns_here = runs_of<LPH>(j, p.rot, run0, run1);

  // cosines and sines of the lane's 8 pairs: 2 (1 at D = 64) are computed, the others
  // fetched from the lanes of the warp's other heads, which share the token's angles
  float cs[8], sn[8];
  if (p.rot > 0) {
    constexpr int kMine = 8 / HPI > 0 ? 8 / HPI : 1;
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.pos[tok]));
    float c[kMine], s[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = sub * kMine + i;   // of the lane's 8 pairs
      c[i] = 1.f;
      s[i] = 0.f;
      if (turns_here) angle(p.turns, kPairs ? (e < 4 ? 4 * run0 + e : 4 * run1 + e - 4) : 8 * run0 + e, pos, c[i], s[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = __shfl_sync(0xffffffffu, c[e % kMine], (e / kMine) * LPH + j);
      sn[e] = __shfl_sync(0xffffffffu, s[e % kMine], (e / kMine) * LPH + j);
    }
  }

  const int it_q = (p.heads[0] + HPI - 1) / HPI, it_all = it_q + (p.heads[1] + HPI - 1) / HPI;
  const int lo = static_cast<int>(static_cast<int64_t>(part) * it_all / p.parts);
  const int hi = static_cast<int>(static_cast<int64_t>(part + 1) * it_all / p.parts);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int i_lo = which == 0 ? lo : max(lo, it_q) - it_q, i_hi = which == 0 ? min(hi, it_q) : hi - it_q;
    if (i_lo >= i_hi) continue;
    const int heads = p.heads[which];
    const uint16_t* x = p.x[which] + tok * p.xt[which];
    uint16_t* y = p.y[which] + tok * p.yt[which];
    const float* wp = p.w[which];
#pragma unroll 1
    for (int i0 = i_lo; i0 < i_hi; i0 += kUnroll) {
      uint4 a[kUnroll], b[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = (i0 + u) * HPI + sub;
        a[u] = b[u] = make_uint4(0, 0, 0, 0);
        if (i0 + u < i_hi && h < heads) {
          a[u] = load16_stream(x + h * p.xh[which] + run0 * 8);
          b[u] = load16_stream(x + h * p.xh[which] + run1 * 8);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = (i0 + u) * HPI + sub;
        turn_row<D, kPairs>(a[u], b[u], wp != nullptr, p.eps, turns_here, cs, sn, w_s + which * 4 * LPH + j,
                              i0 + u < i_hi && h < heads, y + h * p.yh[which], run0, run1);
      }
    }
  }
}

// The same for few heads: a warp takes 32 / LPH tokens, a row of each at a time, and every lane works out its own
// token's angles; a warp that took one token's heads side by side would leave lanes idle and spend most of its time on
// angles. q's and k's rows are dealt to different warps.
template <int D, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32, kCtas) rotate_tokens_kernel(const RotateParams p) {
  constexpr int LPH = D / 16, TPW = 32 / LPH;
  __shared__ float4 w_s[2 * 4 * LPH];
  pdl_wait();
  load_weights<LPH>(p, w_s);
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= p.n_items) return;
  const int64_t tok = item / p.parts * TPW + lane / LPH;
  const int part = static_cast<int>(item % p.parts);
  const bool live = tok < p.n_tok;
  const int which = part < p.parts_q ? 0 : 1, mine = which == 0 ? part : part - p.parts_q;
  const int of = which == 0 ? p.parts_q : p.parts - p.parts_q;
  const int lo = mine * p.heads[which] / of, hi = (mine + 1) * p.heads[which] / of;
  int run0, run1;
  const bool turns_here = runs_of<LPH>(lane % LPH, p.rot, run0, run1);
  const uint16_t* x = p.x[which] + tok * p.xt[which];
  uint16_t* y = p.y[which] + tok * p.yt[which];
  const int64_t xh = p.xh[which], yh = p.yh[which];
  uint4 a[kUnroll], b[kUnroll];
  auto request = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      a[u] = b[u] = make_uint4(0, 0, 0, 0);
      if (live && h0 + u < hi) {
        a[u] = load16_stream(x + (h0 + u) * xh + run0 * 8);
        b[u] = load16_stream(x + (h0 + u) * xh + run1 * 8);
      }
    }
  };
  request(lo);  // on their way while the angles are worked out
  const uint64_t pos = turns_here && live ? static_cast<uint64_t>(static_cast<int64_t>(p.pos[tok])) : 0;
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (turns_here) angle(p.turns, kPairs ? (e < 4 ? 4 * run0 + e : 4 * run1 + e - 4) : 8 * run0 + e, pos, cs[e], sn[e]);
  }
#pragma unroll 1
  for (int h0 = lo; h0 < hi; h0 += kUnroll) {
    if (h0 > lo) request(h0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      turn_row<D, kPairs>(a[u], b[u], p.w[which] != nullptr, p.eps, turns_here, cs, sn,
                          w_s + which * 4 * LPH + lane % LPH, live && h0 + u < hi, y + (h0 + u) * yh, run0, run1);
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" kvp_status kvp_rope_turns(int n, const double* inv_freq, uint64_t* turns) {
  if (n < 0) return KVP_ERR_INVALID;
  if (n == 0) return KVP_OK;
  if (inv_freq == nullptr || turns == nullptr) return KVP_ERR_INVALID;
  // 1 / (2 pi) as the sum of two doubles, and the quotient as the sum of two with it (the product's own rounding error by
  // a fused multiply-add): a position multiplies the quotient's error by up to 2^31, so one double's 2^-53 of it would
  // show at far positions. Below 2^32 radians the sum is within 2^-74 of a turn.
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57, kOne = 18446744073709551616.0;  // 2^64
  for (int i = 0; i < n; ++i) {
    const double f = std::fabs(inv_freq[i]);
    if (!(f <= 4294967296.0)) return KVP_ERR_INVALID;
    const double hi = f * kHi, lo = std::fma(f, kHi, -hi) + f * kLo;
    const double x = (hi - std::floor(hi)) * kOne, whole = std::floor(x);  // both exact
    const uint64_t u = static_cast<uint64_t>(whole) +
                       static_cast<uint64_t>(static_cast<int64_t>(std::floor(x - whole + lo * kOne + 0.5)));
    turns[i] = inv_freq[i] < 0 ? 0 - u : u;
  }
  return KVP_OK;
}

extern "C" kvp_status kvp_qk_norm_rope(int64_t n_tok, int n_q_heads, int n_k_heads, int head_dim, int rot_dim,
                                       int interleaved, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                                       const void* k, int64_t k_stride_t, int64_t k_stride_h, const int32_t* pos,
                                       const uint64_t* turns, const float* wq, const float* wk, float eps,
                                       void* q_out, int64_t qo_stride_t, int64_t qo_stride_h, void* k_out,
                                       int64_t ko_stride_t, int64_t ko_stride_h, void* stream) {
  if (n_tok < 0 || n_q_heads < 0 || n_k_heads < 0 || (n_q_heads == 0 && n_k_heads == 0)) return KVP_ERR_INVALID;
  if (!(eps >= 0.f) || eps > 3.402823466e38f) return KVP_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128) return KVP_ERR_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > head_dim) return KVP_ERR_INVALID;
  if (rot_dim % 16 != 0) return KVP_ERR_UNSUPPORTED;
  if (n_q_heads > 65536 || n_k_heads > 65536) return KVP_ERR_UNSUPPORTED;
  if (n_tok == 0) return KVP_OK;
  if (rot_dim > 0 && (pos == nullptr || turns == nullptr)) return KVP_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(pos) & 3u) != 0 || (reinterpret_cast<uintptr_t>(turns) & 7u) != 0)
    return KVP_ERR_ALIGN;
  RotateParams p;
  p.x[0] = static_cast<const uint16_t*>(q);
  p.x[1] = static_cast<const uint16_t*>(k);
  p.y[0] = static_cast<uint16_t*>(q_out);
  p.y[1] = static_cast<uint16_t*>(k_out);
  p.xt[0] = q_stride_t, p.xh[0] = q_stride_h, p.yt[0] = qo_stride_t, p.yh[0] = qo_stride_h;
  p.xt[1] = k_stride_t, p.xh[1] = k_stride_h, p.yt[1] = ko_stride_t, p.yh[1] = ko_stride_h;
  p.w[0] = wq;
  p.w[1] = wk;
  p.heads[0] = n_q_heads;
  p.heads[1] = n_k_heads;
  for (int i = 0; i < 2; ++i) {
    if (p.heads[i] == 0) continue;
    if (p.x[i] == nullptr || p.y[i] == nullptr) return KVP_ERR_INVALID;
    if (!al16(p.x[i]) || !al16(p.y[i]) || !al16(p.w[i])) return KVP_ERR_ALIGN;
    for (const int64_t s : {p.xt[i], p.xh[i], p.yt[i], p.yh[i]}) {
      if (s < 0) return KVP_ERR_INVALID;
      if (s % 8 != 0) return KVP_ERR_ALIGN;
    }
    if (!rows_apart({{{p.yt[i], n_tok}, {p.yh[i], p.heads[i]}, {0, 1}}}, head_dim)) return KVP_ERR_INVALID;
    if (p.x[i] == p.y[i] && ((n_tok > 1 && p.xt[i] != p.yt[i]) || (p.heads[i] > 1 && p.xh[i] != p.yh[i])))
      return KVP_ERR_INVALID;
  }
  p.pos = pos;
  p.turns = turns;
  p.rot = rot_dim;
  p.eps = eps;
  if (n_tok > 0x7fffffffll) return KVP_ERR_UNSUPPORTED;
  p.n_tok = n_tok;
  const int rows = 32 / (head_dim / 16);  // rows a warp takes at a time
  // Few tokens: their heads are dealt to more warps, until there are about 4,096 of them (27 for each SM) to hide the
  // loads' latency.
  const bool by_token = n_q_heads + n_k_heads <= kFewSteps * rows && n_tok * (n_q_heads + n_k_heads) >= 4096 * rows;
  if (by_token) {
    p.parts_q = n_q_heads > 0;
    p.parts = p.parts_q + (n_k_heads > 0);
    p.n_items = (n_tok + rows - 1) / rows * p.parts;
  } else {
    const int its = (n_q_heads + rows - 1) / rows + (n_k_heads + rows - 1) / rows;
    const int64_t parts = (4096 + n_tok - 1) / n_tok;
    p.parts = static_cast<int>(parts < its ? parts : its);
    p.parts_q = 0;
    p.n_items = n_tok * p.parts;
  }
  const int64_t ctas = (p.n_items + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), 0, static_cast<cudaStream_t>(stream),
                      p) == cudaSuccess
               ? KVP_OK
               : KVP_ERR_CUDA;
  };
  if (by_token) {
    if (head_dim == 128) return interleaved ? go(rotate_tokens_kernel<128, true>) : go(rotate_tokens_kernel<128, false>);
    return interleaved ? go(rotate_tokens_kernel<64, true>) : go(rotate_tokens_kernel<64, false>);
  }
  if (head_dim == 128) return interleaved ? go(rotate_kernel<128, true>) : go(rotate_kernel<128, false>);
  return interleaved ? go(rotate_kernel<64, true>) : go(rotate_kernel<64, false>);
}
