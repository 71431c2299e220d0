// kvp_prompt_attn, kvp_prompt_weights: causal attention over packed prompts,
// and the weight that every key received (DMS article, "DMS 작동 방식" step 5:
// the standard attention, here of a whole prompt).
//
// The simplest form of both: a warp a row, its lanes over the head's values, an
// online softmax key by key.
#include "kvp_common.cuh"

namespace kvp {
namespace {

constexpr int kTile = 128;       // rows of a sequence that a CTA takes
constexpr int kPWarps = 8;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
// A weight is held as 2^(x - reference - kHeadroom): sums of up to 2^20 values of any bf16 size (the reference may
// lag by 2^8) stay below 2^128 that way.
constexpr float kHeadroom = 28.f;

struct Seqs {
  const int32_t* start;
  const int32_t* len;
  int n;
  int64_t n_tok;
  int32_t* status;
};

struct PromptParams {
  Seqs seqs;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t qt, qh, kt, kh, vt, vh, ot, oh;
  int Hq, G;
  float qscale;   // scale * log2 e
  uint16_t* out;
  float* lse;
  // weights
  const float* lse_in;
  int n_last;
  float* acc;
  int64_t as, at, ah;
  int acc_len;
};

struct Tile {
  int seq, start, len, r;  // sequence, its first row and length, tile of it
};

// A sequence's rows; one that breaks the rules is recorded and has none.
KVP_DEV int seq_rows(const Seqs& s, int i, int& start) {
  start = s.start[i];
  const int end = s.start[i + 1];
  const int len = s.len != nullptr ? s.len[i] : end - start;
  if (start < 0 || end < start || end > s.n_tok || len < 0 || len > end - start) {
    record_error(s.status, KVP_ERR_BOUNDS);
    return 0;
  }
  return len;
}

// Tile number `idx` of all sequences' (a whole warp calls this); false past the last.
KVP_DEV bool find_tile(const Seqs& s, int idx, Tile& t) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < s.n; base += 32) {
    const int i = base + lane;
    int start = 0;
    const int len = i < s.n ? seq_rows(s, i, start) : 0;
    const int tiles = (len + kTile - 1) / kTile;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, idx < before + incl);
    if (hit != 0) {
      const int src = __ffs(hit) - 1;
      t.seq = base + src;
      t.start = __shfl_sync(0xffffffffu, start, src);
      t.len = __shfl_sync(0xffffffffu, len, src);
      t.r = idx - before - __shfl_sync(0xffffffffu, incl - tiles, src);
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

template <int D>
KVP_DEV void load_row(const uint16_t* p, float (&x)[D / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i * 32 + lane]) << 16);
}
template <int D>
KVP_DEV float dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D>
__global__ void __launch_bounds__(kPWarps * 32) prompt_attn_kernel(const PromptParams p) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.y, h = j / p.G;
  Tile t;
  if (!find_tile(p.seqs, blockIdx.x, t)) return;
  for (int r = t.r * kTile + warp; r < min(t.len, (t.r + 1) * kTile); r += kPWarps) {
    const int64_t row = t.start + r;
    float q[D / 32], o[D / 32] = {}, m = -INFINITY, l = 0.f;
    load_row<D>(p.q + row * p.qt + j * p.qh, q);
    for (int c = 0; c <= r; ++c) {
      float k[D / 32], v[D / 32];
      load_row<D>(p.k + (t.start + c) * p.kt + h * p.kh, k);
      load_row<D>(p.v + (t.start + c) * p.vt + h * p.vh, v);
      const float x = dot<D>(q, k) * p.qscale;
      const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn;
      const float al = exp2f(m - ref), w = exp2f(x - ref - kHeadroom);
      m = mn;
      l = l * al + w;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(w, v[i], o[i] * al);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      p.out[row * p.ot + j * p.oh + i * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
    if (p.lse != nullptr && lane == 0)
      p.lse[j * p.seqs.n_tok + row] = l == 0.f ? -INFINITY : (m + kHeadroom + log2f(l)) * kLn2;
  }
}

template <int D>
__global__ void __launch_bounds__(kPWarps * 32) prompt_weights_kernel(const PromptParams p) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  Tile t;
  if (!find_tile(p.seqs, blockIdx.x, t)) return;
  const int first = p.n_last > 0 ? max(0, t.len - p.n_last) : 0;
  for (int c = t.r * kTile + warp; c < min(t.len, (t.r + 1) * kTile); c += kPWarps) {
    float k[D / 32], total = 0.f;
    load_row<D>(p.k + (t.start + c) * p.kt + h * p.kh, k);
    for (int r0 = max(first, c) / kTile * kTile; r0 < t.len; r0 += kTile)
      for (int j = h * p.G; j < (h + 1) * p.G; ++j) {
        float part = 0.f;
        for (int r = max(r0, max(first, c)); r < min(t.len, r0 + kTile); ++r) {
          const int64_t row = t.start + r;
          float q[D / 32];
          load_row<D>(p.q + row * p.qt + j * p.qh, q);
          const float x = dot<D>(q, k) * p.qscale, lse = p.lse_in[j * p.seqs.n_tok + row];
          if (lse != -INFINITY) part += exp2f(x - lse * kLog2e);
        }
        total += part;
      }
    if (lane == 0) {
      if (p.as < 0) {
        p.acc[(t.start + c) * p.at + h * p.ah] = total;
      } else if (c < p.acc_len) {
        p.acc[t.seq * p.as + c * p.at + h * p.ah] = total;
      } else {
        record_error(p.seqs.status, KVP_ERR_BOUNDS);
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Strides of an input whose rows are read in place.
kvp_status check_rows(const void* p, int64_t n_tok, int64_t st, int heads, int64_t sh) {
  if (p == nullptr) return KVP_ERR_INVALID;
  if (st < 0 || sh < 0 || (n_tok > 1 && st == 0) || (heads > 1 && sh == 0)) return KVP_ERR_INVALID;
  if (!aligned16(p) || st % 8 != 0 || sh % 8 != 0) return KVP_ERR_ALIGN;
  if (st > (int64_t{1} << 38) || sh > (int64_t{1} << 38)) return KVP_ERR_UNSUPPORTED;
  return KVP_OK;
}

kvp_status check_prompt(int n_seqs, int64_t n_tok, int n_q_heads, int n_kv_heads, int head_dim,
                        const int32_t* seq_start, const int32_t* seq_len, float scale) {
  if (n_seqs < 0 || n_tok < 0 || n_q_heads <= 0 || n_kv_heads <= 0) return KVP_ERR_INVALID;
  if (!(scale >= 0.f) || scale > 3.402823466e38f) return KVP_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128) return KVP_ERR_UNSUPPORTED;
  if (n_q_heads % n_kv_heads != 0) return KVP_ERR_INVALID;
  if (n_q_heads > 65535 || n_tok > 0x7fffffffll) return KVP_ERR_UNSUPPORTED;
  if (n_seqs > 0 && n_tok > 0 && seq_start == nullptr) return KVP_ERR_INVALID;
  if (!aligned4(seq_start) || !aligned4(seq_len)) return KVP_ERR_ALIGN;
  return KVP_OK;
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" kvp_status kvp_prompt_attn(int n_seqs, int64_t n_tok, int n_q_heads, int n_kv_heads, int head_dim,
                                      const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                      int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                                      int64_t v_stride_h, const int32_t* seq_start, const int32_t* seq_len,
                                      float scale, void* out, int64_t out_stride_t, int64_t out_stride_h, float* lse,
                                      int32_t* status, void* stream) {
  kvp_status r = check_prompt(n_seqs, n_tok, n_q_heads, n_kv_heads, head_dim, seq_start, seq_len, scale);
  if (r != KVP_OK) return r;
  if (n_seqs == 0 || n_tok == 0) return KVP_OK;
  if ((r = check_rows(q, n_tok, q_stride_t, n_q_heads, q_stride_h)) != KVP_OK) return r;
  if ((r = check_rows(k, n_tok, k_stride_t, n_kv_heads, k_stride_h)) != KVP_OK) return r;
  if ((r = check_rows(v, n_tok, v_stride_t, n_kv_heads, v_stride_h)) != KVP_OK) return r;
  if ((r = check_rows(out, n_tok, out_stride_t, n_q_heads, out_stride_h)) != KVP_OK) return r;
  if (!rows_apart({{{out_stride_t, n_tok}, {out_stride_h, n_q_heads}, {0, 1}}}, head_dim)) return KVP_ERR_INVALID;
  if (!aligned4(lse)) return KVP_ERR_ALIGN;
  PromptParams p{};
  p.seqs = Seqs{seq_start, seq_len, n_seqs, n_tok, status};
  p.q = static_cast<const uint16_t*>(q), p.qt = q_stride_t, p.qh = q_stride_h;
  p.k = static_cast<const uint16_t*>(k), p.kt = k_stride_t, p.kh = k_stride_h;
  p.v = static_cast<const uint16_t*>(v), p.vt = v_stride_t, p.vh = v_stride_h;
  p.out = static_cast<uint16_t*>(out), p.ot = out_stride_t, p.oh = out_stride_h;
  p.Hq = n_q_heads, p.G = n_q_heads / n_kv_heads;
  p.qscale = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(head_dim))) * kLog2e;
  p.lse = lse;
  const int64_t tiles = n_tok / kTile + n_seqs;
  if (tiles > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(n_q_heads));
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(kPWarps * 32), 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess
               ? KVP_OK
               : KVP_ERR_CUDA;
  };
  return head_dim == 128 ? go(prompt_attn_kernel<128>) : go(prompt_attn_kernel<64>);
}

extern "C" kvp_status kvp_prompt_weights(int n_seqs, int64_t n_tok, int n_q_heads, int n_kv_heads, int head_dim,
                                         const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k,
                                         int64_t k_stride_t, int64_t k_stride_h, const int32_t* seq_start,
                                         const int32_t* seq_len, const float* lse, float scale, int n_last, float* acc,
                                         int64_t acc_stride_s, int64_t acc_stride_t, int64_t acc_stride_h, int acc_len,
                                         int32_t* status, void* stream) {
  kvp_status r = check_prompt(n_seqs, n_tok, n_q_heads, n_kv_heads, head_dim, seq_start, seq_len, scale);
  if (r != KVP_OK) return r;
  if (n_last < 0 || acc_stride_s < -1 || acc_stride_t < 0 || acc_stride_h < 0) return KVP_ERR_INVALID;
  if (acc_stride_s >= 0 && acc_len < 0) return KVP_ERR_INVALID;
  if (n_seqs == 0 || n_tok == 0) return KVP_OK;
  if ((r = check_rows(q, n_tok, q_stride_t, n_q_heads, q_stride_h)) != KVP_OK) return r;
  if ((r = check_rows(k, n_tok, k_stride_t, n_kv_heads, k_stride_h)) != KVP_OK) return r;
  if (lse == nullptr || acc == nullptr) return KVP_ERR_INVALID;
  if (!aligned4(lse) || !aligned4(acc)) return KVP_ERR_ALIGN;
  const bool by_token = acc_stride_s < 0;
  if (!rows_apart({{{by_token ? 0 : acc_stride_s, by_token ? 1 : n_seqs},
                    {acc_stride_t, by_token ? n_tok : acc_len},
                    {acc_stride_h, n_kv_heads}}},
                  1))
    return KVP_ERR_INVALID;
  PromptParams p{};
  p.seqs = Seqs{seq_start, seq_len, n_seqs, n_tok, status};
  p.q = static_cast<const uint16_t*>(q), p.qt = q_stride_t, p.qh = q_stride_h;
  p.k = static_cast<const uint16_t*>(k), p.kt = k_stride_t, p.kh = k_stride_h;
  p.Hq = n_q_heads, p.G = n_q_heads / n_kv_heads;
  p.qscale = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(head_dim))) * kLog2e;
  p.lse_in = lse;
  p.n_last = n_last;
  p.acc = acc, p.as = acc_stride_s, p.at = acc_stride_t, p.ah = acc_stride_h, p.acc_len = acc_len;
  const int64_t tiles = n_tok / kTile + n_seqs;
  if (tiles > 0x7fffffff) return KVP_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(n_kv_heads));
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(kPWarps * 32), 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess
               ? KVP_OK
               : KVP_ERR_CUDA;
  };
  return head_dim == 128 ? go(prompt_weights_kernel<128>) : go(prompt_weights_kernel<64>);
}
