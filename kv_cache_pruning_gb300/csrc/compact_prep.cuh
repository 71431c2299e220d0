// What the compactions share: the keep rules, the masked dense source, and the
// preparation passes (entry counts per segment and (b, h), page bases), each
// translation unit with its own copies.
#pragma once

#include "kvp_common.cuh"

namespace kvp {
namespace {

constexpr int kSeg = 128;           // entries per warp segment
constexpr int kWarpsPerCta = 4;     // segments per CTA in the count and copy passes

KVP_DEV int32_t expire_kvzap(float s, float tau, int pos, int window) {
  return (s >= tau) ? kNever : pos + window;  // NaN compares false: treated as low
}
KVP_DEV int32_t expire_dms(int flag, int pos, int delay, int window) {
  return flag < 0 ? kNever : max(flag + delay, pos + window);
}

// Masked dense source: the same rows as DenseSrc, but each entry's expire is
// derived where it is needed from its score and the (b, h)'s threshold (KVzap)
// or its flag step (DMS), with the mask kernel's rule and position t, so that
// no [B, H, n] expire array is written or read.
struct MaskedSrc {
  const uint16_t* k;
  const uint16_t* v;
  int64_t sb, st, sh;
  int mode;
  const float* scores;     // KVzap: [B, n, H]
  const float* tau;        // KVzap: [B, H]
  const int32_t* flag;     // DMS: [B, H, n]
  int window, delay;
  int H;
  int n;
  struct View {
    const uint16_t* kb;
    const uint16_t* vb;
    int64_t stride;
    int mode;
    const float* sc;       // this (b, h)'s scores, entry t at sc[t * H]
    const int32_t* fl;     // this (b, h)'s flag steps, entry t at fl[t]
    float th;
    int H, window, delay, n;
    KVP_DEV int length() const { return n; }
    KVP_DEV int32_t expire_row(int t, int64_t& row) const {
      row = t;
      return mode == KVP_MASK_KVZAP ? expire_kvzap(sc[static_cast<int64_t>(t) * H], th, t, window)
                                    : expire_dms(fl[t], t, delay, window);
    }
    KVP_DEV int position_of(int t) const { return t; }
    KVP_DEV bool keep(int32_t e, int now) const { return now < e; }
  };
  KVP_DEV View view(int bh) const {
    const int b = bh / H, h = bh - b * H;
    const int64_t off = b * sb + h * sh;
    const bool kvz = mode == KVP_MASK_KVZAP;
    return View{k + off,
                v + off,
                st,
                mode,
                kvz ? scores + static_cast<int64_t>(b) * n * H + h : nullptr,
                kvz ? nullptr : flag + static_cast<int64_t>(bh) * n,
                kvz ? tau[bh] : 0.f,
                H,
                window,
                delay,
                n};
  }
};

// Workspace layout (int32): segment counts [BH*NS], a second [BH*NS] block
// (the block-scaled write's sums of several segments), page base [BH], flag [1] (1 = budget ok);
// base and flag are used only above kFusedBH pairs.
struct CompactWs {
  int32_t* seg_cnt;
  int32_t* seg_off;
  int32_t* base;
  int32_t* ok;
};
size_t compact_ws_bytes(int64_t BH, int NS) { return (static_cast<size_t>(2) * BH * NS + BH + 1) * sizeof(int32_t); }
// (b, h) pairs a compaction takes: the count pass puts them on the grid's y
// dimension.
constexpr int64_t kMaxCompactBH = 65535;
CompactWs carve(void* ws, int BH, int NS) {
  int32_t* p = static_cast<int32_t*>(ws);
  const size_t n = static_cast<size_t>(BH) * NS;
  return CompactWs{p, p + n, p + 2 * n, p + 2 * n + BH};
}
int n_segments(int n) { return n > 0 ? (n + kSeg - 1) / kSeg : 1; }

// Preparation: present entries per segment (one warp each); the CTA's
// segments (all of one (b, h)) are summed and added to the (b, h)'s count
// with one atomic.
template <class Src>
__global__ void __launch_bounds__(kWarpsPerCta * 32) count_kernel(Src src, int now, int NS,
                                                                   int32_t* __restrict__ seg_cnt,
                                                                   int32_t* __restrict__ count) {
  __shared__ int cta_kept[kWarpsPerCta];
  pdl_launch_dependents();  // the copy pass may be scheduled now; it waits for this grid's end
  const int bh = blockIdx.y;
  const int warp = threadIdx.x >> 5;
  const int sg = blockIdx.x * kWarpsPerCta + warp;
  const int lane = threadIdx.x & 31;
  int kept = 0;
  if (sg < NS) {
    const auto sv = src.view(bh);
    const int lo = sg * kSeg, hi = min(lo + kSeg, sv.length());
#pragma unroll
    for (int u = 0; u < kSeg / 32; ++u) {  // independent loads, all in flight together
      const int t = lo + u * 32 + lane;
      if (t < hi) {
        int64_t row;
        const int32_t e = sv.expire_row(t, row);
        kept += (row >= 0 && sv.keep(e, now));
      }
    }
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 0) seg_cnt[static_cast<int64_t>(bh) * NS + sg] = kept;
  }
  if (lane == 0) cta_kept[warp] = kept;
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWarpsPerCta; ++w) t += cta_kept[w];
    if (t) atomicAdd(&count[bh], t);  // count was zeroed before this kernel
  }
}

// Page bases for B*H above kFusedBH (one CTA): bases in (b-major, h-minor)
// order and the budget checks. Up to kFusedBH pairs every copy-pass CTA
// derives its own base and the checks from the counts instead.
constexpr int kFusedBH = 1024;

__global__ void __launch_bounds__(1024) base_kernel(int BH, int reserve, int max_pages, int n_pages_cap,
                                                    CompactWs ws, const int32_t* __restrict__ count,
                                                    int32_t* __restrict__ status) {
  __shared__ int warp_tot[32];
  __shared__ int carry_s;
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    carry_s = 0;
    bad_s = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < BH; b0 += 1024) {
    const int bh = b0 + tid;
    int pages = 0;
    if (bh < BH) {
      pages = (count[bh] + reserve + kPage - 1) / kPage;
      if (pages > max_pages) atomicExch(&bad_s, 1);
    }
    int incl = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int wt = warp_tot[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, wt, o);
        if (lane >= o) wt += y;
      }
      warp_tot[lane] = wt;  // inclusive over warps
    }
    __syncthreads();
    const int before = (warp > 0 ? warp_tot[warp - 1] : 0) + incl - pages;
    const int carry = carry_s;
    if (bh < BH) ws.base[bh] = carry + before;
    __syncthreads();
    if (tid == 0) carry_s = carry + warp_tot[31];
    __syncthreads();
  }
  if (tid == 0) {
    const bool ok = !bad_s && carry_s <= n_pages_cap;
    ws.ok[0] = ok ? 1 : 0;
    if (!ok) record_error(status, KVP_ERR_CAPACITY);
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace kvp
