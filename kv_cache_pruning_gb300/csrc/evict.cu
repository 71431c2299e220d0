// kvp_evict, kvp_evict_paged: which entries stay within a budget, by the
// attention weight that they have received.
//
// Of one (b, h) with n entries: the recent ones stay; of the c others the
// m = min(c, max(0, budget - recent ones)) heaviest, the first of equal ones.
// With order-preserving 32-bit keys (-0 = 0, NaN lowest) the m-th largest key T
// is found by radix selection, 8 bits a pass from the top, and the entries kept
// are those above T and the first m - #{> T} of those equal to it.
#include "kvp_common.cuh"

namespace kvp {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;

enum Kind { kAbsent = 0, kRecent = 1, kCandidate = 2 };

// fp32 to a key whose unsigned order is the values': NaN 0, -inf 0x007fffff, zeros 0x80000000.
KVP_DEV uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u ^ ((u >> 31) != 0u ? 0xFFFFFFFFu : 0x80000000u);
}

struct DenseEvict {
  const float* acc;
  int64_t stride_b, stride_t, stride_h;
  int H, n_pos, recent, now;
  int32_t* expire;
  int32_t* kept;
  const float* row;
  int32_t* out;
  KVP_DEV void open(int bh, int /*now*/) {
    row = acc + (bh / H) * stride_b + (bh % H) * stride_h;
    out = expire + static_cast<int64_t>(bh) * n_pos;
  }
  KVP_DEV int size() const { return n_pos; }
  KVP_DEV Kind get(int i, uint32_t& key) const {
    if (i > static_cast<int64_t>(now) - recent) return kRecent;
    key = weight_key(row[i * stride_t]);
    return kCandidate;
  }
  KVP_DEV void put(int i, bool stays) const { out[i] = stays ? kNever : now; }
};

struct PagedEvict {
  const float* acc;
  int64_t stride_b, stride_h;
  int acc_len, H;
  int32_t* expire_pool;
  int n_pages_cap, max_pages;
  const int32_t* page_table;
  const int32_t* remap;
  const int32_t* count;
  int recent, now;
  const int32_t* now_dev;
  int32_t* kept;
  int32_t* status;
  const float* row;
  const int32_t* pages;
  const int32_t* pos;
  int n;
  KVP_DEV void open(int bh, int step) {
    now = step;
    row = acc + (bh / H) * stride_b + (bh % H) * stride_h;
    pages = page_table + static_cast<int64_t>(bh) * max_pages;
    pos = remap + static_cast<int64_t>(bh) * max_pages * kPage;
    n = min(max(count[bh], 0), max_pages * kPage);
  }
  KVP_DEV int size() const { return n; }
  KVP_DEV Kind get(int i, uint32_t& key) const {
    const int page = pages[i / kPage];
    if (page < 0 || page >= n_pages_cap) {
      record_error(status, KVP_ERR_BOUNDS);
      return kAbsent;
    }
    if (expire_pool[static_cast<int64_t>(page) * kPage + i % kPage] <= now) return kAbsent;
    const int at = pos[i];
    if (at < 0 || at >= acc_len) {
      record_error(status, KVP_ERR_BOUNDS);
      return kAbsent;
    }
    if (at > static_cast<int64_t>(now) - recent) return kRecent;
    key = weight_key(row[at]);
    return kCandidate;
  }
  KVP_DEV void put(int i, bool stays) const {
    if (!stays) expire_pool[static_cast<int64_t>(pages[i / kPage]) * kPage + i % kPage] = now;
  }
};

// One CTA a (b, h), every pass over its entries from memory.
template <class Src>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(Src src, int budget, const int32_t* now_dev, int now,
                                                             int32_t* kept, int32_t* status) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sum[kEvictWarps];
  __shared__ uint32_t s_recent, s_cand, s_digit, s_left;
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x;
  if (now_dev != nullptr) {
    now = *now_dev;
    if (now < 0 || now == kNever) {
      if (tid == 0) record_error(status, KVP_ERR_INVALID);
      return;
    }
  }
  src.open(bh, now);
  const int n = src.size();
  uint32_t prefix = 0, mask = 0, left = 0;
  if (tid == 0) s_recent = s_cand = 0;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
    uint32_t recent = 0, cand = 0;
    for (int i = tid; i < n; i += kEvictThreads) {
      uint32_t key = 0;
      const Kind kind = src.get(i, key);
      recent += kind == kRecent;
      if (kind != kCandidate) continue;
      ++cand;
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    if (pass == 0) {
      atomicAdd(&s_recent, recent);
      atomicAdd(&s_cand, cand);
    }
    __syncthreads();
    if (pass == 0) left = min(s_cand, static_cast<uint32_t>(max(budget - static_cast<int64_t>(s_recent), int64_t{0})));
    if (left == 0 || (pass == 0 && left == s_cand)) break;  // none or all of the others stay
    if (tid == 0) {
      uint32_t above = 0;
      int d = 255;
      while (above + hist[d] < left) above += hist[d--];
      s_digit = d;
      s_left = left - above;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    left = s_left;
  }
  const uint32_t m = min(s_cand, static_cast<uint32_t>(max(budget - static_cast<int64_t>(s_recent), int64_t{0})));
  const bool all = m == s_cand, none = m == 0;
  uint32_t before = 0;  // entries equal to the key so far, in order
  for (int base = 0; base < n; base += kEvictThreads) {
    const int i = base + tid;
    uint32_t key = 0;
    const Kind kind = i < n ? src.get(i, key) : kAbsent;
    const bool eq = kind == kCandidate && key == prefix;
    const uint32_t bits = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) warp_sum[warp] = __popc(bits);
    __syncthreads();
    uint32_t rank = before + __popc(bits & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < kEvictWarps; ++w) {
      if (w < warp) rank += warp_sum[w];
      total += warp_sum[w];
    }
    before += total;
    __syncthreads();
    const bool stays = kind == kRecent || all || (!none && (key > prefix || (eq && rank < left)));
    if (kind != kAbsent) src.put(i, stays);
  }
  if (kept != nullptr && tid == 0) kept[bh] = static_cast<int32_t>(s_recent + m);
}

kvp_status evict_paged_impl(int batch, int n_kv_heads, const float* acc, int64_t acc_stride_b, int64_t acc_stride_h,
                            int acc_len, int32_t* expire_pool, int n_pages_cap, const int32_t* page_table,
                            int max_pages, const int32_t* remap, const int32_t* count, int budget, int recent, int now,
                            const int32_t* now_dev, int32_t* kept, int32_t* status, void* stream) {
  if (batch <= 0 || n_kv_heads <= 0 || max_pages < 0 || n_pages_cap < 0 || acc_len < 0 || acc_stride_b < 0 ||
      acc_stride_h < 0 || budget < 0 || recent < 0 || now < 0 || now == kNever)
    return KVP_ERR_INVALID;
  if (acc == nullptr || expire_pool == nullptr || page_table == nullptr || remap == nullptr || count == nullptr)
    return KVP_ERR_INVALID;
  for (const void* x : {static_cast<const void*>(acc), static_cast<const void*>(expire_pool),
                        static_cast<const void*>(page_table), static_cast<const void*>(remap),
                        static_cast<const void*>(count), static_cast<const void*>(now_dev),
                        static_cast<const void*>(kept)})
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return KVP_ERR_ALIGN;
  const int64_t BH = static_cast<int64_t>(batch) * n_kv_heads;
  if (BH > (1 << 24) || static_cast<int64_t>(max_pages) * kPage > 0x7fff0000) return KVP_ERR_UNSUPPORTED;
  const PagedEvict src{acc,   acc_stride_b, acc_stride_h, acc_len, n_kv_heads, expire_pool, n_pages_cap, max_pages,
                       page_table, remap, count, recent, now, now_dev, kept, status, nullptr, nullptr, nullptr, 0};
  return launch_pdl(evict_kernel<PagedEvict>, dim3(static_cast<unsigned>(BH)), dim3(kEvictThreads), 0,
                    static_cast<cudaStream_t>(stream), src, budget, now_dev, now, kept, status) == cudaSuccess
             ? KVP_OK
             : KVP_ERR_CUDA;
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" kvp_status kvp_evict(int batch, int n_kv_heads, int n_pos, const float* acc, int64_t stride_b,
                                int64_t stride_t, int64_t stride_h, int budget, int recent, int now, int32_t* expire,
                                int32_t* count, void* stream) {
  if (batch <= 0 || n_kv_heads <= 0 || n_pos < 0 || stride_b < 0 || stride_t < 0 || stride_h < 0 || budget < 0 ||
      recent < 0 || now < 0 || now == kNever)
    return KVP_ERR_INVALID;
  if (n_pos > 0 && (acc == nullptr || expire == nullptr)) return KVP_ERR_INVALID;
  for (const void* x :
       {static_cast<const void*>(acc), static_cast<const void*>(expire), static_cast<const void*>(count)})
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return KVP_ERR_ALIGN;
  const int64_t BH = static_cast<int64_t>(batch) * n_kv_heads;
  if (BH > (1 << 24) || n_pos > 0x7fff0000) return KVP_ERR_UNSUPPORTED;
  const DenseEvict src{acc, stride_b, stride_t, stride_h, n_kv_heads, n_pos, recent, now, expire, count, nullptr, nullptr};
  return launch_pdl(evict_kernel<DenseEvict>, dim3(static_cast<unsigned>(BH)), dim3(kEvictThreads), 0,
                    static_cast<cudaStream_t>(stream), src, budget, nullptr, now, count,
                    static_cast<int32_t*>(nullptr)) == cudaSuccess
             ? KVP_OK
             : KVP_ERR_CUDA;
}

extern "C" kvp_status kvp_evict_paged(int batch, int n_kv_heads, const float* acc, int64_t acc_stride_b,
                                      int64_t acc_stride_h, int acc_len, int32_t* expire_pool, int n_pages_cap,
                                      const int32_t* page_table, int max_pages, const int32_t* remap,
                                      const int32_t* count, int budget, int recent, int now, int32_t* kept,
                                      int32_t* status, void* stream) {
  return evict_paged_impl(batch, n_kv_heads, acc, acc_stride_b, acc_stride_h, acc_len, expire_pool, n_pages_cap,
                          page_table, max_pages, remap, count, budget, recent, now, nullptr, kept, status, stream);
}

extern "C" kvp_status kvp_evict_paged_devpos(int batch, int n_kv_heads, const float* acc, int64_t acc_stride_b,
                                             int64_t acc_stride_h, int acc_len, int32_t* expire_pool, int n_pages_cap,
                                             const int32_t* page_table, int max_pages, const int32_t* remap,
                                             const int32_t* count, int budget, int recent, const int32_t* now_dev,
                                             int32_t* kept, int32_t* status, void* stream) {
  if (now_dev == nullptr) return KVP_ERR_INVALID;
  return evict_paged_impl(batch, n_kv_heads, acc, acc_stride_b, acc_stride_h, acc_len, expire_pool, n_pages_cap,
                          page_table, max_pages, remap, count, budget, recent, 0, now_dev, kept, status, stream);
}
