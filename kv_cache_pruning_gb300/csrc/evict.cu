// kvp_evict, kvp_evict_paged: which entries stay within a budget, by the
// attention weight that they have received.
//
// Of one (b, h) with n entries: the recent ones stay; of the c others (the
// candidates) the m = min(c, max(0, budget - recent ones)) heaviest, the first of
// equal ones. With order-preserving 32-bit keys (-0 = 0, NaN lowest) the m-th
// largest key T is found by radix selection, 11, 11 and 10 bits from the top, and
// the entries kept are those above T and the first m - #{> T} of those equal to it.
//
// A cluster of CTAs takes a (b, h), each a run of its entries. Each pass counts into
// a histogram of each CTA, and after a cluster barrier every CTA adds them all up
// (through distributed shared memory) and comes to the same digit. How many entries
// equal to T the CTAs before it have is in their last histograms. A thread takes
// four entries at a time, with 16-byte loads and stores where they lie side by side.
//
// Bound: the weights read and the expire values written, 8 bytes an entry; what it takes is
// the passes' latencies, one after the other (131,072 x 64 weights: 29 us, of them 11 for
// the first pass; issue slots 41 % used). Keys of runs up to 8,192 are kept in shared memory
// (a paged cache's entry is three dependent loads). Those of longer runs are made again from
// what L2 holds, but for the keys with the first digit, which the second pass lists: with the
// room that all would take only half as many CTAs run at once (67 us with all keys kept).
// Loads of two steps are under way at once: of four, 27.6 us there but 4 % more at runs of
// 2,048 and 10,007; of one, 32 us.
#include "kvp_common.cuh"

namespace kvp {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048;                 // 11 bits
constexpr int kKeysCap = 8192;              // keys that a CTA keeps (32 KB)
constexpr int kListCap = 4096;              // of longer runs: keys with the first pass's digit (16 KB)
constexpr int kStep = 4 * kEvictThreads;    // entries of a step of the block's threads, four each
constexpr int kBatch = 2;                   // steps whose loads a thread has under way
constexpr uint32_t kNoKey = 0xFFFFFFFFu;    // not a candidate: above the key of any weight, and of a first digit of its own

// fp32 to a key whose unsigned order is the values': -inf 0x00800000, zeros 0x80000001, inf 0xff800001, and NaN, which
// the sum makes 0x7fffffff whatever its bits were, 0.
KVP_DEV uint32_t weight_key(float x) {
  const int32_t u = __float_as_int(x + 0.f);  // -0 becomes 0
  return (static_cast<uint32_t>(u) ^ (static_cast<uint32_t>(u >> 31) | 0x80000000u)) + 1u;
}

// The entries of a prompt: positions 0 .. n_pos - 1, the recent ones last.
struct DenseEvict {
  static constexpr bool kExact = true;   // size() is what the call names
  const float* acc;
  int64_t stride_b, stride_t, stride_h;
  int H, n_pos, recent, now;
  int32_t* expire;
  const float* row;
  int32_t* out;
  int old;  // entries that are not recent
  bool loads4, stores4;
  KVP_DEV void open(int bh, int /*step*/) {
    row = acc + (bh / H) * stride_b + (bh % H) * stride_h;
    out = expire + static_cast<int64_t>(bh) * n_pos;
    old = static_cast<int>(min(static_cast<int64_t>(n_pos), max(int64_t{0}, static_cast<int64_t>(now) - recent + 1)));
    loads4 = stride_t == 1 && (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    stores4 = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
  }
  KVP_DEV int size() const { return n_pos; }
  // keys of entries i .. i + 3 (i a multiple of 4; those from e on: kNoKey), and how many of them are recent
  KVP_DEV uint32_t keys4(int i, int e, uint32_t (&k)[4]) const {
    const int end = min(old, e);
    if (loads4 && i + 4 <= end) {
      const float4 w = *reinterpret_cast<const float4*>(row + i);
      k[0] = weight_key(w.x), k[1] = weight_key(w.y), k[2] = weight_key(w.z), k[3] = weight_key(w.w);
      return 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = i + j < end ? weight_key(row[(i + j) * stride_t]) : kNoKey;
    return max(0, min(i + 4, e) - max(i, end));
  }
  // the same for entries base + u kStep + 4 thread .. + 3 of each u, loads before what uses them
  KVP_DEV uint32_t keys_of(int base, int tid, int e, uint32_t (&k)[kBatch][4]) const {
    uint32_t recents = 0;
    if (loads4 && base + kBatch * kStep <= min(old, e)) {  // the whole block
      float4 w[kBatch];
      const float4* at = reinterpret_cast<const float4*>(row + base) + tid;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) w[u] = at[u * (kStep / 4)];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        k[u][0] = weight_key(w[u].x), k[u][1] = weight_key(w[u].y);
        k[u][2] = weight_key(w[u].z), k[u][3] = weight_key(w[u].w);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) recents += keys4(base + u * kStep + 4 * tid, e, k[u]);
    }
    return recents;
  }
  KVP_DEV void put4(int i, int e, const bool (&stays)[4]) const {
    if (i >= e) return;
    int32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = stays[j] ? kNever : now;
    if (stores4 && i + 4 <= e) {
      *reinterpret_cast<int4*>(out + i) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < e) out[i + j] = v[j];
    }
  }
};

// The present slots of a paged cache.
struct PagedEvict {
  static constexpr bool kExact = false;  // ... or less
  const float* acc;
  int64_t stride_b, stride_h;
  int acc_len, H;
  int32_t* expire_pool;
  int n_pages_cap, max_pages;
  const int32_t* page_table;
  const int32_t* remap;
  const int32_t* count;
  int recent, now;
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
  // (four slots of one page: i is a multiple of 4)
  KVP_DEV uint32_t keys4(int i, int e, uint32_t (&k)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = kNoKey;
    if (i >= e) return 0;
    const int page = pages[i / kPage];
    if (page < 0 || page >= n_pages_cap) {
      record_error(status, KVP_ERR_BOUNDS);
      return 0;
    }
    const int32_t* gone = expire_pool + static_cast<int64_t>(page) * kPage + i % kPage;
    int at[4], until[4];
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at[j] = i + j < e ? pos[i + j] : -1;
      until[j] = i + j < e ? gone[j] : INT32_MIN;
    }
    // (the weights are asked for beside the expire values: most slots are present)
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = at[j] >= 0 && at[j] < acc_len ? row[at[j]] : 0.f;
    uint32_t recents = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (until[j] <= now) continue;
      if (at[j] < 0 || at[j] >= acc_len) {
        record_error(status, KVP_ERR_BOUNDS);
      } else if (at[j] > static_cast<int64_t>(now) - recent) {
        ++recents;
      } else {
        k[j] = weight_key(w[j]);
      }
    }
    return recents;
  }
  KVP_DEV uint32_t keys_of(int base, int tid, int e, uint32_t (&k)[kBatch][4]) const {
    uint32_t recents = 0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) recents += keys4(base + u * kStep + 4 * tid, e, k[u]);
    return recents;
  }
  KVP_DEV void put4(int i, int /*e*/, const bool (&stays)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!stays[j])
        expire_pool[static_cast<int64_t>(pages[i / kPage]) * kPage + i % kPage + j] = now;
  }
};

// The word at `local`'s offset in the shared memory of CTA `rank` of the cluster.
KVP_DEV uint32_t cluster_address(const void* local, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  return r;
}
KVP_DEV uint4 load_cluster4(uint32_t address) {
  uint4 r;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(address)
               : "memory");
  return r;
}
KVP_DEV uint32_t load_cluster(uint32_t address) {
  uint32_t r;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(address) : "memory");
  return r;
}

struct EvictShared {
  uint32_t hist[3][kBins];        // one a pass: no CTA clears what another may still read
  uint32_t recent;
  uint32_t warp_sum[kEvictWarps];
  uint32_t digit, left, equal, before;
  uint32_t listed;                // keys on the list (or more: then it is not used)
};

template <class Src>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(Src src, int cluster, int budget, const int32_t* now_dev,
                                                             int now, int32_t* kept, int32_t* status) {
  extern __shared__ uint4 evict_smem[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(evict_smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(evict_smem + (sizeof(EvictShared) + 15) / 16);
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  if (now_dev != nullptr) {
    now = *now_dev;
    if (now < 0 || now == kNever) {  // the whole grid
      if (tid == 0) record_error(status, KVP_ERR_INVALID);
      return;
    }
  }
  for (int i = tid; i < 3 * kBins; i += kEvictThreads) sh.hist[0][i] = 0;
  if (tid == 0) sh.recent = sh.listed = 0;
  src.open(bh, now);
  const int n = src.size();
  // this CTA's run of entries, in multiples of 32
  const int run = static_cast<int>((static_cast<int64_t>(n) + 32 * cluster - 1) / (32 * cluster)) * 32;
  const int e0 = min(static_cast<int64_t>(n), static_cast<int64_t>(rank) * run), e1 = min(n - e0, run) + e0;
  const bool cached = run <= kKeysCap;
  __syncthreads();

  auto kept_keys = [&](int base, uint32_t (&k)[kBatch][4]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * kStep + 4 * tid;
      uint4 v = make_uint4(kNoKey, kNoKey, kNoKey, kNoKey);
      if (i < e1) v = *reinterpret_cast<const uint4*>(keys + (i - e0));
      k[u][0] = v.x, k[u][1] = v.y, k[u][2] = v.z, k[u][3] = v.w;
    }
  };
  uint32_t prefix = 0, mask = 0, left = 0, m = 0, cand = 0, recents = 0, before = 0;
  bool all = false;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : kBins;
    uint32_t mine = 0;
    if (pass == 1 && !cached) {  // the keys with the first digit, as many as there is room for
      for (int base = e0; base < e1; base += kBatch * kStep) {
        uint32_t k[kBatch][4], hits = 0;
        (void)src.keys_of(base, tid, e1, k);
#pragma unroll
        for (int j = 0; j < 4 * kBatch; ++j)
          if (((k[j / 4][j % 4] ^ prefix) & mask) == 0) hits |= 1u << j;
        if (hits == 0) continue;
        uint32_t at = atomicAdd(&sh.listed, static_cast<uint32_t>(__popc(hits)));
        for (; hits != 0 && at < kListCap; hits &= hits - 1) {  // (few: read once more rather than picked from registers)
          const int j = __ffs(hits) - 1;
          uint32_t again[4];
          (void)src.keys4(base + j / 4 * kStep + 4 * tid, e1, again);
          keys[at++] = (j & 2) != 0 ? (j & 1) != 0 ? again[3] : again[2] : (j & 1) != 0 ? again[1] : again[0];
        }
      }
      __syncthreads();
    }
    if (pass > 0 && !cached && sh.listed <= kListCap) {
      for (uint32_t i = tid; i < sh.listed; i += kEvictThreads)
        if (((keys[i] ^ prefix) & mask) == 0) atomicAdd(&sh.hist[pass][(keys[i] >> shift) & (bins - 1)], 1u);
    } else {
      for (int base = e0; base < e1; base += kBatch * kStep) {
        uint32_t k[kBatch][4];
        if (pass == 0 || !cached) mine += src.keys_of(base, tid, e1, k);
        else kept_keys(base, k);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = base + u * kStep + 4 * tid;
          if (base + u * kStep >= e1) break;
          if (pass == 0) {
            if (cached && i < e1)
              *reinterpret_cast<uint4*>(keys + (i - e0)) = make_uint4(k[u][0], k[u][1], k[u][2], k[u][3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) atomicAdd(&sh.hist[0][k[u][j] >> 21], 1u);
            continue;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (((k[u][j] ^ prefix) & mask) == 0) atomicAdd(&sh.hist[pass][(k[u][j] >> shift) & (bins - 1)], 1u);
        }
      }
    }
    if (pass == 0) {
      mine = __reduce_add_sync(0xffffffffu, mine);
      if (lane == 0 && mine != 0) atomicAdd(&sh.recent, mine);
    }
    if (cluster > 1) cluster_sync(); else __syncthreads();
    // all CTAs' counts of bins 4 tid ..
    uint32_t c[4] = {0, 0, 0, 0}, equal_before[4] = {0, 0, 0, 0};
    if (4u * tid < bins) {
      for (int r = 0; r < cluster; ++r) {
        const uint4 v = cluster > 1 ? load_cluster4(cluster_address(&sh.hist[pass][4 * tid], r))
                                    : *reinterpret_cast<const uint4*>(&sh.hist[pass][4 * tid]);
        c[0] += v.x, c[1] += v.y, c[2] += v.z, c[3] += v.w;
        if (r < rank) equal_before[0] += v.x, equal_before[1] += v.y, equal_before[2] += v.z, equal_before[3] += v.w;
      }
    }
    if (pass == 0 && tid == kBins / 4 - 1) c[3] = 0;  // kNoKey's
    // entries in this thread's bins and in all above: a scan over the threads from the last to the first
    const uint32_t own = c[0] + c[1] + c[2] + c[3];
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_down_sync(0xffffffffu, incl, o);
      if (lane + o < 32) incl += y;
    }
    if (lane == 0) sh.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t total = 0;
    for (int w = 0; w < kEvictWarps; ++w) {
      const uint32_t s = sh.warp_sum[w];
      if (w > warp) incl += s;
      total += s;
    }
    if (pass == 0) {
      for (int r = 0; r < cluster; ++r)
        recents += cluster > 1 ? load_cluster(cluster_address(&sh.recent, r)) : sh.recent;
      cand = total;
      const int64_t room = static_cast<int64_t>(budget) - recents;
      m = room <= 0 ? 0u : room < cand ? static_cast<uint32_t>(room) : cand;
      left = m;
      all = m == cand;
      if (m == 0 || all) break;  // none or all of the candidates stay
    }
    uint32_t above = incl - own;
    if (above < left && incl >= left) {
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        if (above < left && above + c[k] >= left) {
          sh.digit = 4 * tid + k;
          sh.left = left - above;
          sh.equal = c[k];
          sh.before = equal_before[k];
        }
        above += c[k];
      }
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= (bins - 1) << shift;
    left = sh.left;
    before = sh.before;
  }
  // ---- who stays: the candidates above the key, and of those equal to it the first `left`
  const bool ranked = m != 0 && !all && sh.equal != left;
  const uint32_t least = all ? 0u : m == 0 ? kNoKey : prefix;
  __syncthreads();  // sh.equal has been read: what follows uses the same memory
#pragma unroll 1
  for (int base = e0; base < e1; base += kBatch * kStep) {
    uint32_t k[kBatch][4];
    if (cached) kept_keys(base, k);
    else (void)src.keys_of(base, tid, e1, k);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * kStep + 4 * tid;
      if (base + u * kStep >= e1) break;
      bool stays[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) stays[j] = k[u][j] >= least;
      if (ranked) {  // entries equal to the key, counted in order
        uint32_t equal = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) equal += k[u][j] == prefix;
        uint32_t incl = equal;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (lane == 31) sh.warp_sum[warp] = incl;
        __syncthreads();
        uint32_t place = before + incl - equal;
        for (int w = 0; w < kEvictWarps; ++w) {
          const uint32_t c = sh.warp_sum[w];
          if (w < warp) place += c;
          before += c;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k[u][j] == prefix) stays[j] = place++ < left;
        __syncthreads();
      }
      src.put4(i, e1, stays);
    }
  }
  if (kept != nullptr && rank == 0 && tid == 0) kept[bh] = static_cast<int32_t>(recents + m);
  if (cluster > 1) cluster_sync();  // no CTA leaves while another may still read its counts
}

// CTAs a (b, h), up to 8: more while a run is over 4,096 entries and the CTAs fit the device side by side (two an SM).
int cluster_for(int64_t n, int64_t BH, int sms) {
  int c = 1;
  while (c < 8 && n > 4096 * c && BH * c * 2 <= 2 * static_cast<int64_t>(sms)) c *= 2;
  return c;
}

template <class Src>
kvp_status launch_evict(const Src& src, int64_t BH, int64_t most, int budget, const int32_t* now_dev, int now,
                        int32_t* kept, int32_t* status, void* stream) {
  int device = 0;
  const int sms = current_sms(&device);
  if (sms == 0) return KVP_ERR_CUDA;
  const int cluster = cluster_for(most, BH, sms);
  const int64_t run = (most + 32 * cluster - 1) / (32 * cluster) * 32;
  constexpr size_t base = (sizeof(EvictShared) + 15) / 16 * 16;
  // room for the keys of every run that the kernel keeps: a run is no longer than this one, and shorter only if !kExact
  const size_t smem = base + (run <= kKeysCap ? static_cast<size_t>(run) * 4 : (Src::kExact ? kListCap : kKeysCap) * 4);
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  if (device > 63 || (ready.load(std::memory_order_relaxed) >> device & 1u) == 0) {
    if (cudaFuncSetAttribute(evict_kernel<Src>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(base + kKeysCap * 4)) != cudaSuccess) {
      (void)cudaGetLastError();
      return KVP_ERR_CUDA;
    }
    if (device <= 63) ready.fetch_or(uint64_t{1} << device, std::memory_order_relaxed);
  }
  const dim3 grid(static_cast<unsigned>(BH * cluster));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      cluster > 1 ? launch_pdl_cluster(evict_kernel<Src>, grid, dim3(kEvictThreads), smem, st, cluster, src, cluster,
                                       budget, now_dev, now, kept, status)
                  : launch_pdl(evict_kernel<Src>, grid, dim3(kEvictThreads), smem, st, src, cluster, budget, now_dev, now,
                               kept, status);
  return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
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
  const PagedEvict src{acc,        acc_stride_b, acc_stride_h, acc_len, n_kv_heads, expire_pool, n_pages_cap, max_pages,
                       page_table, remap,        count,        recent,  now,        status,      nullptr,     nullptr,
                       nullptr,    0};
  return launch_evict(src, BH, static_cast<int64_t>(max_pages) * kPage, budget, now_dev, now, kept, status, stream);
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
  const DenseEvict src{acc, stride_b, stride_t, stride_h, n_kv_heads, n_pos, recent, now, expire, nullptr, nullptr, 0};
  return launch_evict(src, BH, n_pos, budget, nullptr, now, count, nullptr, stream);
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
