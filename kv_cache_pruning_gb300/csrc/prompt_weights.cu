// kvp_prompt_weights: the attention weight that every key of packed prompts
// received (DMS article, "DMS 작동 방식" step 5: the weights of the standard
// attention, summed over queries and shared heads).
#include <type_traits>

#include "prompt.cuh"

namespace kvp {
namespace {

// S = K Q^T on tcgen05 with the keys as rows: a thread owns a key, and its sum
// over queries stays in its register, without exchange or atomics. A work item is
// two tiles of 128 keys (A and B) of one kv head; every tile of 128 queries (QB
// rows of 128 / QB heads of the group) that either sees goes by once for both.
// Weights are 2^(x c - lse log2 e): the row's normaliser is known, so no maximum
// and no second product.
//
// Bound: an exponential and 2 D flops for each (query, key) pair. 128 x 128 pairs
// take the special-function units 512 cycles and, at D = 128, the tensor cores as
// many. So S of both tiles has two buffers (all 512 columns of tensor memory),
// and four warps on each scheduler hide each other's latencies: of a tile's keys
// each thread sums half the queries, 32 at a time, in a loop short enough to stay
// in the instruction cache. (Eight warps with 128 logits in registers each: 281 us
// for 267 at that stage; 64 logits a round of a loop unrolled further: 294.) 8,192
// tokens, 32/8 heads of 128: 246 us, 1.12 PFLOP/s; its longest items, which see every
// query, are 15 % longer than an SM's share.
//
// Warps 0-7 and 8-15 sum for A and B, warp 16 issues the products, warp 17
// copies, warp 18 brings the normalisers, warp 19 works out items ahead.
//
// A query whose lse is -inf pays nothing, whatever its logits are: its addend is the
// lowest number, which sees to that while they are finite. Where a sum is no number
// the tile is summed again without the columns of that addend. (With a bit for each such
// column, looked at before each tile: 261 us for 251, and 198 for 185 with 64 heads.)

// The warp that brings the normalisers reads kAhead tiles on, which may be as many items, before it writes the first of
// them, and no item's place is taken again before every warp has read it.
constexpr int kItems = 8, kAhead = 4;
static_assert(kItems > kAhead, "a warp would wait for one that waits for it");

template <int D, int QB>
struct WeightsCfg {
  static constexpr int kHeads = kTile / QB;              // query heads of a tile
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;          // 128 rows x 64 columns
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  // A window is one query tile or two an item: there the next item's keys come while this one's are used. Else the
  // room goes to query tiles.
  static constexpr int kKeyBufs = QB < kTile ? 2 : 1;
  static constexpr int kStages = (D == 128 ? 6 : 12) - 2 * kKeyBufs;  // ring of query tiles
  static constexpr int kKOff = 0;                        // keys of A and B
  static constexpr int kRingOff = 2 * kKeyBufs * kTileBytes;
  static constexpr int kLseOff = kRingOff + kStages * kTileBytes;  // normalisers of each buffer of S
  static constexpr int kXchOff = kLseOff + 2 * kTile * 4;          // a sum for each key
  static constexpr int kBarOff = kXchOff + 2 * kTile * 4;
  static constexpr int kBars = 2 * kStages + 2 * kKeyBufs + 8 + 1 + 2 * kItems;
  static constexpr int kInfoOff = (kBarOff + kBars * 8 + 15) / 16 * 16;  // [slot]{sequence, first row, length, head}, {pair}
  static constexpr int kFlagOff = kInfoOff + kItems * 32;                // tensor memory's address, abort
  static constexpr int kSmem = 1024 + kFlagOff + 8;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kRingOff % 1024 == 0 && kLseOff % 16 == 0 && kBarOff % 8 == 0 && kInfoOff % 16 == 0, "alignment");
};
constexpr int kSumWarps = 16, kMmaWarp = 16, kCopyWarp = 17, kLseWarp = 18, kPlanWarp = 19;
constexpr int kWeightsThreads = 640;
constexpr int kUsers = kSumWarps + 3;  // warps that read a work item
constexpr int kWindowRows = 32;        // rows of a query tile where at most twice as many count: heads share a tile

struct WeightsMaps {
  CUtensorMap q, k;  // [D, heads, rows], boxes of 64 x 1 x QB and 64 x 1 x 128
};

enum Columns { kWhole, kCut, kMarked };             // which columns of a tile are left out
constexpr float kPaysNothing = -3.402823466e38f;    // addend of a column whose lse is -inf

template <int D, int QB>
__global__ void __launch_bounds__(kWeightsThreads, 1) prompt_weights_kernel(const PromptParams p,
                                                                            const __grid_constant__ WeightsMaps maps) {
  using C = WeightsCfg<D, QB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in every lane, as the compiler can see
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint64_t* k_full = empty + C::kStages;       // [item % kKeyBufs]
  uint64_t* k_empty = k_full + C::kKeyBufs;
  uint64_t* s_full = k_empty + C::kKeyBufs;    // [A, B][buffer]
  uint64_t* s_empty = s_full + 4;              // [buffer]: S of A and B and the normalisers have been used
  uint64_t* lse_full = s_empty + 2;
  uint64_t* fin = lse_full + 2;
  uint64_t* info_full = fin + 1;
  uint64_t* info_empty = info_full + kItems;
  int4* info = reinterpret_cast<int4*>(smem + C::kInfoOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kFlagOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kKeyBufs; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_empty[i], kSumWarps);
      mbar_init(&lse_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&info_full[i], 1);
      mbar_init(&info_empty[i], kUsers);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int H = p.Hq / p.G;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_quietly(bar, parity, abort_flag, p.seqs.status); };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  auto gave_up = [&]() {
    if (lane == 0) {
      record_error(p.seqs.status, KVP_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  // A work item: keys k0 .. k0 + 255 of kv head h of a sequence; its query tiles are tile i of the `heads` groups of
  // kHeads query heads, i0 <= i < i1, rows q0(i) = first + i QB of the sequence.
  struct Item {
    int seq, start, len, h, k0, first, i0, i1;
    KVP_DEV int q0(int i) const { return first + i * QB; }
    // whether tile x has keys that some query of tile i sees
    KVP_DEV bool sees(int x, int i) const {
      return k0 + x * kTile < len && q0(i) + QB > k0 + x * kTile;
    }
  };
  const int groups = (p.G + C::kHeads - 1) / C::kHeads;
  auto next_item = [&](int i, Item& t, bool& ok) {
    const int slot = i % kItems;
    ok = wait_all(&info_full[slot], (i / kItems) & 1);
    if (!ok) return false;
    const int4 v = info[2 * slot];
    const int pair = info[2 * slot + 1].x;
    __syncwarp();
    if (lane == 0) mbar_arrive(&info_empty[slot]);
    if (v.x < 0) return false;
    t.seq = v.x;
    t.start = v.y;
    t.len = v.z;
    t.h = v.w;
    t.k0 = pair * 2 * kTile;
    t.first = p.n_last > 0 ? max(0, t.len - p.n_last) : 0;
    t.i0 = t.k0 > t.first ? (t.k0 - t.first) / QB : 0;
    t.i1 = (t.len - t.first + QB - 1) / QB;
    return true;
  };
  Item t;
  bool ok = true;

  if (warp >= kSumWarps) {
    if (warp == kPlanWarp) {
      // ------------------------------------------------------------ work items
      TileOrder order(p.seqs, 2 * kTile);
      const int64_t items = static_cast<int64_t>(order.total) * H;
      for (int i = 0;; ++i) {
        const int64_t at = static_cast<int64_t>(i) * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        int4 v = make_int4(-1, 0, 0, 0);
        int pair = 0;
        if (at < items) {
          // the order is of attention's rows, the last first; the first keys are seen by most queries
          const Tile f = order.find(static_cast<int>(at / H));
          v = make_int4(f.seq, f.start, f.len, static_cast<int>(at % H));
          pair = (f.len + 2 * kTile - 1) / (2 * kTile) - 1 - f.r;
        }
        const int slot = i % kItems;
        if (i >= kItems) ok = wait_all(&info_empty[slot], (i / kItems - 1) & 1);
        if (!ok) {
          gave_up();
          break;
        }
        if (lane == 0) {
          info[2 * slot] = v;
          info[2 * slot + 1].x = pair;
          mbar_arrive(&info_full[slot]);
        }
        __syncwarp();
        if (v.x < 0) break;
      }
    } else if (warp == kCopyWarp) {
      // ------------------------------------------------------------ copies
      int g = 0, i = 0, nk = 0;  // query tiles, items and pairs of key tiles so far
      for (; next_item(i, t, ok); ++i) {
        if (lane == 0) {
          auto keys = [&]() {  // once the item that has used their room before is done
            const int kb = i % C::kKeyBufs;
            if (i >= C::kKeyBufs) ok = wait(&k_empty[kb], (i / C::kKeyBufs - 1) & 1);
            if (!ok) return;
            ++nk;
            const int tiles = t.k0 + kTile < t.len ? 2 : 1;
            mbar_arrive_expect_tx(&k_full[kb], tiles * C::kTileBytes);
            for (int x = 0; x < tiles; ++x)
#pragma unroll
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_3d(smem + C::kKOff + (2 * kb + x) * C::kTileBytes + b * C::kBoxBytes, &maps.k, 64 * b, t.h,
                            t.start + t.k0 + x * kTile, &k_full[kb]);
          };
          for (int hg = 0; ok && hg < groups; ++hg) {
            const int heads = min(C::kHeads, p.G - hg * C::kHeads);
            for (int qi = t.i0; ok && qi < t.i1; ++qi) {
              const int st = g % C::kStages;
              if (g >= C::kStages) ok = wait(&empty[st], (g / C::kStages - 1) & 1);
              if (!ok) break;
              mbar_arrive_expect_tx(&full[st], heads * QB * D * 2);
              for (int hh = 0; hh < heads; ++hh)
#pragma unroll
                for (int b = 0; b < C::kBoxes; ++b)
                  tma_load_3d(smem + C::kRingOff + st * C::kTileBytes + b * C::kBoxBytes + hh * QB * 128, &maps.q, 64 * b,
                              t.h * p.G + hg * C::kHeads + hh, t.start + t.q0(qi), &full[st]);
              ++g;
              if (hg == 0 && qi == t.i0) keys();  // the first query tile waits for nothing but its stage
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
      if (!ok) gave_up();
      if (lane == 0) {
        if (ok) {  // no arrival is left on its way when the CTA ends
          for (int k = max(0, nk - C::kKeyBufs); ok && k < nk; ++k)
            ok = wait(&k_empty[k % C::kKeyBufs], (k / C::kKeyBufs) & 1);
          for (int k = max(0, g - C::kStages); ok && k < g; ++k) ok = wait(&empty[k % C::kStages], (k / C::kStages) & 1);
        }
        if (!ok) {  // what was issued lands before the shared memory can go to another CTA (each wait bounded again)
          for (int k = max(0, nk - C::kKeyBufs); k < nk; ++k)
            (void)mbar_wait(&k_full[k % C::kKeyBufs], (k / C::kKeyBufs) & 1);
          for (int k = max(0, g - C::kStages); k < g; ++k) (void)mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1);
        }
      }
      __syncwarp();
    } else if (warp == kLseWarp) {
      // ------------------------------------------------------------ normalisers
      // Loads are issued kAhead tiles before their values are written (one takes as long as a tile's exponentials).
      int i = 0, hg = groups, qi = 0, g = 0;
      t.i1 = 0;
      // lane's columns of the next tile, 0 for those that are no query; false: there is none
      auto load = [&](float (&v)[4]) {
        if (qi + 1 < t.i1 && hg < groups) {
          ++qi;
        } else {
          if (++hg >= groups) {
            if (!next_item(i++, t, ok)) return false;
            hg = 0;
          }
          qi = t.i0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int col = lane + 32 * k, hh = hg * C::kHeads + col / QB, q = t.q0(qi) + col % QB;
          v[k] = 0.f;
          if (hh < p.G && q < t.len) v[k] = p.lse_in[(t.h * p.G + hh) * p.seqs.n_tok + t.start + q];
        }
        return true;
      };
      auto write = [&](const float (&v)[4]) {
        const int buf = g & 1;
        if (g >= 2) ok = wait_all(&s_empty[buf], ((g >> 1) - 1) & 1);
        if (!ok) return;
        float* to = reinterpret_cast<float*>(smem + C::kLseOff) + buf * kTile;
#pragma unroll
        for (int k = 0; k < 4; ++k) to[lane + 32 * k] = v[k] == -INFINITY ? kPaysNothing : -v[k] * kLog2e;
        __syncwarp();
        if (lane == 0) mbar_arrive(&lse_full[buf]);
        ++g;
      };
      float v[kAhead][4];
      int left = 0;  // tiles loaded and not written
      bool more = true;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        more = more && load(v[k]);
        left += more;
      }
      while (ok && left > 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (!ok || left == 0) break;
          write(v[k]);
          --left;
          more = more && ok && load(v[k]);
          left += more;
        }
      }
      if (!ok) gave_up();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      const uint32_t leader = elect_one();
      const uint32_t keys = smem_u32(smem + C::kKOff), ring = smem_u32(smem + C::kRingOff);
      int st = 0;                 // ring stage and its phase
      uint32_t ph = 0;
      uint32_t n = 0;             // query tiles so far: buffer n & 1, its phase n >> 1
      int i = 0;
      for (; next_item(i, t, ok); ++i) {
        const int kb = i % C::kKeyBufs;
        ok = wait_all(&k_full[kb], (i / C::kKeyBufs) & 1);
        for (int hg = 0; ok && hg < groups; ++hg) {
          const uint32_t idS = idesc_bf16_f32(kTile, QB * min(C::kHeads, p.G - hg * C::kHeads));
          for (int qi = t.i0; ok && qi < t.i1; ++qi, ++n) {
            const uint32_t buf = n & 1;
            // (the normalisers come once the buffer's last logits have been used)
            ok = wait_all(&full[st], ph) && wait_all(&lse_full[buf], (n >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b0 = sw128_kmajor_desc(ring + st * C::kTileBytes);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (t.sees(x, qi)) {
                const uint64_t a0 = sw128_kmajor_desc(keys + (2 * kb + x) * C::kTileBytes);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
                  mma_ss(leader, tmem + (2 * x + buf) * kTile, a0 + off, b0 + off, idS, kk > 0);
                }
              }
              commit_to(leader, &s_full[2 * x + buf]);
            }
            commit_to(leader, &empty[st]);
            if (++st == C::kStages) {
              st = 0;
              ph ^= 1;
            }
          }
        }
        if (!ok) break;
        commit_to(leader, &k_empty[kb]);
      }
      if (!ok) gave_up();
      commit_to(leader, fin);
      (void)mbar_wait(fin, 0);  // every product has completed before tensor and shared memory go
    }
  } else {
    // ------------------------------------------------------------ sums
    // tile x, key `row`, columns 64 half .. of each query tile
    const int x = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t scol = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 2 * x * kTile + half * 64;
    const float* lse = reinterpret_cast<const float*>(smem + C::kLseOff) + half * 64;
    float* xch = reinterpret_cast<float*>(smem + C::kXchOff) + x * kTile + row;
    const uint64_t c2 = pack2(p.qscale, p.qscale);
    const int pair = 1 + x * 4 + quad;  // named barrier of the two warps of a key, which leave together
    uint32_t n = 0;
    for (int i = 0;; ++i) {
      const bool more = next_item(i, t, ok);
      if (!ok) gave_up();  // before the barrier: the other warp may be waiting for what does not come now
      if (named_bar_or(pair, 64, !ok)) {
        ok = false;
        break;
      }
      if (!more) break;
      const int k0 = t.k0 + x * kTile, pos = k0 + row;  // the key's position; past the sequence's end: nothing is stored
      float total = 0.f, lost = 0.f;                    // the sum of the tiles' sums and what its additions rounded off
      for (int hg = 0; ok && hg < groups; ++hg) {
        const int cols = QB * min(C::kHeads, p.G - hg * C::kHeads) - half * 64;
        for (int qi = t.i0; qi < t.i1; ++qi, ++n) {
          const uint32_t buf = n & 1;
          ok = wait_all(&s_full[2 * x + buf], (n >> 1) & 1);
          if (!ok) break;
          if (t.sees(x, qi)) {
            tc_fence_after();
            const int q0 = t.q0(qi);
            uint64_t sum[4] = {0, 0, 0, 0};
            // kCut: a tile with columns that this key does not see, or that are no query; kMarked: that pay nothing too. They
            // count for nothing, whatever their logits and normalisers are.
            auto add_up = [&](auto how) {
              constexpr int kHow = decltype(how)::value;
#pragma unroll 1
              for (int o = 0; o < 64; o += 32) {
                if (o >= cols) break;
                float s[32];
                tmem_ld32(scol + buf * kTile + o, s);
                const float4* to_add = reinterpret_cast<const float4*>(lse + buf * kTile + o);
                // columns o + k with from <= k < to are queries that see the key
                const int first = QB == kTile ? half * 64 + o : 0;
                const int from = pos - q0 - first, to = t.len - q0 - first;
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                  const float4 r = to_add[k / 4];
                  float e[4];
                  unpack2(fma2(pack2(s[k], s[k + 1]), c2, pack2(r.x, r.y)), e[0], e[1]);
                  unpack2(fma2(pack2(s[k + 2], s[k + 3]), c2, pack2(r.z, r.w)), e[2], e[3]);
                  if constexpr (kHow == kMarked) {
                    const float mark[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      if (mark[j] == kPaysNothing) e[j] = -INFINITY;
                  }
                  if constexpr (kHow != kWhole) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      if (k + j < from || k + j >= to) e[j] = -INFINITY;
                  }
                  sum[k / 2 & 3] = add2(sum[k / 2 & 3], pack2(ex2_approx(e[0]), ex2_approx(e[1])));
                  sum[(k / 2 + 1) & 3] = add2(sum[(k / 2 + 1) & 3], pack2(ex2_approx(e[2]), ex2_approx(e[3])));
                }
              }
            };
            float a, b;
            auto total_of = [&]() {
              unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
              a += b;
            };
            if (q0 < k0 + kTile - 1 || q0 + QB > t.len) {
              add_up(std::integral_constant<int, kCut>{});
            } else {
              add_up(std::integral_constant<int, kWhole>{});
            }
            total_of();
            if (__any_sync(0xffffffffu, !(a < INFINITY))) {
              sum[0] = sum[1] = sum[2] = sum[3] = 0;
              add_up(std::integral_constant<int, kMarked>{});
              total_of();
            }
            // total + a exactly: the rounded sum, and the rest kept apart
            const float both = total + a, back = both - total;
            lost += (total - (both - back)) + (a - back);
            total = both;
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[buf]);
        }
      }
      // the two halves of the key's sum meet (the next item's after both have come past its barrier)
      float sum = total + (fabsf(lost) < INFINITY ? lost : 0.f);
      if (half == 1) *xch = sum;
      if (!ok) gave_up();
      if (named_bar_or(pair, 64, !ok)) {
        ok = false;
        break;
      }
      if (half == 0) sum += *xch;
      if (half == 0 && pos < t.len) {
        if (p.as < 0) {
          p.acc[(t.start + pos) * p.at + t.h * p.ah] = sum;
        } else if (pos < p.acc_len) {
          p.acc[t.seq * p.as + pos * p.at + t.h * p.ah] = sum;
        } else {
          record_error(p.seqs.status, KVP_ERR_BOUNDS);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int QB>
kvp_status launch_weights(const PromptParams& p, cudaStream_t st) {
  using C = WeightsCfg<D, QB>;
  const int H = p.Hq / p.G;
  WeightsMaps maps;
  if (!make_tmap_heads<D>(&maps.q, p.q, p.seqs.n_tok, p.qt, p.Hq, p.qh, QB) ||
      !make_tmap_heads<D>(&maps.k, p.k, p.seqs.n_tok, p.kt, H, p.kh))
    return KVP_ERR_CUDA;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int device = 0;
  const int sms = current_sms(&device);
  if (sms == 0) return KVP_ERR_CUDA;
  if (device > 63 || (ready.load(std::memory_order_relaxed) >> device & 1u) == 0) {
    if (cudaFuncSetAttribute(prompt_weights_kernel<D, QB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return KVP_ERR_CUDA;
    }
    if (device <= 63) ready.fetch_or(uint64_t{1} << device, std::memory_order_relaxed);
  }
  const int64_t most = (p.seqs.n_tok / (2 * kTile) + p.seqs.n) * H;
  return launch_pdl(prompt_weights_kernel<D, QB>, dim3(static_cast<unsigned>(std::min<int64_t>(sms, most))),
                    dim3(kWeightsThreads), C::kSmem, st, p, maps) == cudaSuccess
             ? KVP_OK
             : KVP_ERR_CUDA;
}

}  // namespace
}  // namespace kvp

using namespace kvp;

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
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (n_last > 0 && n_last <= 2 * kWindowRows)
    return head_dim == 128 ? launch_weights<128, kWindowRows>(p, cs) : launch_weights<64, kWindowRows>(p, cs);
  return head_dim == 128 ? launch_weights<128, kTile>(p, cs) : launch_weights<64, kTile>(p, cs);
}
