// kvp_prompt_attn: causal attention over packed prompts (DMS article, "DMS 작동
// 방식" step 5: the standard attention, here of a whole prompt).
#include "prompt.cuh"

namespace kvp {
namespace {

// S = Q K^T and O += P V on tcgen05, 128 query rows x 128 keys a step, two such
// query tiles (A and B) a CTA so that the tensor cores work on one while the
// softmax of the other runs. The tiles share their K and V: they are two query
// heads of one kv head over the same 128 rows (G even), or 256 rows of one head
// (G odd; the second may be past the end); a call with few tiles takes one of them
// an item. Tensor memory holds S and O of both (512 columns at D = 128); P, rounded
// to bf16, overwrites its S.
//
// Warps 0-3 and 4-7 are the softmax of A and B: a thread owns a row, so that
// maxima and sums need no exchange. Warp 8 issues the products (at D = 64 those with
// V, and warp 10 those with K), warp 9 the copies: K and V tiles of 128 rows through
// one ring. Tiles and key blocks start with the sequence, so only a tile's last block
// is masked.
//
// The reference M of a row's weights 2^(x c - M), c = scale log2 e, is its first
// block's maximum. It moves only when a block's weights come to more than 128 that
// pass it by 2^8 would (so a single one may pass it by 2^15) and its maximum does
// pass it by 2^8; then the softmax warps rescale O themselves, once the products of
// the block before are done (at D = 128 a block's S comes after them).
//
// P in bf16: both operands of a product are of one type, and V is bf16. A weight is off by
// 2^-8 at most, at random, so that it moves a row of many keys by 2e-4 to 3e-4 (2-norm,
// the measured cases) where out's own rounding to bf16 moves it by 1.6e-3: 1.67e-3
// against 1.65e-3 with exact weights. A second product for the rest of P would take
// half as much tensor time again. Sums of weights are of the unrounded ones, in fp32.
//
// A masked weight is 0, but 0 times an infinite or NaN value is NaN: before the
// products of a masked block its V tile is searched and such values are zeroed.
// Only then do the rows look them up in memory again, and add those they see.
//
// One CTA an SM takes work items in turn (warp 11 works them out ahead): the
// next item's Q, K and V are on their way, and its first S is there, while the
// softmax warps still write the last one's rows. Items go out from the longest
// to the shortest, forwards and backwards over the CTAs by turns. (Handed out as
// CTAs become free instead, 24 packed prompts of 17,365 tokens: 260 us for 255.)
//
// Bound: 4 D flops and an exponential for each (query, key) pair. 128 x 128 pairs
// take the special-function units 512 cycles, and at D = 128 the tensor cores 512
// for each of the two products. 16,384 tokens, 32/8 heads of 128: 1.33 to 1.36 ms
// replayed from a graph, 1.62 to 1.66 PFLOP/s (86 to 88 % of the measured burst rate
// of a bf16 GEMM, 95 to 98 % of its sustained one), at the power limit. Two threads a row with 64 logits each, for twice the warps:
// 1,858 us for 1,529 at that stage. 8,192 tokens at D = 64: 252 us, bound by the chain
// of a block in its softmax warp (the exponentials alone 112 us at their rate).
constexpr int kInfo = 2;                    // work items written down ahead of their use
constexpr int kFlags = 4;                   // items whose flags are apart: no warp is three items ahead of another
template <int D>
struct AttnCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;          // 128 rows x 64 columns
  static constexpr int kTileBytes = kBoxes * kBoxBytes;  // one tile of Q, K or V
  static constexpr int kStages = D == 128 ? 5 : 8;       // ring of K and V tiles
  // At D = 64 tensor memory has room for a third S, and the products are short: one warp issues those with K, another
  // those with V, each block's S as soon as a buffer is free (8,192 tokens, 32/8 heads: 311 us with one warp and two
  // buffers, where it waited for every signal in turn; 252 us so).
  static constexpr bool kApart = D == 64;
  static constexpr int kBufs = kApart ? 3 : 2;           // buffers of S (and then P)
  static constexpr uint32_t kOCol = kBufs * kTile;       // O of A and B
  static_assert(kOCol + 2 * D <= 512, "tensor memory");
  static constexpr int kPairs = 8;                       // ring of barriers that give stages back
  static_assert(!kApart || kPairs == kStages, "one for each stage");
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
  static constexpr int kSignals = kApart ? 2 * kBufs : kBufs;  // barriers that tell of S, and of O
  static constexpr int kBars = 2 + kStages + kPairs + kBufs + 2 * kSignals + 2 + 2 * kInfo;
  static constexpr int kInfoOff = (kBarOff + kBars * 8 + 15) / 16 * 16;  // [slot]{first row, length, tile, column}
  static constexpr int kFlagOff = kInfoOff + kInfo * 16;           // tensor memory's address, abort, bad values
  static constexpr int kSmem = 1024 + kFlagOff + 8 + 8 * kFlags;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kRingOff % 1024 == 0 && kBarOff % 8 == 0 && kInfoOff % 16 == 0 && kFlagOff % 4 == 0,
                "alignment");
};
constexpr int kSoftWarps = 8, kMmaWarp = 8, kCopyWarp = 9, kKeysWarp = 10, kPlanWarp = 11;
constexpr int kAttnThreads = 384;
// A row's 128 logits stay in registers: the softmax warps take 216 each and the
// others 72, of the 168 a thread that the block is launched with:
// 256 x 216 + 128 x 72 = 384 x 168.
constexpr int kRegsSoft = 216, kRegsRest = 72;
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;                // how far a row's maximum may pass its reference (base 2)
constexpr float kMostSum = 1.f / 8192;      // 128 weights of 2^(kLazy - kHeadroom)
constexpr float kBig = 268435456.f;         // from references of 2^28 on, x c - M is taken as (x - max) c

KVP_DEV uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The weights 2^(s c + ref) of a row's 128 logits: to tensor memory as bf16 pairs, and their sums (of the unrounded ones)
// in four pairs. One warp a scheduler does this at a time, so its order counts: the exponential of one value takes the
// special-function unit four cycles, and the products, conversions and sums of other values are placed in between.
KVP_DEV void weigh_block(const float (&s)[kTile], float c, float ref, uint32_t taddr, uint64_t (&sum)[4]) {
  constexpr int kAhead = 4, kBehind = 4;
  const uint64_t c2 = pack2(c, c), r2 = pack2(ref, ref);
  uint64_t t[kTile / 2];
  float e[kTile];
  uint32_t w[kTile / 2];
  sum[0] = sum[1] = sum[2] = sum[3] = 0;
  auto scale = [&](int i) {
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t[i]) : "l"(pack2(s[2 * i], s[2 * i + 1])), "l"(c2), "l"(r2));
  };
  auto finish = [&](int i) {
    asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(e[2 * i + 1]), "f"(e[2 * i]));
    asm volatile("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[i & 3]) : "l"(pack2(e[2 * i], e[2 * i + 1])));
    if (i % 16 == 15) tmem_st16(taddr + (i & ~15), w + (i & ~15));
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) scale(i);
#pragma unroll
  for (int i = 0; i < kTile / 2; ++i) {
    float a, b;
    unpack2(t[i], a, b);
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[2 * i]) : "f"(a));
    if (i + kAhead < kTile / 2) scale(i + kAhead);
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[2 * i + 1]) : "f"(b));
    if (i >= kBehind) finish(i - kBehind);
  }
#pragma unroll
  for (int i = kTile / 2 - kBehind; i < kTile / 2; ++i) finish(i);
}

// Searches row t of a V tile (swizzled boxes) for infinities and NaN, which times 0 are NaN, and makes them zeros; if the
// row is one of the sequence (`inside`), both tiles' flags get `tag` first.
template <int D>
KVP_DEV void clear_bad_values(uint8_t* tile, int t, bool inside, volatile int* flags, int tag) {
  using C = AttnCfg<D>;
  auto at = [&](int c) {
    return reinterpret_cast<uint4*>(tile + (c >> 3) * C::kBoxBytes + t * 128 + (((c & 7) ^ (t & 7)) << 4));
  };
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 found[4] = {zero, zero, zero, zero};
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 w = *at(c);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) found[i] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), zero, found[i]);
  }
  const __nv_bfloat162 sum = __hadd2(__hadd2(found[0], found[1]), __hadd2(found[2], found[3]));
  if (__low2float(sum) == 0.f && __high2float(sum) == 0.f) return;
  if (inside) {
    flags[0] = tag;
    flags[1] = tag;
    __threadfence_block();
  }
  for (int c = 0; c < D / 8; ++c) {
    uint32_t* w = reinterpret_cast<uint32_t*>(at(c));
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0x0000FFFFu;
    }
  }
}

// Adds the infinities and NaN of 32 columns of V that clear_bad_values took out, from memory: rows 0 .. last, `stride`
// values apart.
KVP_DEV void add_bad_values(float (&v)[32], const uint16_t* rows, int64_t stride, int last) {
#pragma unroll 1
  for (int r = 0; r <= last; ++r) {
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(rows + r * stride + k);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7F80u) == 0x7F80u) v[k + 2 * i] += bf16_lo(w[i]);
        if ((w[i] & 0x7F800000u) == 0x7F800000u) v[k + 2 * i + 1] += bf16_hi(w[i]);
      }
    }
  }
}

// 16 bf16 to a 32-byte aligned address, a whole sector in one store (24 prompts, 17,365 rows, 32/8 heads of 128: stores of
// 16 bytes, for each of which a warp's 32 rows take a pass of their own through L1, made 20 us of 253).
KVP_DEV void store32(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// What the two tiles of a work item are: two heads of a kv head, 256 rows of a head; or there is only one.
enum Tiles { kByHead = 0, kByRow = 1, kOneTile = 2 };

struct AttnMaps {
  CUtensorMap q, k, v;  // [D, heads, rows], boxes of 64 x 1 x 128
};

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1) prompt_attn_kernel(const PromptParams p, const int tiles,
                                                                      const __grid_constant__ AttnMaps maps) {
  using C = AttnCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in every lane, as the compiler can see
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* q_empty = q_full + 1;
  uint64_t* full = q_empty + 1;
  uint64_t* empty = full + C::kStages;
  // [A, B], o_full of a tile's last block. Where the products are issued apart, p_full is by buffer and the others, both of
  // every block, by tile and the number that the block has in it, % kBufs: a tile that has no blocks in some items and a
  // tile that goes on without it meet no phases of each other's.
  uint64_t* s_full = empty + C::kPairs;
  uint64_t* o_full = s_full + C::kSignals;
  uint64_t* p_full = o_full + C::kSignals;
  uint64_t* fin = p_full + C::kBufs;
  uint64_t* info_full = fin + 2;
  uint64_t* info_empty = info_full + kInfo;
  int4* info = reinterpret_cast<int4*>(smem + C::kInfoOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kFlagOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* bad_values = abort_flag + 1;  // [item % kFlags][A, B]: item + 1 if masked blocks hold some

  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1);
    for (int i = 0; i < C::kPairs; ++i) mbar_init(&empty[i], 1);
    for (int x = 0; x < C::kSignals; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&o_full[x], 1);
    }
    for (int x = 0; x < C::kBufs; ++x) mbar_init(&p_full[x], 4);
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&info_full[i], 1);
      mbar_init(&info_empty[i], kSoftWarps + 2 + C::kApart);
    }
    *abort_flag = 0;
    for (int i = 0; i < 2 * kFlags; ++i) bad_values[i] = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool by_head = tiles != kByRow;
  const int cols = tiles == kByHead ? p.Hq / 2 : p.Hq;  // work items of one tile
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_quietly(bar, parity, abort_flag, p.seqs.status); };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  auto gave_up = [&]() {
    if (lane == 0) {
      record_error(p.seqs.status, KVP_ERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  // A work item: A and B are heads hA, hB over tiles tA, tB of rows from `start` on, with nA and nB key blocks.
  struct Item {
    int start, len, tA, tB, hA, hB, nA, nB;
  };
  // Item number i of this CTA, as warp 11 leaves it (a whole warp calls this); false: there are no more, or a wait gave up.
  auto next_item = [&](int i, Item& t, bool& ok) {
    const int slot = i % kInfo;
    ok = wait_all(&info_full[slot], (i / kInfo) & 1);
    if (!ok) return false;
    const int4 v = info[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&info_empty[slot]);
    if (v.z < 0) return false;
    t.start = v.x;
    t.len = v.y;
    t.tA = v.z;
    t.tB = by_head ? v.z : v.z + 1;
    t.hA = tiles == kByHead ? 2 * v.w : v.w;
    t.hB = tiles == kByHead ? 2 * v.w + 1 : v.w;
    t.nA = t.tA + 1;
    t.nB = tiles != kOneTile && t.tB * kTile < t.len ? t.tB + 1 : 0;
    return true;
  };
  Item t;
  bool ok = true;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kPlanWarp) {
      // ------------------------------------------------------------ work items
      TileOrder order(p.seqs, by_head ? kTile : 2 * kTile);
      const int64_t items = static_cast<int64_t>(order.total) * cols;
      for (int i = 0;; ++i) {
        const int64_t at = static_cast<int64_t>(i) * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        int4 v = make_int4(0, 0, -1, 0);
        if (at < items) {
          const Tile f = order.find(static_cast<int>(at / cols));
          v = make_int4(f.start, f.len, by_head ? f.r : 2 * f.r, static_cast<int>(at % cols));
        }
        const int slot = i % kInfo;
        if (i >= kInfo) ok = wait_all(&info_empty[slot], (i / kInfo - 1) & 1);
        if (!ok) {
          gave_up();
          break;
        }
        if (lane == 0) {
          info[slot] = v;
          mbar_arrive(&info_full[slot]);
        }
        __syncwarp();
        if (v.z < 0) break;
      }
    } else if (warp == kCopyWarp) {
      // ------------------------------------------------------------ copies
      int g = 0, i = 0, nq = 0;  // tiles, items and pairs of query tiles so far
      // a tile is given back with the pair (V of a block, K of the next) that it is of, or by itself
      auto given_back = [&](int tile) {
        const int k = C::kApart ? tile : (tile + 1) / 2;
        return wait(&empty[k % C::kPairs], (k / C::kPairs) & 1);
      };
      auto load = [&](const CUtensorMap* m, uint8_t* dst, int head, int row, uint64_t* bar) {
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b) tma_load_3d(dst + b * C::kBoxBytes, m, 64 * b, head, row, bar);
      };
      for (; next_item(i, t, ok); ++i) {
        const int kv = t.hA / p.G, n = max(t.nA, t.nB);
        if (lane == 0) {
          for (int k = 0; ok && k < 2 * n; ++k) {  // K of block 0, V of block 0, K of block 1, ...
            const int st = g % C::kStages;
            if (g >= C::kStages) {
              ok = given_back(g - C::kStages);
              if (!ok) break;
            }
            mbar_arrive_expect_tx(&full[st], C::kTileBytes);
            load((k & 1) ? &maps.v : &maps.k, smem + C::kRingOff + st * C::kTileBytes, kv, t.start + (k >> 1) * kTile,
                 &full[st]);
            ++g;
            if (k == 1) {  // the queries, once the last item's products with its own are done
              if (i > 0) ok = wait(q_empty, (i - 1) & 1);
              if (!ok) break;
              ++nq;
              mbar_arrive_expect_tx(q_full, (t.nB > 0 ? 2 : 1) * C::kTileBytes);
              load(&maps.q, smem + C::kQOff, t.hA, t.start + t.tA * kTile, q_full);
              if (t.nB > 0) load(&maps.q, smem + C::kQOff + C::kTileBytes, t.hB, t.start + t.tB * kTile, q_full);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
      if (!ok) gave_up();
      if (lane == 0 && g > 0) {
        if (ok) {  // no arrival is left on its way when the CTA ends
          ok = wait(q_empty, (i - 1) & 1);
          for (int k = max(0, g - C::kStages); ok && k < g; ++k) ok = given_back(k);
        }
        // what was issued lands before the shared memory can go to another CTA (each wait bounded again)
        if (!ok) {
          if (nq > 0) (void)mbar_wait(q_full, (nq - 1) & 1);
          for (int k = max(0, g - C::kStages); k < g; ++k) (void)mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1);
        }
      }
      __syncwarp();
    } else if (C::kApart && (warp == kMmaWarp || warp == kKeysWarp)) {
      // ------------------------------------------------------------ products, apart
      // Blocks in the order A 0, B 0, A 1, B 1, ... (those that there are), numbered through all items: block number n is
      // in buffer n % kBufs, and its S comes once the products of block n - kBufs, which read P from there, are done.
      const bool keys = warp == kKeysWarp;
      const uint32_t leader = elect_one();
      const uint32_t q0 = smem_u32(smem + C::kQOff), ring = smem_u32(smem + C::kRingOff);
      uint32_t n = 0, g = 0;         // blocks, and tiles of K and V before this item
      uint32_t buf = 0, ph = 0;      // block n's buffer, and the phase of what is by buffer
      uint32_t at[2] = {0, C::kBufs}, par[2] = {0, 0};  // the signals of A's and B's next block, and their phase
      uint32_t before[3] = {0, 0, 0};  // those of block n - 1 - i: 2 x signal + phase
      static_assert(!C::kApart || C::kBufs == 3, "before[2] had this block's buffer");
      for (int i = 0; next_item(i, t, ok); ++i) {
        const int blocks = max(t.nA, t.nB);
        if (keys) ok = wait_all(q_full, i & 1);
        for (int j = 0; ok && j < blocks; ++j) {
          const uint32_t k = g + 2 * j + !keys, stage = k % C::kStages;
          ok = wait_all(&full[stage], (k / C::kStages) & 1);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || j >= (x == 0 ? t.nA : t.nB)) continue;
            if (keys) {
              if (n >= C::kBufs) ok = wait_all(&o_full[before[2] >> 1], before[2] & 1);
              if (!ok) continue;
              before[2] = before[1], before[1] = before[0], before[0] = 2 * at[x] + par[x];
              tc_fence_after();
              const uint64_t a = sw128_kmajor_desc(q0 + x * C::kTileBytes);
              const uint64_t b = sw128_kmajor_desc(ring + stage * C::kTileBytes);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
                mma_ss(leader, tmem + buf * kTile, a + off, b + off, idesc_bf16_f32(kTile, kTile), kk > 0);
              }
              commit_to(leader, &s_full[at[x]]);
            } else {
              ok = wait_all(&p_full[buf], ph);
              if (!ok) continue;
              tc_fence_after();
              const uint64_t v0 = sw128_mnmajor_desc(ring + stage * C::kTileBytes, C::kBoxBytes, 1024);
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                mma_ts(leader, tmem + C::kOCol + x * D, tmem + buf * kTile + ks * 8, v0 + ((ks * 2048) >> 4),
                       idesc_bf16_f32(kTile, D) | kIdescBMnMajor, j > 0 || ks > 0);
              commit_to(leader, &o_full[at[x]]);
            }
            ++n;
            if (++buf == C::kBufs) {
              buf = 0;
              ph ^= 1;
            }
            if (++at[x] == (x + 1) * C::kBufs) {
              at[x] = x * C::kBufs;
              par[x] ^= 1;
            }
          }
          if (ok) commit_to(leader, &empty[stage]);
        }
        if (!ok) break;
        if (keys) commit_to(leader, q_empty);
        g += 2 * blocks;
      }
      if (!ok) gave_up();
      commit_to(leader, &fin[keys]);
      (void)mbar_wait(&fin[keys], 0);  // every product has completed before tensor and shared memory go
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      // The whole warp runs this, on the same values, and one elected lane issues: so the descriptors stay in uniform
      // registers. (With the loop on one lane alone each product's operands were moved there one by one: 75 to 115
      // cycles a product, where it runs for 64.)
      constexpr uint32_t idS = idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t idO = idesc_bf16_f32(kTile, D) | kIdescBMnMajor;
      const uint32_t leader = elect_one();
      const uint32_t q0 = smem_u32(smem + C::kQOff), ring = smem_u32(smem + C::kRingOff);
      int st = 0;                    // ring stage and phase of the tile to land next
      uint32_t ph = 0;
      auto landed = [&]() {
        const bool r = wait_all(&full[st], ph);
        if (++st == C::kStages) {
          st = 0;
          ph ^= 1;
        }
        return r;
      };
      auto issue_s = [&](int x, int stage) {  // S of tile x with the K in `stage`
        const uint64_t a = sw128_kmajor_desc(q0 + x * C::kTileBytes);
        const uint64_t b = sw128_kmajor_desc(ring + stage * C::kTileBytes);
        const uint32_t d = tmem + x * kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
          mma_ss(leader, d, a + off, b + off, idS, kk > 0);
        }
        commit_to(leader, &s_full[x]);
      };
      int pair = 0;                  // V of an item's last block is given back with K of the next item's first
      auto release = [&]() {
        commit_to(leader, &empty[pair % C::kPairs]);
        ++pair;
      };
      uint32_t pph[2] = {0, 0};      // phases of p_full
      int kst = 0;                   // ring stage of the K to use next; a V's is the one after its block's K
      auto after = [&](int stage, int k) { return stage + k >= C::kStages ? stage + k - C::kStages : stage + k; };
      int i = 0;
      for (; next_item(i, t, ok); ++i) {
        const int nA = t.nA, nB = t.nB, n = max(nA, nB);
        ok = landed() && wait_all(q_full, i & 1);
        if (!ok) break;
        tc_fence_after();
        // S and P of the last item's tiles are used up: its products come first in the pipe
        issue_s(0, kst);
        if (nB > 0) issue_s(1, kst);
        release();
        if (n == 1) commit_to(leader, q_empty);
        ok = landed() && (n < 2 || landed());
        for (int j = 0; ok && j < n; ++j) {
          const int vst = after(kst, 1), nst = after(kst, 2);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int nx = x == 0 ? nA : nB;
            if (ok && j < nx) {
              ok = wait_all(&p_full[x], pph[x]);
              pph[x] ^= 1;
              if (ok) {
                tc_fence_after();
                const uint64_t v0 = sw128_mnmajor_desc(ring + vst * C::kTileBytes, C::kBoxBytes, 1024);
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks)
                  mma_ts(leader, tmem + C::kOCol + x * D, tmem + x * kTile + ks * 8, v0 + ((ks * 2048) >> 4), idO,
                         j > 0 || ks > 0);
                if (j == nx - 1) commit_to(leader, &o_full[x]);
              }
            }
            // the next step's tiles, while these products run: V here, K beside the second tile's
            if (ok && j + 1 + x < n) ok = landed();
            if (ok && j + 1 < nx) issue_s(x, nst);
          }
          if (j + 1 < n) release();
          if (j + 2 == n) commit_to(leader, q_empty);
          kst = nst;
        }
        if (!ok) break;
      }
      if (ok && i > 0) release();    // V of the last item's last block
      if (!ok) gave_up();
      commit_to(leader, fin);
      (void)mbar_wait(fin, 0);  // every product has completed before tensor and shared memory go
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t ocol = trow + C::kOCol + x * D;
    const float c = p.qscale;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.ot * 2) |
                        static_cast<uintptr_t>(p.oh * 2)) & 31u) == 0;  // rows of `out` are 32-byte aligned
    uint32_t g = 0, n0 = 0;     // tiles of K and V, and blocks, before this item
    uint32_t blocks = 0, items = 0;  // of this tile
    // Where the products are issued apart: the tile's block number `b` has been added to O. (Its own S, or a later one, is
    // there when this is asked, so block b - kBufs has: the barrier's phase is this one or the one before.)
    auto added = [&](uint32_t b) { return wait_all(&o_full[x * C::kBufs + b % C::kBufs], (b / C::kBufs) & 1); };
    for (int i = 0; next_item(i, t, ok); ++i) {
      const int nx = x == 0 ? t.nA : t.nB, tile = x == 0 ? t.tA : t.tB, head = x == 0 ? t.hA : t.hB;
      const int pos = tile * kTile + row;  // in the sequence; past its end: nothing is stored
      volatile int* flags = bad_values + i % kFlags * 2;
      float M = -INFINITY, m = -INFINITY, l = 0.f;
      for (int j = 0; j < nx; ++j) {
        // the block's number: after those of both tiles before it
        const auto number = [&](int j) { return n0 + min(j, t.nA) + min(j, t.nB) + (x == 1 && j < t.nA); };
        const uint32_t buf = C::kApart ? number(j) % C::kBufs : x;
        ok = C::kApart ? wait_all(&s_full[x * C::kBufs + blocks % C::kBufs], (blocks / C::kBufs) & 1)
                       : wait_all(&s_full[x], blocks & 1);
        if (!ok) break;
        ++blocks;
        tc_fence_after();
        const uint32_t scol = trow + buf * kTile;
        float s[kTile];
        tmem_ld128(scol, s);
        if (j == nx - 1) {  // keys after the row's own: those of its own 32 by their lane, those after by the warp
#pragma unroll
          for (int o = 0; o < kTile; o += 32) {
            if (o / 32 < (warp & 3)) continue;
            const int cut = o / 32 == (warp & 3) ? lane : -1;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k > cut) s[o + k] = -INFINITY;
          }
        }
        uint64_t sum[4];
        // With the reference as it is: no maximum is taken. If a row's sum says that some weight may have passed it by
        // 2^8 (or is no number, or the row has no reference yet), the block is taken again below, by its whole warp.
        bool again = M == -INFINITY || fabsf(M) >= kBig;
        if (!__all_sync(0xffffffffu, again)) {
          weigh_block(s, c, -M, scol, sum);
          float e, f;
          unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), e, f);
          again |= !(e + f <= kMostSum);
        }
        if (__any_sync(0xffffffffu, again)) {
          float top[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) top[k] = fmaxf(s[k], s[8 + k]);
#pragma unroll
          for (int k = 16; k < kTile; k += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) top[i] = fmaxf(top[i], fmaxf(s[k + i], s[k + 8 + i]));
          float mx = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])),
                           fmaxf(fmaxf(top[4], top[5]), fmaxf(top[6], top[7])));
          // Only the rows that ask for it move their reference, so that no row's bits depend on what its neighbours, which
          // may be of no sequence, hold. (The same as a condition of `grow`: 226 us for 222 with the 24 prompts.)
          if (!again) mx = -INFINITY;
          bool big = fabsf(M) >= kBig && M != -INFINITY;
          const bool grow = big ? (mx - m) * c > kLazy : fmaf(mx, c, -M) > kLazy - kHeadroom;
          const float M_new = fmaf(mx, c, kHeadroom);
          const bool big_new = fabsf(M_new) >= kBig;
          float al = 1.f;
          if (grow) {
            const float e = big_new ? (big ? (m - mx) * c : fmaf(-mx, c, M) - kHeadroom)
                                    : (big ? fmaf(m, c, kHeadroom - M_new) : M - M_new);
            al = M == -INFINITY ? 0.f : ex2_approx(e);
            M = M_new;
            m = mx;
            big = big_new;
            l *= al;
          }
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // (else a block's S comes after the products of the tile's block before)
            if (C::kApart) ok = added(blocks - 2);  // (`blocks` counts this one)
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int o = 0; o < D; o += 32) {
              float v[32];
              tmem_ld32(ocol + o, v);
              uint32_t y[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(v[i] * al);
              tmem_st32(ocol + o, y);
            }
          }
          // 2^(x c - M); where a reference is so large that its rounding counts, 2^((x - max) c - headroom)
          if (__any_sync(0xffffffffu, big)) {
            const float off = big ? m : 0.f;
#pragma unroll
            for (int k = 0; k < kTile; ++k) s[k] -= off;
          }
          weigh_block(s, c, big ? -kHeadroom : M == -INFINITY ? 0.f : -M, scol, sum);
        }
        float l0, l1;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), l0, l1);
        l += l0 + l1;
        // the masked block's values (of two heads the first tile's warps see to them: its products come first)
        if (j == nx - 1 && (x == 0 || !by_head)) {
          const uint32_t k = g + 2 * j + 1;
          ok = wait_all(&full[k % C::kStages], (k / C::kStages) & 1);
          if (!ok) break;
          clear_bad_values<D>(smem + C::kRingOff + (k % C::kStages) * C::kTileBytes, row, pos < t.len, flags, i + 1);
          fence_proxy_async();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      g += 2 * max(t.nA, t.nB);
      n0 += t.nA + t.nB;
      if (nx == 0) continue;
      ok = C::kApart ? added(blocks - 1) : wait_all(&o_full[x], items & 1);
      ++items;
      if (!ok) break;
      tc_fence_after();
      const bool some = flags[x] == i + 1;
      const bool mine = pos < t.len;
      const int64_t r = t.start + pos;
      uint16_t* out = p.out + r * p.ot + head * p.oh;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (!__any_sync(0xffffffffu, some || l == 0.f)) {
        float v[D];
        if constexpr (D == 128) tmem_ld128(ocol, v); else tmem_ld64(ocol, v);
        const uint64_t inv2 = pack2(inv, inv);
        // Two lanes trade halves of 32 columns, so that a store takes 64 bytes of each row (227 -> 222 us with the prompts
        // named at store32; 2 to 4 % of short calls).
        const bool odd = (lane & 1) != 0;
        uint16_t* to = out - (odd ? p.ot - 16 : 0);  // this lane's half, in the row of the even one
        const int pos0 = pos - odd;
#pragma unroll
        for (int k = 0; k < D; k += 32) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e, f;
            unpack2(mul2(pack2(v[k + 2 * i], v[k + 2 * i + 1]), inv2), e, f);
            w[i] = bf16x2(e, f);
          }
          if (wide) {
            uint32_t y0[8], y1[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w[i] : w[8 + i], 1);
              y0[i] = odd ? other : w[i];
              y1[i] = odd ? w[8 + i] : other;
            }
            if (pos0 < t.len) store32(to + k, y0);
            if (pos0 + 1 < t.len) store32(to + p.ot + k, y1);
          } else if (mine) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(out + k + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
          }
        }
      } else {
#pragma unroll 1
        for (int o = 0; o < D; o += 32) {
          float v[32];
          tmem_ld32(ocol + o, v);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = l == 0.f ? 0.f : v[k] * inv;  // (a value that is no number counts for nothing)
          if (some && mine && l != 0.f)  // (a row without a finite logit is zero, whatever it sees)
            add_bad_values(v, p.v + (t.start + t.tA * kTile) * p.vt + head / p.G * p.vh + o, p.vt, pos - t.tA * kTile);
          if (mine) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(out + o + k) =
                  make_uint4(bf16x2(v[k], v[k + 1]), bf16x2(v[k + 2], v[k + 3]), bf16x2(v[k + 4], v[k + 5]),
                             bf16x2(v[k + 6], v[k + 7]));
          }
        }
      }
      tc_fence_before();  // O has been read: the next item's products may overwrite it once its P is there
      if (mine && p.lse != nullptr) {
        // the reference and the sum's logarithm; a big one as it was taken
        const float ref = fabsf(M) >= kBig ? m * c + kHeadroom : M;
        p.lse[head * p.seqs.n_tok + r] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
      }
    }
    if (!ok) {
      tmem_st_wait();  // weights on their way land before tensor memory goes
      gave_up();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
kvp_status launch_attn(const PromptParams& p, int n_kv_heads, cudaStream_t st) {
  using C = AttnCfg<D>;
  AttnMaps maps;
  if (!make_tmap_heads<D>(&maps.q, p.q, p.seqs.n_tok, p.qt, p.Hq, p.qh) ||
      !make_tmap_heads<D>(&maps.k, p.k, p.seqs.n_tok, p.kt, n_kv_heads, p.kh) ||
      !make_tmap_heads<D>(&maps.v, p.v, p.seqs.n_tok, p.vt, n_kv_heads, p.vh))
    return KVP_ERR_CUDA;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int device = 0;
  const int sms = current_sms(&device);
  if (sms == 0) return KVP_ERR_CUDA;
  if (device > 63 || (ready.load(std::memory_order_relaxed) >> device & 1u) == 0) {
    if (cudaFuncSetAttribute(prompt_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return KVP_ERR_CUDA;
    }
    if (device <= 63) ready.fetch_or(uint64_t{1} << device, std::memory_order_relaxed);
  }
  // Two tiles an item, but where even single ones leave SMs idle: then each has less to do (509 tokens, 32/8 heads:
  // 15.2 us with pairs, 12.4 us so).
  const int64_t singles = (p.seqs.n_tok / kTile + p.seqs.n) * p.Hq;
  const int tiles = singles <= sms ? kOneTile : p.G % 2 == 0 ? kByHead : kByRow;
  const int64_t most = tiles == kOneTile  ? singles
                       : tiles == kByHead ? singles / 2
                                          : (p.seqs.n_tok / (2 * kTile) + p.seqs.n) * p.Hq;
  return launch_pdl(prompt_attn_kernel<D>, dim3(static_cast<unsigned>(std::min<int64_t>(sms, most))), dim3(kAttnThreads),
                    C::kSmem, st, p, tiles, maps) == cudaSuccess
             ? KVP_OK
             : KVP_ERR_CUDA;
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
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch_attn<128>(p, n_kv_heads, cs) : launch_attn<64>(p, n_kv_heads, cs);
}
