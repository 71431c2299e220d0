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

// Number `idx` of all sequences' tiles of `tile` rows, each sequence's last tile first (a whole warp calls this); false
// past the last.
KVP_DEV bool find_tile(const Seqs& s, int tile, int idx, Tile& t) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < s.n; base += 32) {
    const int i = base + lane;
    int start = 0;
    const int len = i < s.n ? seq_rows(s, i, start) : 0;
    const int tiles = (len + tile - 1) / tile;
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
      t.r = before + __shfl_sync(0xffffffffu, incl, src) - 1 - idx;
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// The sequences' tiles of `tile` rows from the longest work to the shortest: by their number in their sequence, the last
// ones first, and sequence by sequence among equal ones (a whole warp calls these).
struct TileOrder {
  const Seqs& s;
  int tile, total, most;
  int mine, my_start, my_len;  // with 32 sequences at most: this lane's
  KVP_DEV TileOrder(const Seqs& seqs, int tile_) : s(seqs), tile(tile_) {
    int sum = 0, top = 0;
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < s.n; i += 32) {
      my_len = seq_rows(s, i, my_start);
      mine = (my_len + tile - 1) / tile;
      sum += mine;
      top = max(top, mine);
    }
    if (lane >= s.n) mine = my_len = my_start = 0;
    total = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, top);
  }
  KVP_DEV int tiles(int i, int& start, int& len) const {
    if (s.n <= 32) {
      start = my_start;
      len = my_len;
      return mine;
    }
    len = i < s.n ? seq_rows(s, i, start) : 0;
    return (len + tile - 1) / tile;
  }
  // tiles of number r and above in their sequences
  KVP_DEV int from(int r) const {
    int sum = 0, start, len;
    for (int i = threadIdx.x & 31; i < (s.n + 31) / 32 * 32; i += 32) sum += max(0, tiles(i, start, len) - r);
    return __reduce_add_sync(0xffffffffu, sum);
  }
  KVP_DEV Tile find(int idx) const {  // idx < total
    int lo = 0, hi = most, above = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2, f = from(mid);
      if (f > idx) {
        lo = mid;
      } else {
        hi = mid;
        above = f;
      }
    }
    Tile t{0, 0, 0, lo};
    int left = idx - above;
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < s.n; base += 32) {
      int start = 0, len = 0;
      const uint32_t has = __ballot_sync(0xffffffffu, tiles(base + lane, start, len) > lo);
      if (left < __popc(has)) {
        const int src = __fns(has, 0, left + 1);
        t.seq = base + src;
        t.start = __shfl_sync(0xffffffffu, start, src);
        t.len = __shfl_sync(0xffffffffu, len, src);
        break;
      }
      left -= __popc(has);
    }
    return t;
  }
};

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

// ---------------------------------------------------------------- attention
// S = Q K^T and O += P V on tcgen05, 128 query rows x 128 keys a step, two such
// query tiles (A and B) a CTA so that the tensor cores work on one while the
// softmax of the other runs. The tiles share their K and V: they are two query
// heads of one kv head over the same 128 rows (G even), or 256 rows of one head
// (G odd; the second may be past the end). Tensor memory holds S and O of both
// (512 columns at D = 128); P, rounded to bf16, overwrites its S.
//
// Warps 0-3 and 4-7 are the softmax of A and B: a thread owns a row, so that
// maxima and sums need no exchange. Warp 8 issues the products, warp 9 the
// copies: K and V tiles of 128 rows through one ring. Tiles and key blocks start
// with the sequence, so only a tile's last block is masked.
//
// The reference M of a row's weights 2^(x c - M), c = scale log2 e, is its first
// block's maximum and moves only when a later one passes it by 2^8; then the
// softmax warps rescale O themselves (a block's S is complete only after the
// products of the block before).
//
// A masked weight is 0, but 0 times an infinite or NaN value is NaN: before the
// products of a masked block its V tile is searched and such values are zeroed.
// Only then do the rows look them up in memory again, and add those they see.
//
// One CTA an SM takes work items in turn (warp 11 works them out one ahead): the
// next item's Q, K and V are on their way, and its first S is there, while the
// softmax warps still write the last one's rows. Items go out from the longest
// to the shortest, forwards and backwards over the CTAs by turns.
constexpr int kInfo = 2;                    // work items ahead
constexpr int kFlags = 4;                   // items whose flags are apart: no warp is three items ahead of another
template <int D>
struct AttnCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;          // 128 rows x 64 columns
  static constexpr int kTileBytes = kBoxes * kBoxBytes;  // one tile of Q, K or V
  static constexpr int kStages = D == 128 ? 5 : 8;       // ring of K and V tiles
  static constexpr int kPairs = 8;                       // ring of barriers that give stages back
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
  static constexpr int kBars = 2 + kStages + kPairs + 3 * 2 + 1 + 2 * kInfo;
  static constexpr int kInfoOff = (kBarOff + kBars * 8 + 15) / 16 * 16;  // [slot]{first row, length, tile, column}
  static constexpr int kFlagOff = kInfoOff + kInfo * 16;           // tensor memory's address, abort, bad values
  static constexpr int kSmem = 1024 + kFlagOff + 8 + 8 * kFlags;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kRingOff % 1024 == 0 && kBarOff % 8 == 0 && kInfoOff % 16 == 0 && kFlagOff % 4 == 0,
                "alignment");
};
constexpr int kSoftWarps = 8, kMmaWarp = 8, kCopyWarp = 9, kPlanWarp = 11;
constexpr int kAttnThreads = 384;             // warp 10 only gives its registers away
// A row's 128 logits stay in registers: the softmax warps take 216 each and the
// others 72, of the 168 a thread that the block is launched with:
// 256 x 216 + 128 x 72 = 384 x 168.
constexpr int kRegsSoft = 216, kRegsRest = 72;
constexpr uint32_t kSCol = 0, kOCol = 256;  // S (and P) of A, B at 0, 128; O at 256, 384
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;                // how far a row's maximum may pass its reference (base 2)
constexpr float kMostSum = 1.f / 8192;      // 128 weights of 2^(kLazy - kHeadroom)
constexpr float kBig = 268435456.f;         // from references of 2^28 on, x c - M is taken as (x - max) c

// Two fp32 values as one register pair: packed arithmetic of sm_100 and later.
KVP_DEV uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
KVP_DEV void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
KVP_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
KVP_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
KVP_DEV uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Loads 128 consecutive fp32 columns of this warp's 32 TMEM lanes (one row per thread) in one round and waits for them,
// in one asm block so that no use can move above the wait.
KVP_DEV void tmem_ld128(uint32_t taddr, float (&v)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]),
        "=f"(v[64]), "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]),
        "=f"(v[72]), "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]),
        "=f"(v[80]), "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]),
        "=f"(v[88]), "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]),
        "=f"(v[96]), "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]),
        "=f"(v[104]), "=f"(v[105]), "=f"(v[106]), "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]),
        "=f"(v[112]), "=f"(v[113]), "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]), "=f"(v[119]),
        "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]), "=f"(v[126]), "=f"(v[127])
      : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
      : "memory");
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

// Searches row t of a V tile (swizzled boxes) for infinities and NaN (exponents of ones), and makes them zeros; if the row
// is one of the sequence (`inside`), both tiles' flags get `tag` first.
template <int D>
KVP_DEV void clear_bad_values(uint8_t* tile, int t, bool inside, volatile int* flags, int tag) {
  using C = AttnCfg<D>;
  auto at = [&](int c) {
    return reinterpret_cast<uint4*>(tile + (c >> 3) * C::kBoxBytes + t * 128 + (((c & 7) ^ (t & 7)) << 4));
  };
  uint32_t found = 0;
#pragma unroll 8
  for (int c = 0; c < D / 8; ++c) {
    const uint4 w = *at(c);
    found |= ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
             ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
  }
  if ((found & 0x80008000u) == 0u) return;
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

// mbar_wait for warps that wait while others of their scheduler compute: a probe may suspend the warp for a microsecond
// (it wakes when the phase completes), so that a waiting warp takes no issue slots, and the flag that ends all waits is
// looked at after a failed probe only.
KVP_DEV bool wait_quietly(uint64_t* bar, uint32_t parity, const volatile int* abort, const volatile int32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (done) return true;
    if ((i & 63u) == 63u) {
      if (*abort) return false;
      if (status != nullptr && *status == KVP_ERR_TIMEOUT) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        return false;
      }
    }
  }
}

// One lane of a converged warp, and products and commits that this lane issues (`leader` nonzero there alone).
KVP_DEV uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
KVP_DEV void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(leader)
      : "memory");
}
KVP_DEV void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(leader)
      : "memory");
}
KVP_DEV void commit_to(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

struct AttnMaps {
  CUtensorMap q, k, v;  // [D, heads, rows], boxes of 64 x 1 x 128
};

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1) prompt_attn_kernel(const PromptParams p,
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
  uint64_t* s_full = empty + C::kPairs;  // [A, B]
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* fin = o_full + 2;
  uint64_t* info_full = fin + 1;
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
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(fin, 1);
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&info_full[i], 1);
      mbar_init(&info_empty[i], kSoftWarps + 2);
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
  const bool by_head = p.G % 2 == 0;
  const int cols = by_head ? p.Hq / 2 : p.Hq;  // work items of one tile
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
    t.hA = by_head ? 2 * v.w : v.w;
    t.hB = by_head ? 2 * v.w + 1 : v.w;
    t.nA = t.tA + 1;
    t.nB = t.tB * kTile < t.len ? t.tB + 1 : 0;
    return true;
  };
  Item t;
  bool ok = true;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kPlanWarp) {
      // ------------------------------------------------------------ work items
      const TileOrder order(p.seqs, by_head ? kTile : 2 * kTile);
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
      auto load = [&](const CUtensorMap* m, uint8_t* dst, int head, int row, uint64_t* bar) {
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b) tma_load_3d(dst + b * C::kBoxBytes, m, 64 * b, head, row, bar);
      };
      for (; next_item(i, t, ok); ++i) {
        const int kv = t.hA / p.G, n = max(t.nA, t.nB);
        if (lane == 0) {
          for (int k = 0; ok && k < 2 * n; ++k) {  // K of block 0, V of block 0, K of block 1, ...
            const int st = g % C::kStages;
            if (g >= C::kStages) {  // tile g - kStages is given back with the pair (V of a block, K of the next) that it is of
              const int pair = (g - C::kStages + 1) / 2;
              ok = wait(&empty[pair % C::kPairs], (pair / C::kPairs) & 1);
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
        if (!ok) {
          gave_up();
          break;
        }
      }
      if (lane == 0 && g > 0) {
        if (ok) {  // no arrival is left on its way when the CTA ends
          ok = wait(q_empty, (i - 1) & 1);
          for (int pair = max(0, (g - C::kStages + 1) / 2); ok && pair <= g / 2; ++pair)
            ok = wait(&empty[pair % C::kPairs], (pair / C::kPairs) & 1);
        }
        // what was issued lands before the shared memory can go to another CTA (each wait bounded again)
        if (!ok) {
          if (nq > 0) (void)mbar_wait(q_full, (nq - 1) & 1);
          for (int k = max(0, g - C::kStages); k < g; ++k) (void)mbar_wait(&full[k % C::kStages], (k / C::kStages) & 1);
        }
      }
      __syncwarp();
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
        const uint32_t d = tmem + kSCol + x * kTile;
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
                  mma_ts(leader, tmem + kOCol + x * 128, tmem + kSCol + x * kTile + ks * 8, v0 + ((ks * 2048) >> 4), idO,
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
    const uint32_t scol = trow + kSCol + x * kTile, ocol = trow + kOCol + x * 128;
    const float c = p.qscale;
    uint32_t sph = 0, oph = 0;  // phases of s_full and o_full
    uint32_t g = 0;             // tiles of K and V before this item
    for (int i = 0; next_item(i, t, ok); ++i) {
      const int nx = x == 0 ? t.nA : t.nB, tile = x == 0 ? t.tA : t.tB, head = x == 0 ? t.hA : t.hB;
      const int pos = tile * kTile + row;  // in the sequence; past its end: nothing is stored
      volatile int* flags = bad_values + i % kFlags * 2;
      float M = -INFINITY, m = -INFINITY, l = 0.f;
      for (int j = 0; j < nx; ++j) {
        ok = wait_all(&s_full[x], sph);
        sph ^= 1;
        if (!ok) break;
        tc_fence_after();
        float s[kTile];
        tmem_ld128(scol, s);
        if (j == nx - 1) {
#pragma unroll
          for (int k = 0; k < kTile; ++k)
            if (k > row) s[k] = -INFINITY;
        }
        uint64_t sum[4];
        // With the reference as it is: no maximum is taken. If a row's sum says that some weight may have passed it by
        // 2^8 (or is no number, or the row has no reference yet), the block is taken again below.
        bool again = M == -INFINITY || fabsf(M) >= kBig;
        if (!__any_sync(0xffffffffu, again)) {
          weigh_block(s, c, -M, scol, sum);
          float e, f;
          unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), e, f);
          again = !(e + f <= kMostSum);
        }
        if (__any_sync(0xffffffffu, again)) {
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < kTile; ++i) mx = fmaxf(mx, s[i]);
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
          const float ref = M == -INFINITY ? 0.f : M;
          sum[0] = sum[1] = sum[2] = sum[3] = 0;
#pragma unroll
          for (int o = 0; o < kTile; o += 32) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float a0 = s[o + 2 * i], a1 = s[o + 2 * i + 1];
              const float e = ex2_approx(big ? fmaf(a0 - m, c, -kHeadroom) : fmaf(a0, c, -ref));
              const float f = ex2_approx(big ? fmaf(a1 - m, c, -kHeadroom) : fmaf(a1, c, -ref));
              sum[i & 3] = add2(sum[i & 3], pack2(e, f));
              w[i] = bf16x2(e, f);
            }
            tmem_st16(scol + o / 2, w);
          }
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
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      g += 2 * max(t.nA, t.nB);
      if (!ok) break;
      if (nx == 0) continue;
      ok = wait_all(&o_full[x], oph);
      oph ^= 1;
      if (!ok) break;
      tc_fence_after();
      const bool some = flags[x] == i + 1;
      const bool mine = pos < t.len;
      const int64_t r = t.start + pos;
      uint16_t* out = p.out + r * p.ot + head * p.oh;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int o = 0; o < D; o += 32) {
        float v[32];
        tmem_ld32(ocol + o, v);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = l == 0.f ? 0.f : v[k] * inv;
        if (some && mine)
          add_bad_values(v, p.v + (t.start + t.tA * kTile) * p.vt + head / p.G * p.vh + o, p.vt, pos - t.tA * kTile);
        if (mine) {
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            *reinterpret_cast<uint4*>(out + o + k) =
                make_uint4(bf16x2(v[k], v[k + 1]), bf16x2(v[k + 2], v[k + 3]), bf16x2(v[k + 4], v[k + 5]),
                           bf16x2(v[k + 6], v[k + 7]));
        }
      }
      tc_fence_before();  // O has been read: the next item's products may overwrite it once its P is there
      if (mine && p.lse != nullptr) {
        // the reference and the sum's logarithm; a big one as it was taken
        const float ref = fabsf(M) >= kBig ? m * c + kHeadroom : M;
        p.lse[head * p.seqs.n_tok + r] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
      }
    }
    if (!ok) gave_up();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows of bf16 [rows, heads, D] with the given strides as a tensor map whose boxes are 128 rows x 64 columns of a head.
template <int D>
bool make_tmap_heads(CUtensorMap* m, const void* base, int64_t rows, int64_t st, int heads, int64_t sh) {
  auto fn = tmap_encode_fn();
  if (fn == nullptr) return false;
  if (heads == 1) sh = D;
  if (rows == 1) st = D;
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(sh) * 2, static_cast<cuuint64_t>(st) * 2};
  const cuuint32_t box[3] = {64, 1, kTile};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  const bool by_head = p.G % 2 == 0;
  const int64_t most = (p.seqs.n_tok / (by_head ? kTile : 2 * kTile) + p.seqs.n) * (by_head ? p.Hq / 2 : p.Hq);
  return launch_pdl(prompt_attn_kernel<D>, dim3(static_cast<unsigned>(std::min<int64_t>(sms, most))), dim3(kAttnThreads),
                    C::kSmem, st, p, maps) == cudaSuccess
             ? KVP_OK
             : KVP_ERR_CUDA;
}

template <int D>
__global__ void __launch_bounds__(kPWarps * 32) prompt_weights_kernel(const PromptParams p) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  Tile t;
  if (!find_tile(p.seqs, kTile, blockIdx.x, t)) return;
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
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return head_dim == 128 ? launch_attn<128>(p, n_kv_heads, cs) : launch_attn<64>(p, n_kv_heads, cs);
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
