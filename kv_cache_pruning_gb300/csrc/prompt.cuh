// What the two calls over packed prompts share: sequences and their tiles in the
// order of work, packed fp32 arithmetic, tensor-memory loads, products issued by
// one lane of a converged warp, waits, tensor maps, argument checks.
#pragma once

#include "kvp_common.cuh"

namespace kvp {
namespace {

constexpr int kTile = 128;       // rows of a sequence that one product takes
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
// A weight is held as 2^(x - reference - kHeadroom). The attention lets the reference lag while a block's 128 weights come to
// 2^-13 or less, so that 2^12 blocks of values of any bf16 size (2^19 keys) sum up to 2^127 at most.
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

// A sequence's rows by its own numbers, or -1 where they break the rules.
KVP_DEV int seq_rows(const Seqs& s, int i, int& start) {
  start = s.start[i];
  const int end = s.start[i + 1];
  if (start >= 0 && end >= start && end <= s.n_tok) {
    const int len = s.len != nullptr ? s.len[i] : end - start;
    if (len >= 0 && len <= end - start) return len;
  }
  return -1;
}

// The sequences' tiles of `tile` rows from the longest work to the shortest: by their number in their sequence, the last
// ones first, and sequence by sequence among equal ones (a whole warp calls these).
struct TileOrder {
  const Seqs& s;
  int tile, total, most;
  int mine, my_start, my_len;  // with 32 sequences at most: this lane's
  // Some sequence breaks the rules (recorded). Only then may a later one's rows start before an earlier one's end: without a
  // step down, starts and ends ascend. So only then is each held against where the rows before it reach.
  bool broken = false;
  KVP_DEV TileOrder(const Seqs& seqs, int tile_) : s(seqs), tile(tile_) {
    const int lane = threadIdx.x & 31;
    int sum = 0, top = 0, reach = 0;
    bool bad = false;
    for (int i = lane; i < s.n; i += 32) {
      my_len = seq_rows(s, i, my_start);
      bad |= my_len < 0;
      mine = (my_len + tile - 1) / tile;
      sum += mine;
      top = max(top, mine);
    }
    if (lane >= s.n) mine = my_len = my_start = 0;
    broken = __any_sync(0xffffffffu, bad);
    if (broken) {
      if (lane == 0) record_error(s.status, KVP_ERR_BOUNDS);
      sum = top = 0;
      for (int base = 0; base < s.n; base += 32) {
        mine = look_up(base + lane, my_start, my_len, reach);
        sum += mine;
        top = max(top, mine);
      }
    }
    total = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, top);
  }
  // Tiles of sequence i, this lane's of a round of 32, whose rows start at `start`: none if it breaks the rules or has rows of
  // an earlier one's. reach: where the rows of all rounds before end, then those of this one too.
  KVP_DEV int look_up(int i, int& start, int& len, int& reach) const {
    start = 0;
    len = i < s.n ? max(0, seq_rows(s, i, start)) : 0;
    if (broken) {
      const int lane = threadIdx.x & 31;
      int far = len > 0 ? start + len : 0;  // the furthest end up to this lane's
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, far, o);
        if (lane >= o) far = max(far, y);
      }
      int before = __shfl_up_sync(0xffffffffu, far, 1);
      before = lane == 0 ? reach : max(before, reach);
      reach = max(reach, __shfl_sync(0xffffffffu, far, 31));
      if (start < before) len = 0;
    }
    return (len + tile - 1) / tile;
  }
  KVP_DEV int tiles(int i, int& start, int& len, int& reach) const {
    if (s.n <= 32) {
      start = my_start;
      len = my_len;
      return mine;
    }
    return look_up(i, start, len, reach);
  }
  // tiles of number r and above in their sequences
  KVP_DEV int from(int r) const {
    int sum = 0, start, len, reach = 0;
    for (int i = threadIdx.x & 31; i < (s.n + 31) / 32 * 32; i += 32) sum += max(0, tiles(i, start, len, reach) - r);
    return __reduce_add_sync(0xffffffffu, sum);
  }
  // Tile idx of the order, idx < total and no less than in the call before: the search goes on from there, so that a
  // CTA's items together cost one walk over the sequences for each number that its tiles have.
  int r = 0, above = 0, end = 0;  // tiles of number r are those from `above` to `end` (end 0: no call yet)
  int base = 0, passed = 0;       // of sequence `base` on: `passed` of them lie before
  int reached = 0;                // where the rows of those before `base` end
  KVP_DEV Tile find(int idx) {
    if (idx >= end) {
      int lo = 0, hi = end > 0 ? r : most;
      above = end;
      end = total;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2, f = from(mid);
        if (f > idx) {
          lo = mid;
          end = f;
        } else {
          hi = mid;
          above = f;
        }
      }
      r = lo;
      base = passed = reached = 0;
    }
    const int lane = threadIdx.x & 31;
    for (; base < s.n; base += 32) {
      int start = 0, len = 0, next = reached;
      const uint32_t has = __ballot_sync(0xffffffffu, tiles(base + lane, start, len, next) > r);
      const int left = idx - above - passed;
      if (left < __popc(has)) {
        const int src = __fns(has, 0, left + 1);
        return Tile{base + src, __shfl_sync(0xffffffffu, start, src), __shfl_sync(0xffffffffu, len, src), r};
      }
      passed += __popc(has);
      reached = next;
    }
    return Tile{0, 0, 0, r};
  }
};

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
KVP_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Loads 128 (64) consecutive fp32 columns of this warp's 32 TMEM lanes (one row per thread) in one round and waits for them,
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

KVP_DEV void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]),
        "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]),
        "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]),
        "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]),
        "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
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

// Rows of bf16 [rows, heads, D] with the given strides as a tensor map whose boxes are box_rows rows x 64 columns
// of a head.
template <int D>
bool make_tmap_heads(CUtensorMap* m, const void* base, int64_t rows, int64_t st, int heads, int64_t sh,
                     int box_rows = kTile) {
  auto fn = tmap_encode_fn();
  if (fn == nullptr) return false;
  if (heads == 1) sh = D;
  if (rows == 1) st = D;
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(sh) * 2, static_cast<cuuint64_t>(st) * 2};
  const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  if (scale > 0x1p127f) return KVP_ERR_UNSUPPORTED;  // times log2 e it would be infinite, and 0 times that NaN
  if (head_dim != 64 && head_dim != 128) return KVP_ERR_UNSUPPORTED;
  if (n_q_heads % n_kv_heads != 0) return KVP_ERR_INVALID;
  // (a tile behind the last row is an int, and so is a round of sequences behind the last one)
  if (n_q_heads > 65535 || n_tok > 0x7fff0000ll || n_seqs > 0x7fff0000) return KVP_ERR_UNSUPPORTED;
  if (n_seqs > 0 && n_tok > 0 && seq_start == nullptr) return KVP_ERR_INVALID;
  if (!aligned4(seq_start) || !aligned4(seq_len)) return KVP_ERR_ALIGN;
  return KVP_OK;
}

}  // namespace
}  // namespace kvp
