"""The block-scaled 8-bit cache on the GPU against the float64 restatement: bulk write, append, read back and
attention, alone and together."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import block8_ref as ref
import kvp_synth as syn
from helpers import dev_bf16, dev_f32, dev_i32, host_bits, status_word

pytestmark = pytest.mark.gpu
FMTS = [ref.E4M3, ref.INT8]


# ---------------------------------------------------------------------------- helpers

def _bits(seed, shape, spread=0):
    """bf16 bits: normals, their magnitudes spread over 2^-spread .. 2^spread from row to row."""
    x = syn.normal_f32(seed, 301, shape)
    if spread:
        u = syn.normal_f32(seed, 302, shape[:-1] + (1,))
        x = x * np.exp2(np.clip(u * spread, -3 * spread, 3 * spread)).astype(np.float32)
    return syn.f32_to_bf16_bits(x.astype(np.float32))


def _alloc(kvp, B, H, d, cap, width, fmt):
    return kvp.Block8PagedKV.allocate(B, H, d, cap, width, fmt=fmt)


def _check_cache(cache, heads, fmt, reserve=None, pages=None):
    """Bit for bit: codes, scales, expire values, tables and counts of the cache against Head[b][h]; with `reserve`
    (right after a bulk write) also the page ids and the zeroed rest of each (b, h)'s pages."""
    kq, vq = cache.kq_pool.cpu().numpy(), cache.vq_pool.cpu().numpy()
    scale, expire = cache.scale_pool.cpu().numpy(), cache.expire_pool.cpu().numpy()
    table, remap, count = cache.page_table.cpu().numpy(), cache.remap.cpu().numpy(), cache.count.cpu().numpy()
    base = 0
    for b, row in enumerate(heads):
        for h, head in enumerate(row):
            n = head.count
            assert count[b, h] == n
            np.testing.assert_array_equal(remap[b, h, :n], head.pos)
            used = (n + 15) // 16
            if reserve is not None:
                used = (n + reserve + 15) // 16
                np.testing.assert_array_equal(table[b, h], [base + p if p < used else -1 for p in range(table.shape[2])])
                assert (remap[b, h, n:] == -1).all()
                base += used
            for p in range(used):
                pg, m = table[b, h, p], min(max(n - p * 16, 0), 16)
                np.testing.assert_array_equal(kq[pg, :m], head.codes[0][p * 16:p * 16 + m])
                np.testing.assert_array_equal(vq[pg, :m], head.codes[1][p * 16:p * 16 + m])
                np.testing.assert_array_equal(expire[pg, :m], head.expire[p * 16:p * 16 + m])
                if m:
                    assert tuple(scale[pg]) == (head.scales[0][p], head.scales[1][p]), (b, h, p)
                if reserve is not None:
                    assert not kq[pg, m:].any() and not vq[pg, m:].any() and not expire[pg, m:].any()
                    if m == 0:
                        assert not scale[pg].any()
    return base


def _inputs(mode, seed, B, T, H, now):
    """(scores, tau, flag) of a mask mode."""
    if mode == 0:
        return syn.normal_f32(seed, 311, (B, T, H)), syn.normal_f32(seed, 312, (B, H), std=0.5), None
    u = syn.normal_f32(seed, 313, (B, H, T))
    age = (np.abs(syn.normal_f32(seed, 314, (B, H, T))) * max(T, 2) / 2).astype(np.int32) % max(now + 1, 1)
    return None, None, np.where(u < 0.3, age, -1).astype(np.int32)


def _build(kvp, fmt, seed, B, T, H, d, keep_all=False, reserve=0, spread=1, shuffle=True, spare=0):
    """A cache written by the library and its Head[b][h], pages moved to shuffled ids."""
    k, v = _bits(seed, (B, T, H, d), spread), _bits(seed + 1, (B, T, H, d), spread)
    now = T - 1
    scores = syn.normal_f32(seed, 321, (B, T, H))
    tau = np.full((B, H), -9.0, np.float32) if keep_all else syn.normal_f32(seed, 322, (B, H), std=0.5)
    heads = ref.compact(fmt, 0, ref.widen(k), ref.widen(v), now, 8, 0, scores, tau)
    width = (T + reserve + 15) // 16 + spare
    cap = B * H * width + 3
    cache = _alloc(kvp, B, H, d, cap, width, fmt)
    st = status_word()
    kvp.kvp_compact_block8(dev_bf16(k), dev_bf16(v), now, reserve, cache, mode=0, scores=dev_f32(scores),
                           tau=dev_f32(tau), window=8, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    _check_cache(cache, heads, fmt, reserve)
    if shuffle:
        perm = torch.from_numpy(np.random.default_rng(seed).permutation(cap)).cuda()
        for t in (cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool):
            t[perm] = t.clone()
        on = cache.page_table >= 0
        cache.page_table[on] = perm[cache.page_table[on].long()].int()
    return cache, heads, now


def _attend(kvp, cache, heads, q_bits, now, scale=0.0, **kw):
    """Runs the attention and compares it, element by element, with the restatement."""
    B, Hq, d = q_bits.shape
    H = len(heads[0])
    G = Hq // H
    lse = torch.full((B, Hq), 7.0, device="cuda")
    st = status_word()
    out = kvp.kvp_decode_attn_block8(dev_bf16(q_bits), cache, now, scale=scale, lse=lse, status=st, **kw)
    torch.cuda.synchronize()
    assert st.item() == 0
    _compare(out, lse, heads, ref.widen(q_bits), now, scale or 1 / math.sqrt(d), G)
    return out, lse


def _compare(out, lse, heads, q, now, scale, G):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, row in enumerate(heads):
        for h, head in enumerate(row):
            sl = slice(h * G, (h + 1) * G)
            want, wlse, size_abs, size = head.attend(q[b, sl], now, scale)
            tol, tol_lse = ref.attention_bounds(q.shape[2], head.count, size_abs, size)
            off = np.abs(out[b, sl] - want)
            assert (off <= tol).all(), (b, h, float((off / tol).max()))
            if np.isinf(wlse).any():
                assert (lse[b, sl] == wlse).all()
            else:
                assert (np.abs(lse[b, sl] - wlse) <= tol_lse + np.abs(wlse) * 2.0**-22).all(), (b, h)


# ---------------------------------------------------------------------------- bulk write

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mode,B,T,H,d,window,delay,reserve", [
    (0, 1, 1, 1, 64, 128, 0, 0),
    (0, 2, 15, 3, 128, 4, 0, 1),
    (1, 1, 16, 2, 64, 0, 0, 0),
    (0, 3, 17, 1, 128, 0, 0, 16),
    (1, 2, 129, 5, 64, 16, 7, 33),
    (0, 2, 700, 4, 128, 128, 0, 5),
    (1, 1, 1300, 2, 128, 128, 50, 0),
    (0, 520, 37, 2, 64, 3, 0, 2),        # above 1,024 (b, h): the separate page-base pass
    (0, 1, 1024, 32, 128, 30, 0, 3),     # the most a single launch takes
    (0, 64, 256, 2, 64, 30, 0, 3),
    (1, 1, 1025, 3, 64, 30, 5, 40),      # a position more: the passes
    (0, 129, 110, 1, 64, 20, 0, 0),      # a (b, h) more: the passes
    (1, 2, 1537, 5, 128, 0, 0, 17),
    (0, 2, 1100, 15, 64, 60, 0, 3),      # heads one by one ..
    (0, 2, 1111, 16, 64, 200, 0, 3),     # .. and side by side: half a warp of them
    (0, 1, 1057, 33, 64, 5, 0, 0),       # a warp and one
    (0, 33, 31, 70, 64, 8, 0, 1),        # the same with the page-base pass
    (0, 1, 4096, 3, 64, 128, 0, 2),      # the most positions whose counts need no zeroing
    (0, 1, 4097, 3, 64, 128, 0, 2),      # a position more
    (1, 2, 4200, 2, 64, 128, 9, 0),
    (1, 57, 1030, 3, 64, 40, 9, 0),      # a (b, h) more: 513 sums
])
def test_bulk_write_is_bit_exact(kvp, fmt, mode, B, T, H, d, window, delay, reserve):
    now = T - 1
    k, v = _bits(11, (B, T, H, d), 3), _bits(12, (B, T, H, d), 3)
    scores, tau, flag = _inputs(mode, 13, B, T, H, now)
    width = (T + reserve + 15) // 16
    cap = B * H * width
    cache = _alloc(kvp, B, H, d, cap, width, fmt)
    for t in (cache.kq_pool, cache.vq_pool):
        t.fill_(0x7F)                     # what the pools held before does not show
    cache.scale_pool.fill_(3.0)
    cache.expire_pool.fill_(9)
    cache.count.fill_(-5)
    st = status_word()
    opt = lambda a, f: None if a is None else f(a)  # noqa: E731
    kvp.kvp_compact_block8(dev_bf16(k), dev_bf16(v), now, reserve, cache, mode=mode, scores=opt(scores, dev_f32),
                           tau=opt(tau, dev_f32), flag_step=opt(flag, dev_i32), window=window, delay=delay, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    heads = ref.compact(fmt, mode, ref.widen(k), ref.widen(v), now, window, delay, scores, tau, flag)
    used = _check_cache(cache, heads, fmt, reserve)
    assert (cache.kq_pool[used:] == 0x7F).all() and (cache.scale_pool[used:] == 3.0).all()   # pages behind: untouched
    # the bf16 compaction's tables, bit for bit
    bf = kvp.PagedKV.allocate(B, H, d, cap, width)
    kvp.kvp_compact_masked(dev_bf16(k), dev_bf16(v), now, reserve, bf, mode=mode, scores=opt(scores, dev_f32),
                           tau=opt(tau, dev_f32), flag_step=opt(flag, dev_i32), window=window, delay=delay, status=st)
    for a, b in ((cache.count, bf.count), (cache.page_table, bf.page_table), (cache.remap, bf.remap)):
        assert torch.equal(a, b)
    assert torch.equal(cache.expire_pool[:used], bf.expire_pool[:used])


@pytest.mark.parametrize("H", [3, 18])
@pytest.mark.parametrize("window", [0, 100])
def test_bulk_write_of_unusual_scores(kvp, H, window):
    """Scores and thresholds that are NaN, infinite, zeros of both signs, or equal."""
    T, d, fmt = 1090, 64, ref.E4M3
    odd = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 0.5, np.float32(2**-149), -1.0], np.float32)
    scores = odd[(np.abs(syn.normal_f32(81, 331, (1, T, H))) * 1000).astype(int) % 8]
    tau = odd[np.arange(H) % 8][None]
    x = _bits(82, (1, T, H, d))
    cache = _alloc(kvp, 1, H, d, 69 * H, 69, fmt)
    st = status_word()
    kvp.kvp_compact_block8(dev_bf16(x), dev_bf16(x), T - 1, 0, cache, mode=0, scores=dev_f32(scores), tau=dev_f32(tau),
                           window=window, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    w = ref.widen(x)
    _check_cache(cache, ref.compact(fmt, 0, w, w, T - 1, window, 0, scores, tau), fmt, 0)


@pytest.mark.parametrize("fmt", FMTS)
def test_bulk_write_of_strided_and_empty_sources(kvp, fmt):
    B, T, H, d = 2, 45, 3, 64
    k, v = _bits(21, (B, H, T, d)), _bits(22, (B, H, T, d))
    heads = ref.compact(fmt, 0, ref.widen(k).transpose(0, 2, 1, 3), ref.widen(v).transpose(0, 2, 1, 3), T - 1, 9, 0,
                        np.ones((B, T, H), np.float32), np.zeros((B, H), np.float32))
    cache = _alloc(kvp, B, H, d, 64, 4, fmt)
    st = status_word()
    one, zero = torch.ones(B, T, H, device="cuda"), torch.zeros(B, H, device="cuda")
    kvp.kvp_compact_block8(dev_bf16(k).transpose(1, 2), dev_bf16(v).transpose(1, 2), T - 1, 0, cache, mode=0, scores=one,
                           tau=zero, window=9, status=st)
    torch.cuda.synchronize()
    _check_cache(cache, heads, fmt, 0)
    # no positions at all: counts 0, only the reserve's pages
    empty = torch.zeros(B, 0, H, d, dtype=torch.bfloat16, device="cuda")
    kvp.kvp_compact_block8(empty, empty, 0, 20, cache, mode=0, scores=one[:, :0], tau=zero, status=st)
    torch.cuda.synchronize()
    _check_cache(cache, [[ref.Head(d, fmt) for _ in range(H)] for _ in range(B)], fmt, 20)
    # every position dropped
    kvp.kvp_compact_block8(dev_bf16(k).transpose(1, 2), dev_bf16(v).transpose(1, 2), T + 8, 0, cache, mode=0,
                           scores=one, tau=zero + 2, window=9, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and not cache.count.any() and (cache.page_table == -1).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_bulk_write_of_unusual_values(kvp, fmt):
    """Pages of zeros, of bf16 subnormals, of the largest numbers, at the formats' borders, with infinities and NaNs."""
    rows = [0x0000, 0x8000, 0x0001, 0x007F, 0x0080, 0x7F7F, 0xFF7F, 0x43E0, 0x43E1, 0x42FE, 0x42FF, 0x4300, 0x7F80, 0xFF80,
            0x7FC0, 0x3F80, 0x3C00, 0xBF80]
    T, d = 16 * len(rows), 64
    base = _bits(31, (1, T, 1, d))
    k = base.copy()
    for i, w in enumerate(rows):
        page = k[0, 16 * i:16 * i + 16, 0]
        if i < 11 or i in (15,):
            page[:] = 0 if i != 15 else w
        page[3, 5] = w                     # one value of each page
        page[15, 63] = w ^ 0x8000
    k[0, 16 * 12:16 * 13, 0, 7] = 0x7F80   # infinities beside finite values
    v = np.ascontiguousarray(k[:, ::-1])
    cache = _alloc(kvp, 1, 1, d, len(rows), len(rows), fmt)
    st = status_word()
    kvp.kvp_compact_block8(dev_bf16(k), dev_bf16(v), T - 1, 0, cache, mode=1,
                           flag_step=torch.full((1, 1, T), -1, dtype=torch.int32, device="cuda"), status=st)
    torch.cuda.synchronize()
    heads = ref.compact(fmt, 1, ref.widen(k), ref.widen(v), T - 1, 128, 0, flag=np.full((1, 1, T), -1))
    if fmt == ref.E4M3:                    # a NaN's sign is not part of the format's meaning
        for t in (cache.kq_pool, cache.vq_pool):
            t[(t & 0x7F) == 0x7F] = 0x7F
    _check_cache(cache, heads, fmt, 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [200, 1040])
def test_bulk_writes_back_to_back(kvp, fmt, T):
    """Many writes one behind the other, each into memory that the ones before it used, inputs made just before: every
    pass sees what the launches before it wrote."""
    H, d = 2, 64
    made = []
    for seed in (0, 1):
        k, v, sc = _bits(401 + seed, (1, T, H, d), 3), _bits(403 + seed, (1, T, H, d), 3), syn.normal_f32(seed, 405, (1, T, H))
        heads = ref.compact(fmt, 0, ref.widen(k), ref.widen(v), T - 1, 40, 0, sc, np.zeros((1, H), np.float32))
        made.append((k, v, sc, heads))
    for i in range(60):
        k, v, sc, heads = made[i % 2]
        cache = _alloc(kvp, 1, H, d, 69 * H, 69, fmt)
        st = status_word()
        kvp.kvp_compact_block8(dev_bf16(k), dev_bf16(v), T - 1, 0, cache, mode=0, scores=dev_f32(sc),
                               tau=torch.zeros(1, H, device="cuda"), window=40, status=st)
        _check_cache(cache, heads, fmt, 0)
        assert st.item() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_steps_back_to_back_give_the_bits_of_steps_apart(kvp, fmt):
    """Rotation, append and attention of 60 steps launched without a pause, and again with the GPU waited for after
    every call."""
    B, H, G, d, steps = 4, 8, 4, 128, 60
    got = []
    turns = kvp.kvp_rope_turns(10000.0 ** (-np.arange(0, d, 2) / d))
    x = dev_bf16(_bits(411, (steps, B, H * (G + 2), d), 1))
    flag = torch.full((B, H), -1, dtype=torch.int32, device="cuda")
    for wait in (torch.cuda.synchronize, lambda: None):
        cache, _, now = _build(kvp, fmt, 412, B, 100, H, d, reserve=steps)
        ws = torch.zeros(kvp.kvp_decode_attn_block8_workspace_bytes(B, H * G, H, d), dtype=torch.uint8, device="cuda")
        q, k = torch.empty_like(x[0, :, :H * G]), torch.empty_like(x[0, :, :H])
        pos = (now + 1 + torch.arange(steps, device="cuda", dtype=torch.int32))[:, None].repeat(1, B)
        out, st = torch.empty(steps, B, H * G, d, device="cuda"), status_word()
        torch.cuda.synchronize()
        for i in range(steps):
            kvp.kvp_qk_norm_rope(x[i, :, :H * G], x[i, :, H * G:H * (G + 1)], pos[i], turns, q_out=q, k_out=k)
            wait()
            kvp.kvp_append_block8(cache, k, x[i, :, H * (G + 1):], now + 1 + i, mode=1, flag_step=flag, status=st)
            wait()
            kvp.kvp_decode_attn_block8(q, cache, now + 1 + i, out=out[i], workspace=ws, status=st)
            wait()
        torch.cuda.synchronize()
        assert st.item() == 0
        got.append((out, cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,T", [(2, 100), (2, 1100), (2, 4200), (600, 20)])   # one launch, the passes, the page-base pass
def test_bulk_write_records_a_full_pool(kvp, B, T):
    H, d = 2, 64
    each = (T + 15) // 16
    k = dev_bf16(_bits(41, (B, T, H, d)))
    flag = torch.full((B, H, T), -1, dtype=torch.int32, device="cuda")
    for cap, width in ((B * H * each - 1, each), (B * H * each, each - 1)):      # one page short; a table one page short
        cache = _alloc(kvp, B, H, d, cap, width, 0)
        st = status_word()
        kvp.kvp_compact_block8(k, k, T - 1, 0, cache, mode=1, flag_step=flag, status=st)
        torch.cuda.synchronize()
        assert st.item() == kvp.KVP_ERR_CAPACITY
        assert not cache.kq_pool.any() and not cache.scale_pool.any()


# ---------------------------------------------------------------------------- append

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,H,d,T", [(1, 1, 64, 1), (2, 3, 128, 30), (5, 2, 64, 16)])
def test_append_is_bit_exact(kvp, fmt, B, H, d, T):
    steps = 37
    cache, heads, now = _build(kvp, fmt, 51, B, T, H, d, reserve=steps)
    st = status_word()
    pos_dev = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(steps):
        pos = now + 1 + i
        # magnitudes that rise and fall from step to step, zero rows among them
        grow = np.float32(0 if i % 11 == 5 else 2.0 ** ((i * 7) % 13 - 6))
        both = syn.f32_to_bf16_bits((syn.normal_f32(60 + i, 331, (B, 2 * H, d)) * grow).astype(np.float32))
        kb, vb = both[:, :H], both[:, H:]
        dev = dev_bf16(both)               # views of one projection's output
        mode = i % 2
        score, tau = syn.normal_f32(i, 332, (B, H)), np.zeros((B, H), np.float32)
        flag = np.where(syn.normal_f32(i, 333, (B, H)) < 0, pos, -1).astype(np.int32)
        kw = dict(mode=0, score=dev_f32(score), tau=dev_f32(tau)) if mode == 0 else dict(mode=1, flag_step=dev_i32(flag))
        if i % 3 == 2:
            pos_dev.fill_(pos)
            kvp.kvp_append_block8_devpos(cache, dev[:, :H], dev[:, H:], pos_dev, window=20, delay=3, status=st, **kw)
        else:
            kvp.kvp_append_block8(cache, dev[:, :H], dev[:, H:], pos, window=20, delay=3, status=st, **kw)
        for b in range(B):
            for h in range(H):
                e = ref.expire_of(mode, pos, 20, 3, score[b, h], tau[b, h], flag[b, h])
                heads[b][h].append(ref.widen(kb[b, h]), ref.widen(vb[b, h]), e, pos)
        if i in (0, 1, 15, 16, steps - 1):
            torch.cuda.synchronize()
            assert st.item() == 0
            _check_cache(cache, heads, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_to_a_page_of_zeros_and_infinities(kvp, fmt):
    """A page without a finite value but zero has scale 0, where an infinity's code is worth 0 like any other; when a row
    gives the page a scale, those rows stay worth 0 (and E4M3's NaN stays NaN)."""
    d = 64
    cache = _alloc(kvp, 1, 1, d, 1, 1, fmt)
    cache.page_table.zero_()
    x = np.zeros((4, 1, 1, d), np.uint16)
    x[0, ..., 3], x[0, ..., 4], x[0, ..., 5] = 0x7F80, 0xFF80, 0x8000       # inf, -inf, -0
    x[1, ..., 7] = 0x7FC0                                                    # NaN
    x[2:] = _bits(73, (2, 1, 1, d))
    heads = [[ref.Head(d, fmt)]]
    flag, st = torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), status_word()
    for i in range(4):
        kvp.kvp_append_block8(cache, dev_bf16(x[i]), dev_bf16(x[i]), i, mode=1, flag_step=flag, status=st)
        w = ref.widen(x[i, 0, 0])
        heads[0][0].append(w, w, ref.NEVER, i)
        torch.cuda.synchronize()
        _check_cache(cache, heads, fmt)
        k, _ = kvp.kvp_read_block8(cache, 0, 2)
        assert not k[0, 0].any() and st.item() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_append_errors_leave_the_head_unchanged(kvp, fmt):
    B, H, d, T = 1, 5, 64, 20
    cache, heads, now = _build(kvp, fmt, 71, B, T, H, d, keep_all=True, reserve=16)
    cache.count[0, 0] = 48                   # its three pages (20 rows and 16 reserved) are full
    cache.count[0, 1] = -1
    cache.page_table[0, 2, 1] = cache.n_pages_cap
    cache.page_table[0, 3, 1] = -1
    before = [t.clone() for t in (cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool, cache.remap)]
    good = int(cache.page_table[0, 4, 1])
    x = dev_bf16(_bits(72, (B, H, d)))
    st = status_word()
    flag = torch.full((B, H), -1, dtype=torch.int32, device="cuda")
    kvp.kvp_append_block8(cache, x, x, now + 1, mode=1, flag_step=flag, status=st)
    torch.cuda.synchronize()
    assert st.item() in (kvp.KVP_ERR_CAPACITY, kvp.KVP_ERR_BOUNDS)
    assert cache.count[0].tolist() == [48, -1, 20, 20, 21]
    for a, b in zip(before, (cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool)):
        keep = torch.arange(a.shape[0], device="cuda") != good
        assert torch.equal(a[keep], b[keep])
    assert torch.equal(before[4][0, :4], cache.remap[0, :4])
    bad = torch.tensor([-1], dtype=torch.int32, device="cuda")    # a position that is none: nothing happens
    st.zero_()
    kvp.kvp_append_block8_devpos(cache, x, x, bad, mode=1, flag_step=flag, status=st)
    torch.cuda.synchronize()
    assert st.item() == kvp.KVP_ERR_INVALID and cache.count[0, 4] == 21


# ---------------------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,H,d,T,first,n", [(1, 1, 64, 1, 0, 1), (2, 3, 128, 77, 0, 90), (3, 2, 64, 50, 5, 11),
                                             (1, 4, 128, 130, 17, 200), (2, 2, 64, 40, 300, 33)])
def test_read_is_exact(kvp, fmt, B, H, d, T, first, n):
    cache, heads, _ = _build(kvp, fmt, 81, B, T, H, d, spread=4)
    st = status_word()
    k, v = kvp.kvp_read_block8(cache, first, n, status=st)
    # the same into strided rows, whose surroundings stay as they are
    wide = torch.full((2, B, H, n + 2, d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    ks, vs = (wide[i, :, :, 1:n + 1, :d].transpose(1, 2) for i in range(2))
    kvp.kvp_read_block8(cache, first, n, k_out=ks, v_out=vs, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert torch.equal(ks, k) and torch.equal(vs, v)
    assert (wide[:, :, :, 0] == 5).all() and (wide[:, :, :, -1] == 5).all() and (wide[..., d:] == 5).all()
    for w, got in ((0, k), (1, v)):
        got = got.double().cpu().numpy()
        for b in range(B):
            for h in range(H):
                want = np.zeros((n, d))
                x = heads[b][h].values(w)[first:first + n]
                want[:len(x)] = x                     # 4 and 7 significant bits: exact in bf16's 8
                np.testing.assert_array_equal(got[b, :, h], want)


def test_read_of_bad_pages_gives_zeros(kvp):
    cache, heads, _ = _build(kvp, 0, 91, 1, 40, 2, 64, keep_all=True)
    cache.page_table[0, 0, 1] = cache.n_pages_cap
    cache.page_table[0, 1, 0] = -7
    cache.count[0, 1] = 10**9                        # clamped to the table
    st = status_word()
    k, v = kvp.kvp_read_block8(cache, 0, 64, status=st)
    torch.cuda.synchronize()
    assert st.item() == kvp.KVP_ERR_BOUNDS
    assert not k[0, 16:32, 0].any() and not v[0, :16, 1].any()
    np.testing.assert_array_equal(k[0, :16, 0].double().cpu().numpy(), heads[0][0].values(0)[:16])
    np.testing.assert_array_equal(k[0, 16:40, 1].double().cpu().numpy(), heads[0][1].values(0)[16:40])
    assert not k[0, 48:].any()                       # past the table
    k, v = kvp.kvp_read_block8(cache, 3, 0)
    assert k.shape == (1, 0, 2, 64)


# ---------------------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,G,T", [(1, 1, 1, 1), (1, 2, 2, 16), (2, 1, 3, 17), (2, 3, 4, 200), (1, 2, 5, 333),
                                     (3, 1, 6, 31), (1, 1, 7, 1000), (2, 2, 8, 129), (4, 8, 1, 257)])
def test_attention(kvp, fmt, d, B, H, G, T):
    cache, heads, now = _build(kvp, fmt, 101 + G, B, T, H, d)
    q = _bits(102, (B, H * G, d))
    base = None
    for limit in (0, 1, 3, 50):                       # the same work cut differently
        out, lse = _attend(kvp, cache, heads, q, now, grid_limit=limit)
        again, lse2 = _attend(kvp, cache, heads, q, now, grid_limit=limit)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        base = out if base is None else base
    _attend(kvp, cache, heads, q, now, scale=0.37)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_of_many_short_heads(kvp, fmt):
    """More (b, h) than warps, some empty; then one long head among empty ones."""
    B, H, d, G = 40, 24, 64, 2
    cache, heads, now = _build(kvp, fmt, 111, B, 21, H, d)
    empty = np.random.default_rng(3).random((B, H)) < 0.3
    cache.count[torch.from_numpy(empty).cuda()] = 0
    for b, h in zip(*np.nonzero(empty)):
        heads[b][h] = ref.Head(d, fmt)
    _attend(kvp, cache, heads, _bits(112, (B, H * G, d)), now)
    cache, heads, now = _build(kvp, fmt, 113, 1, 3000, 6, 128, keep_all=True)
    for h in (0, 1, 3, 4, 5):
        cache.count[0, h] = 0
        heads[0][h] = ref.Head(128, fmt)
    out, lse = _attend(kvp, cache, heads, _bits(114, (1, 24, 128)), now)
    assert not out[0, :8].any() and torch.isneginf(lse[0, :8]).all()


@pytest.mark.parametrize("fmt,d,G", [(ref.E4M3, 128, 8), (ref.INT8, 64, 3)])
def test_attention_of_the_most_heads(kvp, fmt, d, G):
    """4,096 (b, h), the most a call takes."""
    cache, heads, now = _build(kvp, fmt, 115, 64, 3, 64, d)
    cache.count[5, 7:40] = 0
    for h in range(7, 40):
        heads[5][h] = ref.Head(d, fmt)
    _attend(kvp, cache, heads, _bits(116, (64, 64 * G, d)), now)


@pytest.mark.parametrize("fmt,d,G", [(ref.E4M3, 128, 4), (ref.INT8, 64, 6)])
def test_attention_of_one_long_head(kvp, fmt, d, G):
    """2,500 pages of one (b, h): over many CTAs, over a few, and 157 a warp in one."""
    cache, heads, now = _build(kvp, fmt, 117, 1, 40000, 1, d, keep_all=True)
    q = _bits(118, (1, G, d))
    for limit in (0, 5, 1):
        _attend(kvp, cache, heads, q, now, grid_limit=limit)


def test_one_workspace_for_calls_of_any_size(kvp):
    """Few heads, many, and few again: no call's partial results lie where another's arrival counters are."""
    few, few_heads, few_now = _build(kvp, ref.INT8, 127, 1, 4000, 1, 64, keep_all=True)
    many, many_heads, many_now = _build(kvp, ref.E4M3, 128, 40, 300, 4, 128, keep_all=True)
    ws = torch.zeros(max(kvp.kvp_decode_attn_block8_workspace_bytes(1, 8, 1, 64),
                         kvp.kvp_decode_attn_block8_workspace_bytes(40, 16, 4, 128)), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        _attend(kvp, few, few_heads, _bits(129, (1, 8, 64)), few_now, workspace=ws)
        _attend(kvp, many, many_heads, _bits(130, (40, 16, 128)), many_now, workspace=ws)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_writes_its_outputs_only(kvp, fmt):
    """Guard values around the output, the log-sum-exps, the workspace and the cache's buffers."""
    cache, heads, now = _build(kvp, fmt, 119, 2, 700, 3, 64)
    before = [t.clone() for t in (cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool, cache.page_table,
                                  cache.count)]
    q = _bits(120, (2, 15, 64))
    need = kvp.kvp_decode_attn_block8_workspace_bytes(2, 15, 3, 64)
    out, lse = torch.full((2 * 15 * 64 + 256,), 7.0, device="cuda"), torch.full((2 * 15 + 64,), 7.0, device="cuda")
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    ws[256:256 + need] = 0
    o, l = out[128:128 + 1920].view(2, 15, 64), lse[32:62].view(2, 15)
    for limit in (0, 4):
        kvp.kvp_decode_attn_block8(dev_bf16(q), cache, now, out=o, lse=l, workspace=ws[256:256 + need], grid_limit=limit)
        torch.cuda.synchronize()
        _compare(o, l, heads, ref.widen(q), now, 1 / 8, 5)
        assert (out[:128] == 7).all() and (out[128 + 1920:] == 7).all() and (lse[:32] == 7).all() and (lse[62:] == 7).all()
        assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()
        assert not ws[256:256 + 24].any()                # the arrival counters are back at zero
    for a, b in zip(before, (cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool, cache.page_table,
                             cache.count)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 4, 7])
def test_attention_masks(kvp, fmt, G):
    """Expired slots (whose codes may be anything), a row with nothing left, steps on which entries leave."""
    cache, heads, now = _build(kvp, fmt, 121, 2, 150, 2, 128, keep_all=True)
    rng = np.random.default_rng(9)
    table = cache.page_table.cpu().numpy()
    for b in range(2):
        for h in range(2):
            head = heads[b][h]
            gone = rng.random(head.count) < (1.0 if (b, h) == (1, 0) else 0.4)
            for s in np.nonzero(gone)[0]:
                head.expire[s] = int(now - rng.integers(0, 3))
                pg, r = int(table[b, h, s // 16]), int(s % 16)
                cache.expire_pool[pg, r] = head.expire[s]
                if head.expire[s] == now - 2:          # gone at every step below: NaN (E4M3); 127 and -1
                    cache.kq_pool[pg, r] = 0x7F
                    cache.vq_pool[pg, r] = 0xFF
            # behind the last row, too
            n = head.count
            if n % 16:
                pg = int(table[b, h, n // 16])
                cache.vq_pool[pg, n % 16:] = 0x7F
                cache.kq_pool[pg, n % 16:] = 0xFF
                cache.expire_pool[pg, n % 16:] = ref.NEVER
    q = _bits(122, (2, 2 * G, 128))
    for at in (now - 2, now - 1, now, now + 1):
        out, lse = _attend(kvp, cache, heads, q, at)
    assert not out[1, :G].any() and torch.isneginf(lse[1, :G]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_of_large_and_small_magnitudes(kvp, fmt):
    """Queries of very different sizes in one group, sharp softmaxes whose maximum moves late, tiny and huge pages."""
    cache, heads, now = _build(kvp, fmt, 131, 1, 400, 2, 128, keep_all=True, spread=3)
    q = ref.widen(_bits(132, (1, 8, 128)))
    q *= np.array([2.0**-40, 2.0**-3, 1, 4, 2.0**-20, 2, 0, 2.0**-100])[None, :, None]
    qb = syn.f32_to_bf16_bits(q.astype(np.float32))
    _attend(kvp, cache, heads, qb, now)
    _attend(kvp, cache, heads, qb, now, scale=2.0**-12)
    # logits that rise along the sequence by about 3 a token, and the same order backwards
    for flip in (False, True):
        T, d = 200, 64
        ramp = np.arange(T, dtype=np.float64)
        ramp = ramp[::-1] if flip else ramp
        k = np.zeros((1, T, 1, d))
        k[0, :, 0, 0] = ramp
        v = ref.widen(_bits(133, (1, T, 1, d)))
        kb, vb = syn.f32_to_bf16_bits(k.astype(np.float32)), syn.f32_to_bf16_bits(v.astype(np.float32))
        cache = _alloc(kvp, 1, 1, d, 13, 13, fmt)
        st = status_word()
        kvp.kvp_compact_block8(dev_bf16(kb), dev_bf16(vb), T - 1, 0, cache, mode=1,
                               flag_step=torch.full((1, 1, T), -1, dtype=torch.int32, device="cuda"), status=st)
        heads = ref.compact(fmt, 1, ref.widen(kb), ref.widen(vb), T - 1, 128, 0, flag=np.full((1, 1, T), -1))
        q = np.zeros((1, 4, d))
        q[0, :, 0] = [3.0, -3.0, 0.25, 0.0]
        qb = syn.f32_to_bf16_bits(q.astype(np.float32))
        for limit in (0, 1):
            _attend(kvp, cache, heads, qb, T - 1, scale=1.0, grid_limit=limit)


def test_attention_lets_nan_through_where_it_is_present(kvp):
    """A NaN value of a present token shows in its channel and nowhere else; a NaN key or query in its rows."""
    cache, heads, now = _build(kvp, 0, 141, 1, 100, 2, 64, keep_all=True)
    q = dev_bf16(_bits(142, (1, 4, 64)))
    clean = kvp.kvp_decode_attn_block8(q, cache, now)
    pg = int(cache.page_table[0, 1, 2])
    cache.vq_pool[pg, 3, 9] = 0x7F
    out = kvp.kvp_decode_attn_block8(q, cache, now)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 2:, 9]).all()
    out[0, 2:, 9] = clean[0, 2:, 9]
    assert torch.equal(out, clean)
    cache.kq_pool[pg, 3, 9] = 0x7F
    lse = torch.zeros(1, 4, device="cuda")
    out = kvp.kvp_decode_attn_block8(q, cache, now, lse=lse)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all() and torch.equal(out[0, :2], clean[0, :2])
    q[0, 0, 0] = float("nan")
    out = kvp.kvp_decode_attn_block8(q, cache, now)
    assert torch.isnan(out[0, 0]).all() and torch.equal(out[0, 1], clean[0, 1])


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_of_bad_pages(kvp, fmt):
    """A page id out of range is recorded and its slots count as absent; the workspace stays usable."""
    cache, heads, now = _build(kvp, fmt, 151, 2, 100, 2, 64, keep_all=True)
    q = _bits(152, (2, 8, 64))
    ws = torch.zeros(kvp.kvp_decode_attn_block8_workspace_bytes(2, 8, 2, 64), dtype=torch.uint8, device="cuda")
    good = cache.page_table.clone()
    cache.page_table[0, 0, 1] = cache.n_pages_cap
    cache.page_table[1, 1, :] = -1
    st = status_word()
    lse = torch.zeros(2, 8, device="cuda")
    out = kvp.kvp_decode_attn_block8(dev_bf16(q), cache, now, lse=lse, workspace=ws, status=st)
    torch.cuda.synchronize()
    assert st.item() == kvp.KVP_ERR_BOUNDS
    heads[0][0].expire[16:32] = [now] * 16
    heads[1][1].expire = [now] * 100
    _compare(out, lse, heads, ref.widen(q), now, 1 / 8, 4)
    cache.page_table.copy_(good)
    heads[0][0].expire[16:32] = [ref.NEVER] * 16
    heads[1][1].expire = [ref.NEVER] * 100
    _attend(kvp, cache, heads, q, now, workspace=ws)
    kvp.kvp_decode_attn_block8(dev_bf16(q), cache, now, workspace=ws)      # no status word: nothing to record into
    cache.count.fill_(10**9)                                              # clamped to the table, whose tail is -1
    kvp.kvp_decode_attn_block8(dev_bf16(q), cache, now, workspace=ws, status=st)
    torch.cuda.synchronize()


def test_attention_past_32_bit_offsets(kvp):
    """Pools of more than 2^32 bytes, the pages in use at their end."""
    cap, d = 2_200_000, 128                            # 4.5 GB each
    small, heads, now = _build(kvp, 1, 161, 1, 300, 2, d, reserve=4)
    big = _alloc(kvp, 1, 2, d, cap, small.max_pages, 1)
    n = small.n_pages_cap
    for a, b in ((big.kq_pool, small.kq_pool), (big.vq_pool, small.vq_pool), (big.scale_pool, small.scale_pool),
                 (big.expire_pool, small.expire_pool)):
        a[cap - n:] = b
    on = small.page_table >= 0
    big.page_table.copy_(torch.where(on, small.page_table + (cap - n), -1))
    big.count.copy_(small.count)
    big.remap.copy_(small.remap)
    _attend(kvp, big, heads, _bits(162, (1, 6, d)), now)
    k, v = kvp.kvp_read_block8(big, 0, 60)
    k2, v2 = kvp.kvp_read_block8(small, 0, 60)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    st, flag = status_word(), torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    for i in range(3):                                 # larger and larger: the page's rows are rounded anew
        x = dev_bf16(_bits(163, (1, 2, d))) * 4.0**i
        for c in (big, small):
            kvp.kvp_append_block8(c, x, x, now + 1 + i, mode=1, flag_step=flag, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for a, b in ((big.kq_pool, small.kq_pool), (big.vq_pool, small.vq_pool), (big.scale_pool, small.scale_pool),
                 (big.expire_pool, small.expire_pool)):
        assert torch.equal(a[cap - n:], b)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_over_two_caches_merges(kvp, fmt):
    """A sequence kept in two caches: both parts' rows and log-sum-exps, merged, are the whole's."""
    B, T, H, G, d = 2, 260, 2, 4, 128
    a, ha, now = _build(kvp, fmt, 171, B, T, H, d)
    b, hb, _ = _build(kvp, fmt, 173, B, T, H, d)
    b.count[1, 1] = 0                                  # one part without rows
    hb[1][1] = ref.Head(d, fmt)
    q = _bits(174, (B, H * G, d))
    parts = [_attend(kvp, c, hs, q, now) for c, hs in ((a, ha), (b, hb))]
    out, lse = kvp.kvp_attn_merge(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    torch.cuda.synchronize()
    for i in range(B):
        for h in range(H):
            sl = slice(h * G, (h + 1) * G)
            x, y = (hs[i][h].attend(ref.widen(q)[i, sl], now, 1 / math.sqrt(d)) for hs in (ha, hb))
            top = np.maximum(x[1], y[1])
            wx, wy = np.exp(x[1] - top), np.exp(y[1] - top)
            want = (wx[:, None] * x[0] + wy[:, None] * y[0]) / (wx + wy)[:, None]
            size = tuple((wx[:, None] * s + wy[:, None] * t) / (wx + wy)[:, None] for s, t in zip(x[2], y[2]))
            tol, _ = ref.attention_bounds(d, 2 * T, size, np.maximum(x[3], y[3]))
            assert (np.abs(out[i, sl].double().cpu().numpy() - want) <= 2 * tol).all()


# ---------------------------------------------------------------------------- together, streams, graphs

def test_two_streams_with_their_own_workspaces(kvp):
    """Calls in flight at once on two streams, each with its own cache and allocating its own workspace."""
    made = [_build(kvp, f, 181 + f, 4, 900, 8, 128) for f in FMTS]
    q = [_bits(183 + f, (4, 32, 128)) for f in FMTS]
    streams = [torch.cuda.Stream() for _ in FMTS]
    qd = [dev_bf16(x) for x in q]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            lse = torch.empty(4, 32, device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            outs[i].append((kvp.kvp_decode_attn_block8(qd[i], made[i][0], made[i][2], lse=lse, stream=s), lse))
    torch.cuda.synchronize()
    for i in range(2):
        _compare(*outs[i][0], made[i][1], ref.widen(q[i]), made[i][2], 1 / math.sqrt(128), 4)
        for o, l in outs[i][1:]:
            assert torch.equal(o, outs[i][0][0]) and torch.equal(l, outs[i][0][1])


def test_calls_on_a_raw_stream(kvp):
    """A stream given as its handle: outputs and workspaces that the binding makes belong to it."""
    cache, heads, now = _build(kvp, 0, 187, 2, 400, 4, 64)
    q = _bits(188, (2, 8, 64))
    qd = dev_bf16(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [kvp.kvp_decode_attn_block8(qd, cache, now, stream=s.cuda_stream) for _ in range(10)]
    k, v = kvp.kvp_read_block8(cache, 0, 30, stream=s.cuda_stream)
    r, _ = kvp.kvp_qk_norm_rope(qd, None, None, None, stream=s.cuda_stream)
    torch.cuda.synchronize()
    lse = torch.empty(2, 8, device="cuda")
    _compare(kvp.kvp_decode_attn_block8(qd, cache, now, lse=lse), lse, heads, ref.widen(q), now, 1 / 8, 2)
    want = kvp.kvp_decode_attn_block8(qd, cache, now)
    assert all(torch.equal(o, want) for o in outs) and torch.equal(r, qd)
    assert torch.equal(k, kvp.kvp_read_block8(cache, 0, 30)[0])


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_steps_in_one_graph(kvp, fmt):
    """Norm and rotation, append and attention of a decode step captured once and replayed for 20 positions, compared
    with the restatement at each; then the whole cache read back."""
    B, H, G, d, T, steps = 2, 2, 4, 128, 27, 20
    cache, heads, now = _build(kvp, fmt, 191, B, T, H, d, reserve=steps)
    inv_freq = 10000.0 ** (-np.arange(0, d, 2) / d)
    turns = kvp.kvp_rope_turns(inv_freq)
    qw, kw = (1 + 0.1 * syn.normal_f32(192 + i, 341, (d,)) for i in range(2))
    qkv = torch.zeros(B, H * (G + 2), d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.empty(B, H * G, d, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(B, H, d, dtype=torch.bfloat16, device="cuda")
    score, tau = torch.zeros(B, H, device="cuda"), torch.zeros(B, H, device="cuda")
    out, lse = torch.empty(B, H * G, d, device="cuda"), torch.empty(B, H * G, device="cuda")
    ws = torch.zeros(kvp.kvp_decode_attn_block8_workspace_bytes(B, H * G, H, d), dtype=torch.uint8, device="cuda")
    st = status_word()
    qwd, kwd = dev_f32(qw), dev_f32(kw)

    def step():
        kvp.kvp_qk_norm_rope(qkv[:, :H * G], qkv[:, H * G:H * (G + 1)], pos, turns, q_weight=qwd, k_weight=kwd, eps=1e-5,
                             q_out=q, k_out=k)
        kvp.kvp_append_block8_devpos(cache, k, qkv[:, H * (G + 1):], pos[:1], mode=0, score=score, tau=tau, window=6,
                                     status=st)
        kvp.kvp_decode_attn_block8_devpos(q, cache, pos[:1], out=out, lse=lse, workspace=ws, status=st)

    saved = [t.clone() for t in (cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool, cache.remap,
                                 cache.count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, old in zip((cache.kq_pool, cache.vq_pool, cache.scale_pool, cache.expire_pool, cache.remap, cache.count),
                      saved):
        t.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        x = _bits(200 + i, (B, H * (G + 2), d), 1)
        sc = syn.normal_f32(i, 342, (B, H))
        qkv.copy_(dev_bf16(x))
        score.copy_(dev_f32(sc))
        pos.fill_(now + 1 + i)
        graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        p = [now + 1 + i] * B
        xf = ref.widen(x)
        for got, rows, w in ((q, xf[:, :H * G], qw), (k, xf[:, H * G:H * (G + 1)], kw)):
            want = ref.rotate(rows, np.asarray(w, np.float64), 1e-5, p, inv_freq, False)
            # half a bf16 step, and the fp32 norm, angle and rotation: 2^-15 of the pair's size
            pair = np.abs(want) + np.abs(np.roll(want, d // 2, -1))
            assert (np.abs(got.double().cpu().numpy() - want) <= 2.0**-8 * np.abs(want) + 2.0**-15 * pair).all()
        kk, vv = ref.widen(host_bits(k)), xf[:, H * (G + 1):]     # the keys as rounded: what the cache was given
        for b in range(B):
            for h in range(H):
                heads[b][h].append(kk[b, h], vv[b, h], ref.expire_of(0, now + 1 + i, 6, 0, sc[b, h], 0.0), now + 1 + i)
        _compare(out, lse, heads, ref.widen(host_bits(q)), now + 1 + i, 1 / math.sqrt(d), G)
    _check_cache(cache, heads, fmt)
    rows, _ = kvp.kvp_read_block8(cache, 0, T + steps)
    torch.cuda.synchronize()
    for b in range(B):
        for h in range(H):
            np.testing.assert_array_equal(rows[b, :heads[b][h].count, h].double().cpu().numpy(), heads[b][h].values(0))


def test_binding_refusals(kvp):
    cache = _alloc(kvp, 2, 2, 64, 4, 2, 0)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    st = status_word()
    with pytest.raises(TypeError):
        kvp.kvp_decode_attn_block8(x.float(), cache, 0)
    with pytest.raises(ValueError):
        kvp.kvp_decode_attn_block8(x[:1], cache, 0)
    with pytest.raises(ValueError):
        kvp.kvp_decode_attn_block8(x, cache, 0, lse=torch.zeros(2, 3, device="cuda"))
    with pytest.raises(ValueError):
        kvp.kvp_decode_attn_block8(x, cache, 0, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kvp.kvp_append_block8(cache, x, x[:, :1], 0, mode=1, flag_step=None, status=st)
    with pytest.raises(ValueError):
        kvp.kvp_append_block8(cache, x.cpu(), x, 0, mode=1, flag_step=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
                              status=st)
    with pytest.raises(kvp.KvpError):
        kvp.kvp_append_block8(cache, x, x, 0, mode=1, flag_step=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
                              status=None)
    with pytest.raises(ValueError):
        kvp.kvp_read_block8(cache, 0, 4, k_out=x.view(1, 2, 2, 64))
    with pytest.raises(ValueError):
        kvp.kvp_compact_block8(x.view(1, 2, 2, 64), x.view(1, 2, 2, 64), 0, 0, cache, mode=1,
                               flag_step=torch.zeros(4, dtype=torch.int32, device="cuda"), status=st)
    with pytest.raises(Exception):
        cache.fmt = 1                                    # a handle's buffers and format stay
    bad = {f.name: getattr(cache, f.name) for f in dataclasses.fields(cache)}
    bad["scale_pool"] = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        kvp.Block8PagedKV(**bad)
