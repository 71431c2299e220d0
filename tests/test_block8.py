"""CPU checks of the block-scaled 8-bit cache and of kvp_qk_norm_rope: what their entry points refuse on the host (no
call here reaches a GPU), the table of rotation angles, and the float64 restatement that the GPU tests compare with."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block8_ref as ref


@pytest.fixture(scope="module")
def k():
    import __graft_entry__
    __graft_entry__._builder().build()
    import kv_cache_pruning_gb300
    return kv_cache_pruning_gb300


# ---------------------------------------------------------------------------- refusals

def test_compact_refusals(k):
    L = k.library()
    ws = L.kvp_compact_block8_workspace_bytes(2, 3, 16, 4)

    def call(fmt=0, mode=0, b=2, h=3, hd=128, n_pos=16, kp=16, st=8, scores=16, tau=16, flag=None, window=128, delay=0,
             reserve=0, kq=16, sc=16, ep=16, cap=4, width=1, wsp=16, wsb=ws, status=16):
        return L.kvp_compact_block8(fmt, mode, b, h, hd, n_pos, kp, 16, 0, st, 0, scores, tau, flag, window, delay, 15,
                                    reserve, kq, 16, sc, ep, cap, 16, width, 16, 16, wsp, wsb, status, None)

    assert call(fmt=2) == k.KVP_ERR_INVALID
    assert call(mode=2) == k.KVP_ERR_INVALID
    assert call(flag=16) == k.KVP_ERR_INVALID                        # KVzap with flags too
    assert call(tau=None) == k.KVP_ERR_INVALID
    assert call(mode=1, flag=16) == k.KVP_ERR_INVALID                # DMS with scores too
    assert call(mode=1, scores=None, tau=None) == k.KVP_ERR_INVALID  # DMS without flags
    assert call(b=0) == k.KVP_ERR_INVALID
    assert call(n_pos=-1) == k.KVP_ERR_INVALID
    assert call(window=-1) == k.KVP_ERR_INVALID
    assert call(delay=-1) == k.KVP_ERR_INVALID
    assert call(reserve=-1) == k.KVP_ERR_INVALID
    assert call(status=None) == k.KVP_ERR_INVALID
    assert call(kp=None) == k.KVP_ERR_INVALID
    assert call(kq=None) == k.KVP_ERR_INVALID
    assert call(sc=None) == k.KVP_ERR_INVALID
    assert call(ep=None) == k.KVP_ERR_INVALID
    assert call(st=-8) == k.KVP_ERR_INVALID
    assert call(n_pos=2**31 - 200, window=128, delay=100) == k.KVP_ERR_INVALID   # expire would overflow
    assert call(hd=96) == k.KVP_ERR_UNSUPPORTED
    assert call(b=70000, h=1) == k.KVP_ERR_UNSUPPORTED
    assert call(width=2**27) == k.KVP_ERR_UNSUPPORTED
    assert call(reserve=2**31 - 20) == k.KVP_ERR_UNSUPPORTED
    assert call(b=1, h=1, n_pos=65535 * 512 + 1, wsb=1 << 40) == k.KVP_ERR_UNSUPPORTED
    assert call(b=65535, h=1, reserve=2**20, wsb=1 << 40) == k.KVP_ERR_UNSUPPORTED    # page ids past 2^31
    assert call(kp=8) == k.KVP_ERR_ALIGN
    assert call(kq=8) == k.KVP_ERR_ALIGN
    assert call(st=4) == k.KVP_ERR_ALIGN
    assert call(wsp=24, wsb=1 << 20) == k.KVP_ERR_ALIGN
    assert call(wsb=ws - 1) == k.KVP_ERR_WORKSPACE
    assert call(wsp=None) == k.KVP_ERR_WORKSPACE
    assert L.kvp_compact_block8_workspace_bytes(0, 3, 16, 4) == 0
    # the other compactions' words, 16-byte rounded, the page count, 8 bytes a page, a bit for each of a segment's 128 positions
    assert ws == (L.kvp_compact_workspace_bytes(2, 3, 16) + 15) // 16 * 16 + 16 + 4 * 8 + 2 * 3 * 16


def test_append_refusals(k):
    L = k.library()

    def call(fmt=0, mode=0, hd=128, pos=5, kn=16, st=0, score=16, tau=16, flag=None, window=128, sc=16, remap=16,
             status=16):
        return L.kvp_append_block8(fmt, mode, 1, 1, hd, pos, kn, 16, st, 0, 0, 0, score, tau, flag, window, 0, 16, 16,
                                   sc, 16, 1, 16, 1, remap, 16, status, None)

    assert call(fmt=-1) == k.KVP_ERR_INVALID
    assert call(mode=3) == k.KVP_ERR_INVALID
    assert call(flag=16) == k.KVP_ERR_INVALID
    assert call(mode=1, flag=16) == k.KVP_ERR_INVALID
    assert call(mode=1, score=None, tau=None) == k.KVP_ERR_INVALID
    assert call(pos=-1) == k.KVP_ERR_INVALID
    assert call(pos=2**31 - 100) == k.KVP_ERR_INVALID
    assert call(window=-2) == k.KVP_ERR_INVALID
    assert call(kn=None) == k.KVP_ERR_INVALID
    assert call(remap=None) == k.KVP_ERR_INVALID
    assert call(sc=None) == k.KVP_ERR_INVALID
    assert call(status=None) == k.KVP_ERR_INVALID
    assert call(st=-8) == k.KVP_ERR_INVALID
    assert call(hd=32) == k.KVP_ERR_UNSUPPORTED
    assert call(kn=8) == k.KVP_ERR_ALIGN
    assert call(st=12) == k.KVP_ERR_ALIGN
    assert call(sc=8) == k.KVP_ERR_ALIGN

    def devpos(p):
        return L.kvp_append_block8_devpos(0, 0, 1, 1, 128, p, 16, 16, 0, 0, 0, 0, 16, 16, None, 128, 0, 16, 16, 16, 16,
                                          1, 16, 1, 16, 16, 16, None)

    assert devpos(None) == k.KVP_ERR_INVALID
    assert devpos(18) == k.KVP_ERR_ALIGN


def test_read_refusals(k):
    L = k.library()

    def call(fmt=0, b=2, h=2, hd=64, first=0, n=4, ko=16, sb=1024, st=128, sh=64, status=16):
        return L.kvp_read_block8(fmt, b, h, hd, 16, 16, 16, 1, 16, 1, 16, first, n, ko, 16, sb, st, sh, status, None)

    assert call(fmt=7) == k.KVP_ERR_INVALID
    assert call(first=-1) == k.KVP_ERR_INVALID
    assert call(n=-1) == k.KVP_ERR_INVALID
    assert call(ko=None) == k.KVP_ERR_INVALID
    assert call(status=None) == k.KVP_ERR_INVALID
    assert call(sb=0) == k.KVP_ERR_INVALID      # rows written twice
    assert call(st=56) == k.KVP_ERR_INVALID
    assert call(sh=0) == k.KVP_ERR_INVALID
    assert call(hd=256) == k.KVP_ERR_UNSUPPORTED
    assert call(first=2**31 - 20, n=4) == k.KVP_ERR_UNSUPPORTED
    assert call(ko=8) == k.KVP_ERR_ALIGN
    assert call(st=132) == k.KVP_ERR_ALIGN
    # b 2, n 4, h 2 rows of 64: a slot's heads reach into the next slot, a sequence's slots into the next sequence
    assert call(st=64) == k.KVP_ERR_INVALID
    assert call(sb=448) == k.KVP_ERR_INVALID
    assert call(sh=1 << 62) == k.KVP_ERR_INVALID
    assert call(n=0, ko=None) == k.KVP_OK       # nothing to do: nothing is launched


def test_attention_refusals_and_workspace(k):
    L = k.library()
    ws = L.kvp_decode_attn_block8_workspace_bytes(2, 21, 3, 64)
    # counters of the most (b, h) there can be, two partial results for each of 512 CTAs
    assert ws == 4096 * 4 + 2 * 512 * 7 * 66 * 4
    for bad in ((0, 8, 8, 64), (1, 9, 2, 64), (1, 18, 2, 64), (1, 8, 8, 96), (4097, 1, 1, 64)):
        assert L.kvp_decode_attn_block8_workspace_bytes(*bad) == 0

    def call(fmt=0, b=2, hq=21, h=3, d=64, q=16, out=16, lse=None, width=4, now=0, scale=0.0, limit=0, wsp=16, wsb=ws,
             sc=16, ep=16):
        return L.kvp_decode_attn_block8(fmt, b, hq, h, d, q, 16, 16, sc, ep, 1, 16, width, 16, now, scale, out, lse,
                                        limit, wsp, wsb, None, None)

    assert call(fmt=3) == k.KVP_ERR_INVALID
    assert call(b=0) == k.KVP_ERR_INVALID
    assert call(limit=-1) == k.KVP_ERR_INVALID
    for s in (-1.0, float("nan"), float("inf")):
        assert call(scale=s) == k.KVP_ERR_INVALID
    assert call(q=None) == k.KVP_ERR_INVALID
    assert call(sc=None) == k.KVP_ERR_INVALID
    assert call(ep=None) == k.KVP_ERR_INVALID
    assert call(hq=20) == k.KVP_ERR_UNSUPPORTED
    assert call(hq=27) == k.KVP_ERR_UNSUPPORTED      # 9 query heads per kv head
    assert call(d=96) == k.KVP_ERR_UNSUPPORTED
    assert call(b=2000) == k.KVP_ERR_UNSUPPORTED     # 6000 (b, h)
    assert call(width=2**27) == k.KVP_ERR_UNSUPPORTED
    assert call(q=8) == k.KVP_ERR_ALIGN
    assert call(out=24) == k.KVP_ERR_ALIGN
    assert call(lse=18) == k.KVP_ERR_ALIGN
    assert call(wsp=24, wsb=ws + 64) == k.KVP_ERR_ALIGN
    assert call(wsb=ws - 1) == k.KVP_ERR_WORKSPACE
    assert call(wsp=None) == k.KVP_ERR_WORKSPACE
    assert L.kvp_decode_attn_block8_devpos(0, 2, 21, 3, 64, 16, 16, 16, 16, 16, 1, 16, 4, 16, None, 0.0, 16, None, 0,
                                           16, ws, None, None) == k.KVP_ERR_INVALID


def test_rotation_refusals(k):
    L = k.library()

    def call(n=4, hq=2, hk=1, d=128, rot=128, q=16, qst=256, qsh=128, pos=16, turns=16, wq=None, eps=1e-6, qo=4096,
             qot=256, qoh=128):
        return L.kvp_qk_norm_rope(n, hq, hk, d, rot, 0, q, qst, qsh, 16, 128, 0, pos, turns, wq, None, eps, qo, qot, qoh,
                                  8192, 128, 0, None)

    assert call(n=-1) == k.KVP_ERR_INVALID
    assert call(hq=-1) == k.KVP_ERR_INVALID
    assert call(hq=0, hk=0) == k.KVP_ERR_INVALID
    assert call(rot=-16) == k.KVP_ERR_INVALID
    assert call(rot=144) == k.KVP_ERR_INVALID
    for e in (-1e-6, float("nan"), float("inf")):
        assert call(eps=e) == k.KVP_ERR_INVALID
    assert call(q=None) == k.KVP_ERR_INVALID
    assert call(pos=None) == k.KVP_ERR_INVALID
    assert call(turns=None) == k.KVP_ERR_INVALID
    assert call(qst=-8) == k.KVP_ERR_INVALID
    assert call(qot=120) == k.KVP_ERR_INVALID        # rows written twice
    assert call(qoh=0) == k.KVP_ERR_INVALID
    assert call(qot=128) == k.KVP_ERR_INVALID        # a token's second head is the next token's first
    assert call(qot=128, qoh=384) == k.KVP_ERR_INVALID
    assert call(qo=16, qot=512) == k.KVP_ERR_INVALID  # in place with other strides
    assert call(d=96) == k.KVP_ERR_UNSUPPORTED
    assert call(rot=24) == k.KVP_ERR_UNSUPPORTED
    assert call(hq=100000) == k.KVP_ERR_UNSUPPORTED
    assert call(q=24) == k.KVP_ERR_ALIGN
    assert call(wq=20) == k.KVP_ERR_ALIGN
    assert call(turns=20) == k.KVP_ERR_ALIGN
    assert call(pos=18) == k.KVP_ERR_ALIGN
    assert call(qst=260) == k.KVP_ERR_ALIGN
    assert call(n=0, q=None) == k.KVP_OK


def test_binding_refuses_what_is_not_on_a_gpu(k):
    cpu = torch.zeros(2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        k.Block8PagedKV(cpu, cpu, torch.zeros(2, 2), torch.zeros(2, 16, dtype=torch.int32),
                        torch.zeros(1, 1, 2, dtype=torch.int32), torch.zeros(1, 1, 32, dtype=torch.int32),
                        torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        k.Block8PagedKV.allocate(1, 1, 64, 2, 2, fmt=5, device="cpu")
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        k.kvp_qk_norm_rope(x, None, None, None)
    with pytest.raises(ValueError):
        k.kvp_qk_norm_rope(None, None, None, None)


# ---------------------------------------------------------------------------- the table of angles

def test_turns_table(k):
    """Each entry is inv_freq / (2 pi) in units of 2^-64 turns: within float64's rounding of that quotient (2^-52 of
    it), whole turns dropped."""
    freqs = [1.0, 0.5, 1e-4, 500000.0 ** (-63 / 64), 0.0, 7.25, -0.3, 2 * math.pi, -1e-30]
    got = k.kvp_rope_turns(freqs, device="cpu").numpy().view(np.uint64)
    two_pi = Fraction(math.pi) * 2 + Fraction(2449293598294707, 10**31)     # pi to 31 digits: float64 pi + 1.2246e-16
    for f, g in zip(freqs, got):
        want = Fraction(f) / two_pi
        off = (Fraction(int(g), 2**64) - want) % 1
        off = min(off, 1 - off)
        assert off <= abs(want) * Fraction(1, 2**51) + Fraction(1, 2**60), (f, float(off))
    with pytest.raises(k.KvpError):
        k.kvp_rope_turns([float("nan")], device="cpu")
    assert k.kvp_rope_turns([], device="cpu").numel() == 0


# ---------------------------------------------------------------------------- the restatement itself

def test_reference_e4m3_matches_the_format():
    """Against torch's E4M3 type: decoding every byte, and rounding a sweep of values with ties."""
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.nan_to_num(ref.TABLE[ref.E4M3], nan=-1), np.nan_to_num(want, nan=-1))
    x = np.concatenate([np.linspace(-448, 448, 20011), np.ldexp(np.linspace(-1, 1, 4001), -6), np.ldexp(1.0, -np.arange(14))])
    x = x.astype(np.float32)
    got = ref.encode(x, 1.0, ref.E4M3)
    np.testing.assert_array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    x = np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.0, -127.0, 0.0], np.float32)     # int8 ties to even
    np.testing.assert_array_equal(ref.encode(x, 1.0, ref.INT8).view(np.int8), [0, 2, 2, 0, -2, 126, 127, -127, 0])


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.INT8])
def test_reference_scales(fmt):
    """A scale is the smallest power of two that reaches: half of it does not."""
    rng = np.random.default_rng(5)
    for x in [rng.normal(size=40) * 10.0**e for e in range(-30, 31, 5)] + [np.array([ref.LARGEST[fmt]]), np.array([1.0])]:
        s = ref.scale_of(x, fmt)
        a = np.abs(x).max()
        assert math.frexp(s)[0] == 0.5
        assert ref.LARGEST[fmt] * s >= a > ref.LARGEST[fmt] * s / 2
    assert ref.scale_of([0.0, -0.0], fmt) == 0
    assert ref.scale_of([math.inf, math.nan, 3.0], fmt) == ref.scale_of([3.0], fmt)
    assert ref.scale_of([2.0**-133], fmt) == 2.0**-126


def test_reference_growth_error_is_bounded():
    """However often a page's scale grows, an int8 value stays within one step of the last scale, and an E4M3 value
    within half a step of its own rounding plus half a subnormal step of the last scale."""
    rng = np.random.default_rng(7)
    x = rng.normal(size=(16, 64)) * np.ldexp(1.0, np.arange(16))[:, None]
    for fmt in (ref.INT8, ref.E4M3):
        head = ref.Head(64, fmt)
        for r in range(16):
            head.append(x[r], x[r], ref.NEVER, r)
        s = head.scales[0][0]
        off = np.abs(head.values(0) - x)
        if fmt == ref.INT8:
            assert (off <= s).all()
        else:
            assert (off <= np.abs(x) * 2.0**-4 + s * 2.0**-9).all()
