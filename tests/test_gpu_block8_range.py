"""The 8-bit cache's attention at the ends of the number range: logits of millions, values near bf16's largest and
smallest numbers."""
import math

import numpy as np
import pytest
import torch

import block8_ref as ref
import kvp_synth as syn
from helpers import dev_bf16, status_word

pytestmark = pytest.mark.gpu
FMTS = [ref.E4M3, ref.INT8]


def _written(kvp, fmt, kb, vb):
    """A cache of every row of kb, vb [B, T, H, d] (bf16 bits), and its Head[b][h]."""
    B, T, H, d = kb.shape
    width = (T + 15) // 16
    cache = kvp.Block8PagedKV.allocate(B, H, d, B * H * width, width, fmt=fmt)
    st = status_word()
    kvp.kvp_compact_block8(dev_bf16(kb), dev_bf16(vb), T - 1, 0, cache, mode=1,
                           flag_step=torch.full((B, H, T), -1, dtype=torch.int32, device="cuda"), status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    return cache, ref.compact(fmt, 1, ref.widen(kb), ref.widen(vb), T - 1, 128, 0, flag=np.full((B, H, T), -1))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [4, 7])
def test_equal_logits_of_any_size(kvp, fmt, d, G):
    """Keys that are all alike: every logit of a query is the same number, however large, so its output is the mean of
    the values, and its log-sum-exp that logit + ln T."""
    T, H = 55, 2
    k = np.zeros((1, T, H, d), np.float32)
    k[..., 0] = 1.0
    kb, vb = syn.f32_to_bf16_bits(k), syn.f32_to_bf16_bits(syn.normal_f32(501, 1, (1, T, H, d)))
    cache, heads = _written(kvp, fmt, kb, vb)
    lse = torch.empty(1, H * G, device="cuda")
    for e in range(10, 34):
        q = np.zeros((1, H * G, d), np.float32)
        # mantissas that bf16 holds and whose products with log2(e) round to even and to odd last places
        q[0, :, 0] = [math.ldexp(1 + (5 * j + e) % 32 / 32, e) * (-1 if j % 3 == 2 else 1) for j in range(H * G)]
        for limit in (0, 1, 3):
            out = kvp.kvp_decode_attn_block8(dev_bf16(syn.f32_to_bf16_bits(q)), cache, T - 1, scale=1.0, lse=lse,
                                             grid_limit=limit)
            torch.cuda.synchronize()
            got, got_lse = out.double().cpu().numpy()[0], lse.double().cpu().numpy()[0]
            for h in range(H):
                v = heads[0][h].values(1)
                for j in range(h * G, (h + 1) * G):
                    # equal weights: only the sums and the division round (4 pages, the merges, 1 / l: 16 steps)
                    assert (np.abs(got[j] - v.mean(0)) <= 16 * 2.0**-23 * np.abs(v).mean(0)).all(), (e, j)
                    want = float(q[0, j, 0]) + math.log(T)
                    assert abs(got_lse[j] - want) <= abs(want) * 2.0**-21 + 2.0**-20, (e, j)


@pytest.mark.parametrize("fmt", FMTS)
def test_logits_that_tell_one_token_apart(kvp, fmt):
    """Logits of millions that differ: the largest's value is the output, whatever page and warp it is in."""
    T, d, G = 300, 64, 8
    rng = np.random.default_rng(7)
    for e in (20, 23, 24, 25, 26, 27, 30):
        k = np.zeros((1, T, 1, d), np.float32)
        k[0, :, 0, 0] = 1.0 + rng.integers(0, 4, T) / 8          # exact in both formats: ties are exact, too
        kb, vb = syn.f32_to_bf16_bits(k), syn.f32_to_bf16_bits(syn.normal_f32(503, e, (1, T, 1, d)))
        cache, heads = _written(kvp, fmt, kb, vb)
        q = np.zeros((1, G, d), np.float32)
        q[0, :, 0] = [math.ldexp(1 + j / 8, e) * (-1 if j % 2 else 1) for j in range(G)]
        for limit in (0, 1, 2):
            out = kvp.kvp_decode_attn_block8(dev_bf16(syn.f32_to_bf16_bits(q)), cache, T - 1, scale=1.0, grid_limit=limit)
            torch.cuda.synchronize()
            key, v = heads[0][0].values(0)[:, 0], heads[0][0].values(1)
            for j in range(G):
                top = key == (key.max() if q[0, j, 0] > 0 else key.min())
                # the others are 2^(e - 3) log2(e) or more below: weight 0. Equal weights, as above, and a page's add
                off = np.abs(out[0, j].double().cpu().numpy() - v[top].mean(0))
                assert (off <= (16 + T / 16) * 2.0**-23 * np.abs(v[top]).mean(0)).all(), (e, j)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 5])
def test_values_near_the_largest_numbers(kvp, fmt, d, G):
    """Values up to bf16's largest number: their weighted mean is finite, so the output is. Slots enough for partial
    results of several warps and CTAs, one page of one sign and of the largest magnitude among smaller ones."""
    B, T, H = 1, 150, 2
    v = syn.normal_f32(511, 1, (B, T, H, d)).astype(np.float64) * 2.0**100
    v[0, 32:48] = np.sign(v[0, 32:48]) * 2.0**116
    v[0, 64:80] = np.abs(v[0, 64:80]) * 2.0**24                  # up to about 2^126, all positive
    v[0, 70] = 2.0**127
    kb, vb = syn.f32_to_bf16_bits(syn.normal_f32(512, 1, (B, T, H, d))), syn.f32_to_bf16_bits(v.astype(np.float32))
    cache, heads = _written(kvp, fmt, kb, vb)
    assert max(heads[0][0].scales[1]) >= 2.0**118
    q = syn.normal_bf16(513, 1, (B, H * G, d))
    for limit in (0, 1, 3):
        out = kvp.kvp_decode_attn_block8(dev_bf16(q), cache, T - 1, grid_limit=limit)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        for h in range(H):
            sl = slice(h * G, (h + 1) * G)
            want, _, size_abs, size = heads[0][h].attend(ref.widen(q)[0, sl], T - 1, 1 / math.sqrt(d))
            tol, _ = ref.attention_bounds(d, T, size_abs, size)
            assert np.isfinite(got[0, sl]).all() and (np.abs(got[0, sl] - want) <= tol).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [3, 8])
def test_values_near_the_smallest_numbers(kvp, fmt, G):
    """Pages whose scale is the smallest, 2^-126, beside one another: nothing of their values is lost but fp32's own
    subnormal steps."""
    T, d = 150, 64
    kb = syn.f32_to_bf16_bits(syn.normal_f32(521, 1, (1, T, 1, d)))
    vb = syn.f32_to_bf16_bits((syn.normal_f32(522, 1, (1, T, 1, d)).astype(np.float64) * 2.0**-121).astype(np.float32))
    cache, heads = _written(kvp, fmt, kb, vb)
    assert max(heads[0][0].scales[1]) <= 2.0**-124
    q = syn.normal_bf16(523, 1, (1, G, d))
    for limit in (0, 2):
        out = kvp.kvp_decode_attn_block8(dev_bf16(q), cache, T - 1, grid_limit=limit)
        torch.cuda.synchronize()
        want, _, size_abs, size = heads[0][0].attend(ref.widen(q)[0], T - 1, 1 / 8)
        tol, _ = ref.attention_bounds(d, T, size_abs, size)
        # the bounds without their allowance for this range, 1e-37; instead half of fp32's smallest step (2^-150) at each
        # of a sum's T / 16 + 40 additions, 2^11 of the output's units in one of the sum's (weights are 2^12 and more,
        # values enter scaled down by 2^23 at most), and one at the end
        tol = tol - 1e-37 + (T / 16 + 40) * 2.0**-139 + 2.0**-149
        assert (np.abs(out.double().cpu().numpy()[0] - want) <= tol).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_the_largest_numbers_read_back(kvp, fmt):
    """Codes whose value is 2^128 read as infinity, those below as themselves."""
    d = 64
    rows = [0x7F77, 0x7F7D, 0x7F7F, 0xFF7F]       # 2^128 (1 - 9 / 256), (1 - 3 / 256), (1 - 1 / 256), and its negative
    kb = np.zeros((1, len(rows), 1, d), np.uint16)
    kb[0, :, 0, 3] = rows
    cache, heads = _written(kvp, fmt, kb, kb)
    k, v = kvp.kvp_read_block8(cache, 0, len(rows))
    torch.cuda.synchronize()
    want = heads[0][0].values(0)
    top = want.max()
    assert top == 2.0**128 and (np.abs(want[:, 3]) == top).tolist() == [False, fmt == ref.E4M3, True, True]
    want = np.where(np.abs(want) == top, np.copysign(np.inf, want), want)
    for got in (k, v):
        np.testing.assert_array_equal(got[0, :, 0].double().cpu().numpy(), want)
