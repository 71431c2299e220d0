"""The 8-bit cache's attention at the ends of the number range."""
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
