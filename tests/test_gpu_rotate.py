"""kvp_qk_norm_rope on the GPU against the float64 restatement."""
import math

import numpy as np
import pytest
import torch

import block8_ref as ref
import kvp_synth as syn
from helpers import dev_bf16, dev_f32, dev_i32

pytestmark = pytest.mark.gpu


def _freqs(rot, base=10000.0):
    return base ** (-np.arange(0, rot, 2) / rot) if rot else np.zeros(0)


def _check(got, x, w, eps, pos, freqs, interleaved):
    """Half a bf16 step of the value (2^-8), and what fp32 may lose before that rounding, relative to the size of the
    rotated pair: the sum of 128 squares (at most 2^-17 after the root), its root, products and rotation (a few 2^-24
    each) and the angle (2^-32 turns, and 2^-25 of half a turn in its conversion: under 2^-22)."""
    want = ref.rotate(x, w, eps, pos, freqs, interleaved)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w if w is not None else x
    half = len(freqs)
    pair = np.abs(y).copy()
    if half:
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        pair[..., a] = pair[..., b] = np.hypot(y[..., a], y[..., b])
    got = got.double().cpu().numpy()
    off = np.abs(got - want)
    tol = 2.0**-8 * np.abs(want) + 2.0**-16 * pair + 2.0**-134       # and half of bf16's smallest step
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,rot_share,norm", [
    (1, 1, 1, 1.0, True), (1, 32, 8, 1.0, True), (16, 32, 8, 1.0, False), (3, 5, 7, 0.5, True), (7, 0, 3, 0.25, True),
    (7, 9, 0, 0.5, False), (130, 6, 2, 1.0, True), (5000, 3, 1, 1.0, True), (33, 4, 4, 0.0, True), (2, 64, 64, 0.75, False), (9001, 3, 2, 0.5, True),
    (20011, 1, 1, 1.0, False), (4099, 0, 9, 0.25, True)])
def test_rotation(kvp, d, interleaved, n, hq, hk, rot_share, norm):
    rot = int(d * rot_share) // 16 * 16
    freqs = _freqs(rot)
    turns = kvp.kvp_rope_turns(freqs) if rot else None
    pos = (np.abs(syn.normal_f32(1, 351, (n,))) * 50000).astype(np.int32)
    x = syn.normal_bf16(2, 352, (n, hq + 2 * hk + 1, d), std=3.0)
    w = [1 + 0.3 * syn.normal_f32(3 + i, 353, (d,)) if norm else None for i in range(2)]
    dev = dev_bf16(x)
    q, k = (dev[:, :hq] if hq else None), (dev[:, hq:hq + hk] if hk else None)     # views: other rows lie between
    qo, ko = kvp.kvp_qk_norm_rope(q, k, dev_i32(pos) if rot else None, turns,
                                  q_weight=None if w[0] is None or not hq else dev_f32(w[0]),
                                  k_weight=None if w[1] is None or not hk else dev_f32(w[1]), eps=1e-5,
                                  interleaved=interleaved)
    torch.cuda.synchronize()
    xf = ref.widen(x)
    for got, rows, weight in ((qo, xf[:, :hq], w[0]), (ko, xf[:, hq:hq + hk], w[1])):
        if rows.shape[1] == 0:
            assert got is None
            continue
        _check(got, rows, None if weight is None else weight.astype(np.float64), 1e-5, pos, freqs, interleaved)
    # in place, and into every second row of a wider buffer: the same bits, the rows between as they were
    if hq and hk:
        wide = torch.full((n, 2 * (hq + hk), d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
        q2, k2 = wide[:, 0:2 * hq:2, :d], wide[:, 2 * hq::2, :d]
        kvp.kvp_qk_norm_rope(q, k, dev_i32(pos) if rot else None, turns, q_weight=None if w[0] is None else dev_f32(w[0]),
                             k_weight=None if w[1] is None else dev_f32(w[1]), eps=1e-5, interleaved=interleaved,
                             q_out=q2, k_out=k2)
        rest = dev[:, hq + hk:].clone()
        kvp.kvp_qk_norm_rope(q, k, dev_i32(pos) if rot else None, turns, q_weight=None if w[0] is None else dev_f32(w[0]),
                             k_weight=None if w[1] is None else dev_f32(w[1]), eps=1e-5, interleaved=interleaved,
                             q_out=q, k_out=k)
        torch.cuda.synchronize()
        assert torch.equal(q2, qo) and torch.equal(k2, ko) and torch.equal(q, qo) and torch.equal(k, ko)
        assert (wide[:, 1::2] == 3).all() and (wide[..., d:] == 3).all() and torch.equal(dev[:, hq + hk:], rest)


def test_far_and_negative_positions(kvp):
    """Angles keep their digits at every int32 position: compared with exact multiples of a turn fraction."""
    d, rot = 64, 64
    freqs = _freqs(rot, 500000.0)
    freqs[1] = 2 * math.pi / 3                            # a third of a turn, a multiple of which is exact to check
    turns = kvp.kvp_rope_turns(freqs)
    fixed = [int(t) % 2**64 for t in turns.cpu().tolist()]
    pos = np.array([0, 1, -1, 2**20 + 1, 2**30, 2**31 - 1, -2**31, 12345677], np.int32)
    x = syn.normal_bf16(5, 361, (len(pos), 2, d))
    got, _ = kvp.kvp_qk_norm_rope(dev_bf16(x), None, dev_i32(pos), turns)
    torch.cuda.synchronize()
    # the table's own fractions, in whole numbers: what the call promises for these `turns`
    ang = np.array([[2 * math.pi * ((int(p) * f) % 2**64) / 2**64 for f in fixed] for p in pos])
    y = ref.widen(x)
    a, b = y[..., :32], y[..., 32:]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    want = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.hypot(a, b)
    tol = 2.0**-8 * np.abs(want) + 2.0**-16 * np.concatenate([size, size], -1)
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    # and the table's fraction of the third: 2^31 - 1 turns of it are off by 2^31 2^-53 at most
    assert abs((fixed[1] * (2**31 - 1)) % 2**64 / 2**64 - ((2**31 - 1) % 3) / 3) < 2.0**-21


def test_zero_tokens_and_refusals(kvp):
    turns = kvp.kvp_rope_turns(_freqs(64))
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, none = kvp.kvp_qk_norm_rope(q, None, pos, turns)
    assert out.shape == q.shape and none is None
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        kvp.kvp_qk_norm_rope(x, None, pos, turns)                       # positions of other tokens
    with pytest.raises(ValueError):
        kvp.kvp_qk_norm_rope(x, x[:2], torch.zeros(3, dtype=torch.int32, device="cuda"), turns)
    with pytest.raises(ValueError):
        kvp.kvp_qk_norm_rope(x, None, None, turns)
    with pytest.raises(TypeError):
        kvp.kvp_qk_norm_rope(x.half(), None, torch.zeros(3, dtype=torch.int32, device="cuda"), turns)
    with pytest.raises(ValueError):
        kvp.kvp_qk_norm_rope(x, None, None, None, q_weight=torch.ones(32, device="cuda"))
    with pytest.raises(kvp.KvpError):
        kvp.kvp_qk_norm_rope(x, None, torch.zeros(3, dtype=torch.int32, device="cuda"),
                             kvp.kvp_rope_turns(_freqs(128)))             # longer than the head
    with pytest.raises(kvp.KvpError):
        kvp.kvp_qk_norm_rope(x, None, None, None, q_out=torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
                             .expand(3, 4, 64))                           # tokens that share their rows


def test_special_rows(kvp):
    """Zero rows stay zero with a norm; infinities and NaNs stay in their rows; values past rot_dim are not touched by
    the rotation's arithmetic."""
    d = 128
    x = syn.normal_bf16(6, 371, (4, 3, d))
    x[1, 1] = 0
    x[2, 0, 100] = 0x7F80
    x[3, 2, 5] = 0x7FC0
    turns = kvp.kvp_rope_turns(_freqs(64))
    pos = torch.arange(4, dtype=torch.int32, device="cuda") * 1000
    got, _ = kvp.kvp_qk_norm_rope(dev_bf16(x), None, pos, turns, q_weight=torch.ones(d, device="cuda"))
    plain, _ = kvp.kvp_qk_norm_rope(dev_bf16(x), None, pos, turns)
    torch.cuda.synchronize()
    assert not got[1, 1].any()
    bad = ~torch.isfinite(got).all(-1)
    assert bad.nonzero().tolist() == [[2, 0], [3, 2]]
    assert torch.isposinf(plain[2, 0, 100]) and torch.isfinite(plain[2, 0, :100]).all()
    assert torch.equal(plain[..., 64:].view(torch.int16), dev_bf16(x)[..., 64:].view(torch.int16))
