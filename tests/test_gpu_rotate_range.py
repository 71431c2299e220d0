"""kvp_qk_norm_rope at the ends of its range: rows of every size that the norm takes, and positions far out against
exact angles."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block8_ref as ref
import kvp_synth as syn
from helpers import dev_bf16, dev_f32, dev_i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [9, 9001])              # heads side by side in a warp, tokens side by side
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
def test_norm_over_its_range(kvp, d, interleaved, n, eps):
    """Rows over the whole range that the norm takes: values up to 2^60, a mean square plus eps of 2^-100 or more."""
    H, rot = 3, d // 2
    freqs = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    power = np.array([0, 59, 58, 40, 7, -7, -20, -40, -48] + ([-49, -62, -64, -75, -100, -120, -123] if eps >= 2.0**-100 else []))
    x = np.clip(syn.normal_f32(601, 1, (n, H, d)).astype(np.float64), -3.5, 3.5) / 2     # below 2 in magnitude
    x = x * np.ldexp(1.0, power[(np.arange(n)[:, None] + 5 * np.arange(H)) % len(power)])[..., None]
    xb = syn.f32_to_bf16_bits(x.astype(np.float32))
    w = 1 + 0.3 * syn.normal_f32(602, 1, (d,))
    pos = (np.arange(n) * 7 % 1000).astype(np.int32)
    got, _ = kvp.kvp_qk_norm_rope(dev_bf16(xb), None, dev_i32(pos), kvp.kvp_rope_turns(freqs), q_weight=dev_f32(w), eps=eps,
                                  interleaved=interleaved)
    torch.cuda.synchronize()
    xf = ref.widen(xb)
    eps32 = float(np.float32(eps))                     # the call takes eps as fp32
    want = ref.rotate(xf, w.astype(np.float64), eps32, pos, freqs, interleaved)
    y = xf / np.sqrt((xf * xf).mean(-1, keepdims=True) + eps32) * w
    pair = np.abs(y)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    pair[..., a] = pair[..., b] = np.hypot(y[..., a], y[..., b])
    off = np.abs(got.double().cpu().numpy() - want)
    # half a bf16 step, fp32's own rounding of the norm, the angle and the rotation, half of bf16's smallest step
    bad = ~(off <= 2.0**-8 * np.abs(want) + 2.0**-16 * pair + 2.0**-134)
    assert not bad.any(), np.unique(np.argwhere(bad)[:, 0] % len(power))


def test_far_positions_against_exact_angles(kvp):
    """The rotation of (1, 0) at far positions: cos and sin of pos * inv_freq, whose whole turns are taken off in
    rational arithmetic (pi to 45 digits)."""
    d = 64
    freqs = np.concatenate([10000.0 ** (-np.arange(0, 32, 2) / 32), 500000.0 ** (-np.arange(0, 32, 2) / 32)])
    freqs[[3, 20, 31]] = [6.25, -3.0, 1e-9]
    pos = np.array([0, 1, -1, 2**30 + 7, 2**31 - 1, -2**31, 1999999999, -123456789], np.int32)
    two_pi = 2 * Fraction(3141592653589793238462643383279502884197169399, 10**45)
    ang = np.array([[float(Fraction(float(f)) * int(p) / two_pi % 1) for f in freqs] for p in pos]) * 2 * math.pi
    x = np.zeros((len(pos), 1, d), np.float32)
    x[..., :32] = 256.0
    got, _ = kvp.kvp_qk_norm_rope(dev_bf16(syn.f32_to_bf16_bits(x)), None, dev_i32(pos), kvp.kvp_rope_turns(freqs))
    torch.cuda.synchronize()
    want = 256 * np.concatenate([np.cos(ang), np.sin(ang)], -1)
    assert (np.abs(got[:, 0].double().cpu().numpy() - want) <= 2.0**-8 * np.abs(want) + 256 * 2.0**-22).all()
