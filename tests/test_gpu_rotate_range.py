"""kvp_qk_norm_rope at the ends of its range: positions far out against exact angles."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block8_ref as ref
import kvp_synth as syn
from helpers import dev_bf16, dev_f32, dev_i32

pytestmark = pytest.mark.gpu


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
