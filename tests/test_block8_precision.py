"""What the attention over the 8-bit cache promises of its precision on ordinary inputs, and, on the CPU, that the bound
tells a kernel that keeps it from one that does not: weights of one fp16 number instead of a pair."""
import math

import numpy as np
import pytest

import block8_ref as ref
import kvp_synth as syn

# The relative 2-norm that an output block [G, d] of one (b, h) may be off by, for queries, keys and values that are unit
# normals. The error of an output is sum p_i eps_i (v_i - out), about as large beside sum p_i v_i as the relative error
# eps_i of a weight, root mean square. That is, in 2^x with x of 1.44 rms: 8 products' sums of a few, each half of 2^-23
# of it (1.7e-7 times ln 2); the factor (5e-8); the distance to the reference, up to 12, rounded to 2^-20 (2.8e-7 times
# ln 2); 2^x (1e-7); the fp16 pair (7e-8); and for the accumulator's 25 additions 2e-7. Together 4e-7; five times that is
# never passed by a sum of so many terms. One fp16 number instead of the pair: half of 2^-11, uniform, 2e-4.
REL = 2e-6

CASES = [(fmt, d, G, T) for fmt in (ref.E4M3, ref.INT8) for d in (64, 128) for G in (1, 4, 5, 8) for T in (61, 400)]


def inputs(fmt, d, G, T):
    """bf16 bits of q [1, 2 G, d], k and v [1, T, 2, d], and the flags [1, 2, T]: 30 % of the tokens gone at T."""
    q, k, v = (syn.normal_bf16(801 + i, 1, s) for i, s in enumerate([(1, 2 * G, d), (1, T, 2, d), (1, T, 2, d)]))
    flag = np.where(syn.uniform(804, 1, 2 * T).reshape(1, 2, T) < 0.3, 0, -1).astype(np.int32)
    return q, k, v, flag


def relative(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("fmt,d,G,T", CASES)
def test_the_bound_tells_one_fp16_weight_from_a_pair(fmt, d, G, T):
    q, k, v, flag = inputs(fmt, d, G, T)
    heads = ref.compact(fmt, 1, ref.widen(k), ref.widen(v), T - 1, 0, 0, flag=flag)
    for h in range(2):
        qh = ref.widen(q)[0, h * G:(h + 1) * G]
        want, *_ = heads[0][h].attend(qh, T, 1 / math.sqrt(d))
        x = qh @ heads[0][h].values(0).T / math.sqrt(d) * math.log2(math.e)
        w = np.exp2(x - x.max(1, keepdims=True) + 12)
        one = w.astype(np.float16).astype(float)
        pair = one + (w - one).astype(np.float16).astype(float)
        v_h, l = heads[0][h].values(1), w.sum(1, keepdims=True)
        assert relative(pair @ v_h / l, want) < REL / 10
        assert relative(one @ v_h / l, want) > 10 * REL
