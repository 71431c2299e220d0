"""The precision of the attention over the 8-bit cache on ordinary inputs, for every width, format and number of queries
a kv head that has a kernel of its own (the bound and what it tells apart: test_block8_precision.py)."""
import math

import numpy as np
import pytest
import torch

import block8_ref as ref
from helpers import dev_bf16, dev_i32, status_word
from test_block8_precision import CASES, REL, inputs, relative

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,d,G,T", CASES)
def test_attention_is_as_precise_as_promised(kvp, fmt, d, G, T):
    q, k, v, flag = inputs(fmt, d, G, T)
    heads = ref.compact(fmt, 1, ref.widen(k), ref.widen(v), T - 1, 0, 0, flag=flag)
    width = (T + 15) // 16
    cache = kvp.Block8PagedKV.allocate(1, 2, d, 2 * width, width, fmt=fmt)
    st = status_word()
    kvp.kvp_compact_block8(dev_bf16(k), dev_bf16(v), T - 1, 0, cache, mode=1, flag_step=dev_i32(flag), window=0, status=st)
    lse = torch.empty(1, 2 * G, device="cuda")
    for limit in (0, 1, 3):
        out = kvp.kvp_decode_attn_block8(dev_bf16(q), cache, T, lse=lse, grid_limit=limit, status=st)
        torch.cuda.synchronize()
        assert st.item() == 0
        got, got_lse = out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
        for h in range(2):
            sl = slice(h * G, (h + 1) * G)
            want, want_lse, *_ = heads[0][h].attend(ref.widen(q)[0, sl], T, 1 / math.sqrt(d))
            assert relative(got[sl], want) < REL, (limit, h, relative(got[sl], want))
            assert relative(got_lse[sl], want_lse) < REL
            assert np.isfinite(got_lse[sl]).all()
