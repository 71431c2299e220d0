"""CPU checks of refusals by the calls over packed prompts and by the decode attention that adds its weights (nothing here
reaches a GPU: an argument that is not refused ends in KVP_ERR_CUDA)."""
import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._builder().build()
    import kv_cache_pruning_gb300 as k
    return k


# ---------------------------------------------------------------------------- tables that are not 4-byte aligned

@pytest.mark.parametrize("devpos", [False, True])
@pytest.mark.parametrize("which", ["table", "remap", "count"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_decode_sums_refuse_unaligned_tables(L, devpos, which, off):
    p = dict(table=16, remap=16, count=16)
    p[which] += off
    fn = L.library().kvp_decode_attn_acc_devpos if devpos else L.library().kvp_decode_attn_acc
    assert fn(2, 8, 2, 64, 16, 16, 16, 16, 4, p["table"], 3, p["remap"], p["count"], 16 if devpos else 5, 0.0, 16, None, 16,
              200, 100, 100, 0, 16, 1 << 40, None, None) == L.KVP_ERR_ALIGN


@pytest.mark.parametrize("which", ["table", "count", "table_q", "count_q"])
def test_decode_attention_refuses_unaligned_tables(L, which):
    p = dict(table=16, count=16, table_q=16, count_q=16)
    p[which] += 2
    lib = L.library()
    if not which.endswith("_q"):
        head, tail = (2, 8, 2, 64, 16, 16, 16, 16, 4, p["table"], 3, p["count"]), (0, 16, 1 << 40, None, None)
        assert lib.kvp_decode_attn(*head, 5, 0.0, 16, *tail) == L.KVP_ERR_ALIGN
        assert lib.kvp_decode_attn_lse(*head, 5, 0.0, 16, 16, *tail) == L.KVP_ERR_ALIGN
        assert lib.kvp_decode_attn_devpos(*head, 16, 0.0, 16, *tail) == L.KVP_ERR_ALIGN
    assert lib.kvp_decode_attn_two_tier(2, 8, 2, 64, 16, 16, 16, 16, 4, p["table"], 3, p["count"], 16, 16, 16, 4,
                                        p["table_q"], 3, p["count_q"], 5, 0.0, 16, 0, 16, 1 << 40, None,
                                        None) == L.KVP_ERR_ALIGN


# ---------------------------------------------------------------------------- more sequences than the kernels' counters take

@pytest.mark.parametrize("n_seqs", [2**31 - 2**16 + 1, 2**31 - 32, 2**31 - 1])
def test_prompt_calls_refuse_counts_that_pass_32_bits(L, n_seqs):
    lib = L.library()
    assert lib.kvp_prompt_attn(n_seqs, 10, 4, 2, 128, 16, 512, 128, 16, 256, 128, 16, 256, 128, 16, None, 0.0, 16, 512, 128,
                               None, None, None) == L.KVP_ERR_UNSUPPORTED
    assert lib.kvp_prompt_weights(n_seqs, 10, 4, 2, 64, 16, 256, 64, 16, 128, 64, 16, None, 16, 0.0, 0, 16, -1, 2, 1, 0,
                                  None, None) == L.KVP_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------- a scale whose product with log2 e is no number

@pytest.mark.parametrize("scale, name", [(1.1 * 2.0 ** 127, "UNSUPPORTED"), (3.4e38, "UNSUPPORTED"), (2.0 ** 127, "CUDA")])
def test_prompt_calls_refuse_scales_that_overflow(L, scale, name):
    import torch
    if name == "CUDA" and torch.cuda.is_available():
        pytest.skip("reaches the device")
    lib = L.library()
    assert lib.kvp_prompt_attn(2, 10, 4, 2, 128, 16, 512, 128, 16, 256, 128, 16, 256, 128, 16, None, scale, 16, 512, 128,
                               None, None, None) == getattr(L, "KVP_ERR_" + name)
    assert lib.kvp_prompt_weights(2, 10, 4, 2, 64, 16, 256, 64, 16, 128, 64, 16, None, 16, scale, 0, 16, -1, 2, 1, 0,
                                  None, None) == getattr(L, "KVP_ERR_" + name)
