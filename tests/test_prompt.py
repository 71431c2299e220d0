"""CPU checks of the prompt attention, accumulating decode attention and eviction calls: refusals on the host (nothing
here reaches a GPU), workspace sizes, and the restatement that the GPU tests compare with."""
import math

import pytest
import torch

import prompt_ref as ref


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__._builder().build()
    import kv_cache_pruning_gb300 as k
    return k


def prompt(L, n_seqs=2, n=10, hq=4, h=2, d=128, q=16, qt=512, qh=128, k=16, kt=256, kh=128, v=16, vt=256, vh=128,
           start=16, length=None, scale=0.0, out=16, ot=512, oh=128, lse=None):
    return L.library().kvp_prompt_attn(n_seqs, n, hq, h, d, q, qt, qh, k, kt, kh, v, vt, vh, start, length, scale, out, ot,
                                       oh, lse, None, None)


@pytest.mark.parametrize("args, name", [
    (dict(n_seqs=-1), "INVALID"), (dict(n=-1), "INVALID"), (dict(hq=0), "INVALID"), (dict(h=0), "INVALID"),
    (dict(hq=5), "INVALID"), (dict(d=96), "UNSUPPORTED"), (dict(hq=65536, h=65536), "UNSUPPORTED"),
    (dict(n=2**31), "UNSUPPORTED"), (dict(n=2**31 - 1), "UNSUPPORTED"), (dict(q=None), "INVALID"),
    (dict(k=None), "INVALID"), (dict(v=None), "INVALID"), (dict(out=None), "INVALID"), (dict(start=None), "INVALID"), (dict(scale=-1.0), "INVALID"),
    (dict(scale=math.inf), "INVALID"), (dict(scale=math.nan), "INVALID"), (dict(q=8), "ALIGN"), (dict(k=24), "ALIGN"),
    (dict(v=2), "ALIGN"), (dict(out=8), "ALIGN"), (dict(qt=516), "ALIGN"), (dict(kh=4), "ALIGN"), (dict(oh=12), "ALIGN"),
    (dict(vt=0), "INVALID"), (dict(kh=0), "INVALID"), (dict(qh=-128), "INVALID"), (dict(kt=2**39), "UNSUPPORTED"),
    (dict(ot=504), "INVALID"), (dict(oh=64), "INVALID"), (dict(ot=0), "INVALID"), (dict(start=18), "ALIGN"),
    (dict(length=2), "ALIGN"), (dict(lse=2), "ALIGN")])
def test_prompt_attn_refuses(L, args, name):
    assert prompt(L, **args) == getattr(L, "KVP_ERR_" + name)


def test_nothing_to_do(L):
    assert prompt(L, n_seqs=0, start=None) == L.KVP_OK
    assert prompt(L, n=0, q=None, k=None, v=None, out=None, start=None) == L.KVP_OK


def prompt_weights(L, n_seqs=2, n=10, hq=4, h=2, d=64, q=16, qt=256, qh=64, k=16, kt=128, kh=64, start=16, length=None,
                   lse=16, scale=0.0, last=0, acc=16, a_s=20, at=1, ah=10, acc_len=10):
    return L.library().kvp_prompt_weights(n_seqs, n, hq, h, d, q, qt, qh, k, kt, kh, start, length, lse, scale, last, acc,
                                          a_s, at, ah, acc_len, None, None)


@pytest.mark.parametrize("args, name", [
    (dict(n_seqs=-1), "INVALID"), (dict(hq=3), "INVALID"), (dict(d=32), "UNSUPPORTED"), (dict(q=None), "INVALID"),
    (dict(k=None), "INVALID"), (dict(lse=None), "INVALID"), (dict(acc=None), "INVALID"), (dict(last=-1), "INVALID"),
    (dict(scale=-0.5), "INVALID"), (dict(a_s=-2), "INVALID"), (dict(at=-1), "INVALID"), (dict(acc_len=-1), "INVALID"),
    (dict(at=0), "INVALID"), (dict(ah=9), "INVALID"), (dict(a_s=10), "INVALID"), (dict(acc=2), "ALIGN"),
    (dict(lse=6), "ALIGN"), (dict(kt=100), "ALIGN"), (dict(qt=0), "INVALID"), (dict(a_s=-1, at=1, ah=1), "INVALID")])
def test_prompt_weights_refuses(L, args, name):
    assert prompt_weights(L, **args) == getattr(L, "KVP_ERR_" + name)


def decode(L, fn="kvp_decode_attn_acc", B=2, hq=8, h=2, d=64, q=16, cap=4, mp=3, remap=16, now=5, scale=0.0, out=16,
           acc=16, ab=200, ah=100, al=100, ws=16, wsb=None):
    if wsb is None:
        wsb = 1 << 40
    return getattr(L.library(), fn)(B, hq, h, d, q, 16, 16, 16, cap, 16, mp, remap, 16, now, scale, out, None, acc, ab, ah,
                                    al, 0, ws, wsb, None, None)


@pytest.mark.parametrize("args, name", [
    (dict(B=0), "INVALID"), (dict(hq=7), "INVALID"), (dict(hq=6), "UNSUPPORTED"), (dict(d=96), "UNSUPPORTED"),
    (dict(q=None), "INVALID"), (dict(remap=None), "INVALID"), (dict(acc=None), "INVALID"), (dict(acc=2), "ALIGN"),
    (dict(al=-1), "INVALID"), (dict(ab=-1), "INVALID"), (dict(ah=99), "INVALID"), (dict(ab=199), "INVALID"),
    (dict(ws=None), "WORKSPACE"), (dict(wsb=100), "WORKSPACE"), (dict(ws=8), "ALIGN"), (dict(q=8), "ALIGN"),
    (dict(cap=2**27), "UNSUPPORTED"), (dict(mp=2**27 - 1), "UNSUPPORTED"), (dict(B=4097, h=1, hq=1), "UNSUPPORTED"),
    (dict(scale=math.nan), "INVALID")])
def test_decode_attn_acc_refuses(L, args, name):
    assert decode(L, **args) == getattr(L, "KVP_ERR_" + name)


def test_devpos_forms_need_a_position(L):
    assert decode(L, "kvp_decode_attn_acc_devpos", now=None) == L.KVP_ERR_INVALID
    assert decode(L, "kvp_decode_attn_acc_devpos", now=6) == L.KVP_ERR_ALIGN
    lib = L.library()
    assert lib.kvp_evict_paged_devpos(1, 1, 16, 0, 0, 4, 16, 1, 16, 1, 16, 16, 1, 1, None, None, None,
                                      None) == L.KVP_ERR_INVALID


def test_acc_workspace(L):
    f = L.kvp_decode_attn_acc_workspace_bytes
    base = L.kvp_decode_attn_workspace_bytes(2, 8, 2, 64)
    # the attention's own, (m, l) of each row, the logits of each query head and slot
    assert f(2, 8, 2, 64, 3) == base + 2 * 8 * 8 + 2 * 8 * 3 * 16 * 4
    assert f(2, 8, 2, 64, 0) == base + 2 * 8 * 8
    assert f(0, 8, 2, 64, 3) == 0 and f(2, 7, 2, 64, 3) == 0 and f(2, 8, 2, 64, -1) == 0


def evict(L, B=2, h=2, n=10, acc=16, sb=20, st=1, sh=10, budget=3, recent=2, now=9, expire=16, count=16):
    return L.library().kvp_evict(B, h, n, acc, sb, st, sh, budget, recent, now, expire, count, None)


@pytest.mark.parametrize("args, name", [
    (dict(B=0), "INVALID"), (dict(h=0), "INVALID"), (dict(n=-1), "INVALID"), (dict(acc=None), "INVALID"),
    (dict(expire=None), "INVALID"), (dict(budget=-1), "INVALID"), (dict(recent=-1), "INVALID"), (dict(now=-1), "INVALID"),
    (dict(now=2**31 - 1), "INVALID"), (dict(sb=-1), "INVALID"), (dict(acc=2), "ALIGN"), (dict(count=18), "ALIGN"),
    (dict(B=2**13, h=2**12), "UNSUPPORTED"), (dict(n=2**31 - 1), "UNSUPPORTED")])
def test_evict_refuses(L, args, name):
    assert evict(L, **args) == getattr(L, "KVP_ERR_" + name)


def evict_paged(L, B=2, h=2, acc=16, sb=20, sh=10, al=10, expire=16, cap=4, table=16, mp=2, remap=16, count=16, budget=3,
                recent=2, now=9, kept=16):
    return L.library().kvp_evict_paged(B, h, acc, sb, sh, al, expire, cap, table, mp, remap, count, budget, recent, now,
                                       kept, None, None)


@pytest.mark.parametrize("args, name", [
    (dict(B=0), "INVALID"), (dict(acc=None), "INVALID"), (dict(al=-1), "INVALID"), (dict(expire=None), "INVALID"),
    (dict(cap=-1), "INVALID"), (dict(table=None), "INVALID"), (dict(mp=-1), "INVALID"), (dict(remap=None), "INVALID"),
    (dict(count=None), "INVALID"), (dict(budget=-1), "INVALID"), (dict(recent=-1), "INVALID"), (dict(now=-1), "INVALID"),
    (dict(now=2**31 - 1), "INVALID"), (dict(sh=-1), "INVALID"), (dict(expire=18), "ALIGN"), (dict(kept=2), "ALIGN"),
    (dict(mp=2**27), "UNSUPPORTED"), (dict(B=2**13, h=2**12), "UNSUPPORTED")])
def test_evict_paged_refuses(L, args, name):
    assert evict_paged(L, **args) == getattr(L, "KVP_ERR_" + name)


def test_binding_refuses_cpu_tensors(L):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    start = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.kvp_prompt_attn(q, q, q, start)
    with pytest.raises(ValueError, match="CUDA"):
        L.kvp_prompt_weights(q, q, start, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        L.kvp_evict(torch.zeros(1, 1, 4), 3, budget=2)


# ---------------------------------------------------------------------------- the restatement itself

def test_reference_attention_is_torch_s():
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(13, x, 64, generator=gen).bfloat16() for x in (6, 2, 2))
    out, lse, _, _ = ref.attention(q, k, v, ref.sequences([0, 5, 5, 13], None, 13))
    for a, b in ((0, 5), (5, 13)):
        want = torch.nn.functional.scaled_dot_product_attention(
            q[a:b].double().transpose(0, 1), k[a:b].double().transpose(0, 1).repeat_interleave(3, 0),
            v[a:b].double().transpose(0, 1).repeat_interleave(3, 0), is_causal=True)
        assert torch.allclose(out[a:b], want.transpose(0, 1), atol=1e-12)
    acc, _ = ref.weights(q, k, lse, ref.sequences([0, 5, 5, 13], None, 13))
    assert abs(float(acc[:5].sum()) - 5 * 6) < 1e-10 and abs(float(acc[5:].sum()) - 8 * 6) < 1e-10   # a query pays 1 in all
    first = torch.softmax((q[5:6].double() * k[5:6].double().repeat_interleave(3, 1)).sum(-1), 0)
    assert first.numel() == 6 and float(acc[12].sum()) <= 6


def test_reference_eviction_by_hand():
    acc = torch.tensor([[[5.0, 1.0, 5.0, math.nan, -math.inf, 5.0, 0.0, -0.0, 9.0, 9.0]]])
    expire, count = ref.evict_dense(acc, 9, 5, 2)            # positions 8 and 9 are recent, three more stay: 0, 2, 5
    assert (expire[0, 0] == NEVER).nonzero()[:, 0].tolist() == [0, 2, 5, 8, 9] and int(count) == 5
    expire, count = ref.evict_dense(acc, 9, 7, 2)            # ... then 1 and the first of the two zeros
    assert (expire[0, 0] == NEVER).nonzero()[:, 0].tolist() == [0, 1, 2, 5, 6, 8, 9]
    assert int(ref.evict_dense(acc, 9, 9, 2)[1]) == 9        # all but NaN
    assert ref.evict_dense(acc, 9, 9, 2)[0][0, 0, 3] == 9
    assert int(ref.evict_dense(acc, 9, 0, 3)[1]) == 3 and int(ref.evict_dense(acc, 9, 0, 0)[1]) == 0


NEVER = ref.NEVER
