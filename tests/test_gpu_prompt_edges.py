"""Calls over packed prompts at the edges of what they allow, against the restatement in 64 bits (tests/prompt_ref.py)."""
import math

import pytest
import torch

import prompt_ref as ref
from test_gpu_prompt import cache_of, i32, normal, qkv, status

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- sequences that share rows

def disjoint(start, seq_len, n_tok):
    """(first row, length) of every sequence that counts; None: its numbers break the rules, or its rows start before the end
    of an earlier sequence's whose numbers do not."""
    out, reach = [], 0
    for s in ref.sequences(start, seq_len, n_tok):
        if s is not None and s[1] > 0:
            a, n = s
            s = s if a >= reach else None
            reach = max(reach, a + n)
        out.append(s)
    return out


def stepping(seed, n_seqs, n_tok):
    """Starts that mostly ascend, some steps down: sequences that break the rules, and later ones that begin in the rows of
    earlier ones, of the same 32 and of others."""
    gen = torch.Generator().manual_seed(seed)
    start, top = [0], 0
    for i in range(n_seqs):
        if torch.rand((), generator=gen) < 0.08:
            start.append(max(0, start[-1] - int(torch.randint(1, 200, (), generator=gen))))
        elif torch.rand((), generator=gen) < 0.03:
            start.append(n_tok + 7)
            top = start[-2]
        else:
            at = top if start[-1] > n_tok else start[-1]
            start.append(min(n_tok, at + int(torch.randint(0, 90, (), generator=gen))))
    return start


SHARED = [([0, 50, 40, 100], None), ([0, 50, 40, 100], [30, 0, 60]), ([0, 50, 40, 100], [45, 0, 60]),
          ([40, 100, 0, 60, 90], None), ([0, 100, 20, 50, 30, 100], None), ([0, 90, 89, 89, 100], None),
          ([0, 10, 0, 10, 0, 10], None)]


@pytest.mark.parametrize("h, g, d", [(1, 2, 128), (2, 1, 64), (2, 4, 128), (4, 3, 64), (4, 5, 128), (8, 8, 64)])
@pytest.mark.parametrize("case", range(len(SHARED) + 4))
def test_no_row_is_written_twice(kvp, h, g, d, case):
    if case < len(SHARED):
        (start, seq_len), n = SHARED[case], 100
    else:
        n_seqs, n = ((20, 900), (31, 1500), (90, 3000), (400, 9000))[case - len(SHARED)]
        start, seq_len = stepping(40 + case, n_seqs, n), None
        if case % 2:
            seq_len = [max(0, b - a) * 3 // 4 for a, b in zip(start, start[1:])]
    seqs = disjoint(start, seq_len, n)
    assert any(s is None for s in seqs)
    q, k, v = qkv(case, n, h * g, h, d)
    out, lse = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((h * g, n), -7.0, device="cuda")
    st, lens = status(), None if seq_len is None else i32(seq_len)
    kvp.kvp_prompt_attn(q, k, v, i32(start), seq_len=lens, out=out, lse=lse, status=st)
    assert int(st) == kvp.KVP_ERR_BOUNDS
    mine = torch.zeros(n, dtype=torch.bool, device="cuda")
    for s in seqs:
        if s is not None:
            assert not bool(mine[s[0]:s[0] + s[1]].any())
            mine[s[0]:s[0] + s[1]] = True
    want, want_lse, tol, lse_tol = ref.attention(q, k, v, seqs)
    ref.within(out[mine], want[mine], tol[mine], "out")
    ref.within(lse[:, mine], want_lse[:, mine], lse_tol[:, mine], "lse")
    assert bool((out[~mine] == 3.0).all()) and bool((lse[:, ~mine] == -7.0).all())
    most = max(1, max(s[1] for s in seqs if s is not None))
    for n_last in (0, 40):
        want, tol = ref.weights(q, k, lse, seqs, n_last=n_last)
        acc, by_seq = torch.full((n, h), -5.0, device="cuda"), torch.full((len(seqs), h, most), -5.0, device="cuda")
        for a in (acc, by_seq):
            st = status()
            kvp.kvp_prompt_weights(q, k, i32(start), lse, seq_len=lens, n_last=n_last, acc=a, status=st)
            assert int(st) == kvp.KVP_ERR_BOUNDS
        ref.within(acc[mine], want[mine], tol[mine], "sums by token")
        assert bool((acc[~mine] == -5.0).all())
        for i, s in enumerate(seqs):
            a, m = s or (0, 0)
            ref.within(by_seq[i, :, :m].T, want[a:a + m], tol[a:a + m], f"sums of sequence {i}")
            assert bool((by_seq[i, :, m:] == -5.0).all())


# ---------------------------------------------------------------------------- decode sums of slots that share a position

@pytest.mark.parametrize("g, d", [(1, 128), (2, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("share", [2, 3, 1000])
def test_decode_sums_of_slots_that_share_a_position(kvp, g, d, share):
    """Neighbouring slots (of one thread's round, of one warp) and slots a thousand apart on one position. A sum of k terms
    that are all positive rounds k times, each by 2^-24 of at most the whole; the restatement's bound has two of them."""
    n, b, h = 2600, 1, 2
    cache = cache_of(kvp, 31 + g, [[n, 1500]], n // 16 + 2, d, h, n + 10)
    slot = torch.arange(cache.remap.shape[-1], device="cuda", dtype=torch.int32)
    cache.remap[0, 0] = slot // share
    cache.remap[0, 1] = slot % (1500 // share + 1)
    q, acc = normal(3, b, h * g, d), torch.rand(b, h, n + 10, device="cuda")
    want, tol = ref.decode(q, cache, n + 9, acc)
    terms = torch.zeros_like(acc).double()
    for j, m in enumerate((n, 1500)):
        terms[0, j].index_add_(0, cache.remap[0, j, :m].long(), torch.ones(m, dtype=torch.float64, device="cuda"))
    st = status()
    out = kvp.kvp_decode_attn_acc(q, cache, n + 9, acc, status=st)
    assert int(st) == 0
    ref.within(out, want[0], tol[0], "out")
    ref.within(acc, want[2], tol[2] + terms * 2.0 ** -24 * want[2], "acc")


# ---------------------------------------------------------------------------- queries that pay nothing, whatever they hold

def padded_queries(q, lse, rows, bad):
    """Queries that a caller leaves out, by a log-sum-exp of -inf, and that hold what padding may."""
    q, lse = q.clone(), lse.clone()
    q[rows] = bad
    lse[:, rows] = -math.inf
    return q, lse


@pytest.mark.parametrize("h, g, d", [(2, 4, 128), (1, 3, 64), (3, 1, 128), (1, 7, 64)])
@pytest.mark.parametrize("n_last", [0, 7, 40, 64, 65, 300])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_queries_that_pay_nothing_may_hold_anything(kvp, h, g, d, n_last, bad):
    lens = [700, 130, 1, 260]
    start = [0, 700, 830, 831, 1091]
    q, k, _ = (x.contiguous() for x in qkv(5, 1091, h * g, h, d))
    seqs = ref.sequences(start, None, 1091)
    lse = ref.attention(q, k, k, seqs)[1].float()
    rows = torch.tensor([3, 127, 128, 300, 301, 302, 690, 699, 828, 829, 900, 1000, 1085], device="cuda")
    rows = torch.cat([rows, torch.arange(384, 512, device="cuda")])            # a whole tile of queries
    q2, lse2 = padded_queries(q, lse, rows, bad)
    # what they pay is 0 by the definition, whatever their logits are: as if they were finite
    want, tol = ref.weights(q, k, lse2, seqs, n_last=n_last)
    st, acc = status(), torch.full((1091, h), -5.0, device="cuda")
    kvp.kvp_prompt_weights(q2, k, i32(start), lse2, n_last=n_last, acc=acc, status=st)
    assert int(st) == 0
    ref.within(acc, want, tol, "sums")
    # one head's query alone, and keys that are no number: those keys' sums are, the others' are not touched
    lse3, q3, k3 = lse.clone(), q.clone(), k.clone()
    lse3[0, 699], q3[699, 0], k3[10, 0] = -math.inf, bad, math.nan
    k3f = k.clone()
    k3f[10, 0] = 0.0
    want, tol = ref.weights(q, k3f, lse3, seqs, n_last=n_last)
    acc = kvp.kvp_prompt_weights(q3, k3, i32(start), lse3, n_last=n_last)
    paid = torch.arange(700, device="cuda") >= (700 - n_last if n_last else 0)
    paid[699] = g > 1                                                          # some head's query still looks at key 10
    assert bool(torch.isnan(acc[10, 0])) == bool(paid[10:].any())
    other = torch.ones_like(acc, dtype=torch.bool)
    other[10, 0] = False
    ref.within(acc[other], want[other], tol[other], "sums beside a key that is no number")


def test_an_infinite_normaliser_is_no_mark(kvp):
    """exp(x - inf) is 0 for a finite logit and no number for a NaN or infinite one: only -inf leaves a query out."""
    q, k, _ = (x.contiguous() for x in qkv(6, 300, 2, 1, 64))
    lse = ref.attention(q, k, k, [(0, 300)])[1].float()
    lse[:, 200] = math.inf
    want, tol = ref.weights(q, k, lse, [(0, 300)])
    ref.within(kvp.kvp_prompt_weights(q, k, i32([0, 300]), lse), want, tol, "sums")
    q[200, 0] = math.nan
    got = kvp.kvp_prompt_weights(q, k, i32([0, 300]), lse)
    assert bool(torch.isnan(got[:201]).all())
    ref.within(got[201:], want[201:], tol[201:], "sums of the keys after it")


# ---------------------------------------------------------------------------- rows without a finite logit

@pytest.mark.parametrize("h, g, d, repeat", [(1, 2, 128, 1), (2, 4, 128, 12), (1, 3, 128, 40), (1, 3, 64, 40), (2, 2, 64, 20)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_without_a_finite_logit_see_no_value(kvp, h, g, d, repeat, bad):
    """Such a row is zero with lse -inf wherever a value that is no number lies: in its own tile of keys or in one before."""
    n = 300
    start = [n * i for i in range(repeat + 1)]
    q, k, v = (x.contiguous() for x in qkv(45, n * repeat, h * g, h, d))
    q.copy_(q.abs())
    at = torch.arange(n * repeat, device="cuda") % n
    k[at < 290, :, 0] = -math.inf                            # rows 0 .. 289 see nothing finite, the last ten see the last keys
    for row, col in ((5, 3), (130, 4), (270, 5), (280, 6), (289, 7)):
        v[at == row, :, col] = bad
    st, lse = status(), torch.empty(h * g, n * repeat, device="cuda")
    out = kvp.kvp_prompt_attn(q, k, v, i32(start), lse=lse, status=st)
    assert int(st) == 0
    assert bool((out[at < 290] == 0).all()) and bool((lse[:, at < 290] == -math.inf).all())
    assert bool(torch.isfinite(lse[:, at >= 290]).all())


# ---------------------------------------------------------------------------- sums beside pages that are not there

@pytest.mark.parametrize("g, d", [(1, 64), (2, 128), (4, 64), (8, 128)])
def test_decode_sums_beside_bad_pages(kvp, g, d):
    """A page whose number is out of range counts as empty: its slots' sums stay, the others' are those of the rest."""
    cache = cache_of(kvp, 5, [[100, 100], [700, 40]], 44, d, 2, 760, expired=0.1)
    cache.page_table[0, 0, 2], cache.page_table[0, 1, 0], cache.page_table[1, 0, 30] = cache.n_pages_cap, -5, 2**31 - 1
    cache.page_table[1, 1, :3] = -1
    q, acc, st = normal(6, 2, 2 * g, d), torch.rand(2, 2, 800, device="cuda"), status()
    before = acc.clone()
    want, tol = ref.decode(q, cache, 759, acc)
    lse = torch.empty(2, 2 * g, device="cuda")
    out = kvp.kvp_decode_attn_acc(q, cache, 759, acc, lse=lse, status=st)
    assert int(st) == kvp.KVP_ERR_BOUNDS
    for got, w, e, name in zip((out, lse, acc), want, tol, ("out", "lse", "acc")):
        ref.within(got, w, e, name)
    assert torch.equal(acc[1, 1], before[1, 1]) and bool((out[1, g:] == 0).all())


# ---------------------------------------------------------------------------- rows that share a warp

@pytest.mark.parametrize("h, g, d, repeat", [(1, 2, 128, 1), (1, 2, 64, 1), (2, 4, 128, 12), (2, 3, 128, 24), (2, 3, 64, 24)])
@pytest.mark.parametrize("what", ["large", "nan", "first"])
def test_what_lies_behind_a_sequence_changes_no_bit(kvp, h, g, d, repeat, what):
    """The rows behind a sequence's last one share its tile. Logits of the last rows rise in their second block of keys by
    2^8 to 2^15 over the first's, where a row may keep its reference or move it; what they do is theirs alone."""
    n, gap = 200, 56
    start = [(n + gap) * i for i in range(repeat + 1)]
    q, k, v = (x.contiguous() for x in qkv(71, start[-1], h * g, h, d))
    at = torch.arange(start[-1], device="cuda") % (n + gap)
    q[..., 0], k[..., 0] = 1.0, 0.0
    k[(at >= 150) & (at < 153), :, 0] = 7.3                  # in base 2: 10.5 over the others, at a scale of 1
    q[..., 1:] *= 0.05
    lens = i32([n] * repeat)
    behind = at >= n
    outs = []
    for fill in (0.0, 1.0):
        for x in (q, k, v):
            x[behind] = 0.0
        if fill and what == "large":
            q[behind], k[behind] = 3.0, 30.0
        if fill and what == "nan":
            q[behind], k[behind], v[behind] = math.nan, math.nan, math.inf
        if fill and what == "first":                         # rows without a finite logit in their first block
            q[behind], k[behind] = -math.inf, 1.0
        lse = torch.zeros(h * g, start[-1], device="cuda")
        out = kvp.kvp_prompt_attn(q, k, v, i32(start), seq_len=lens, scale=1.0, lse=lse)
        outs.append((out[~behind], lse[:, ~behind]))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    for x in (q, k, v):
        x[behind] = 0.0
    want, want_lse, tol, lse_tol = ref.attention(q, k, v, [(a, n) for a in start[:-1]], 1.0)
    ref.within(outs[1][0], want[~behind], tol[~behind], "out")
    ref.within(outs[1][1], want_lse[:, ~behind], lse_tol[:, ~behind], "lse")


# ---------------------------------------------------------------------------- one workspace for calls of several kinds

def test_decode_sums_share_a_workspace_with_other_groups(kvp):
    """Layers of one batch and as many kv heads, whose query heads, widths and lengths differ: what one call leaves behind its
    arrival counters says nothing to the next."""
    b, h, t = 2, 4, 5200
    kinds = [(8, 128, 5000), (1, 128, 5000), (4, 64, 300), (2, 128, 5000), (1, 64, 40), (8, 64, 5000), (2, 64, 5000), (4, 128, 5000)]
    need = max(kvp.kvp_decode_attn_acc_workspace_bytes(b, h * g, h, d, n // 16 + 2) for g, d, n in kinds)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for i, (g, d, n) in enumerate(kinds * 2):
        cache = cache_of(kvp, i, [[n, 17, n // 2, n], [1, n, n, 0]], n // 16 + 2, d, h, t)
        q, acc = normal(i, b, h * g, d), torch.rand(b, h, t, device="cuda")
        want = acc.clone()
        fresh = kvp.kvp_decode_attn_acc(q, cache, t - 1, want)
        st = status()
        out = kvp.kvp_decode_attn_acc(q, cache, t - 1, acc, workspace=ws, status=st)
        assert int(st) == 0 and torch.equal(out, fresh) and torch.equal(acc, want), (g, d, n)
