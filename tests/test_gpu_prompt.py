"""Prompt attention, the weights it pays, decode attention that adds its weights, and eviction to a budget, against their
restatement in 64 bits (tests/prompt_ref.py, which also says how far a result may be off)."""
import math

import pytest
import torch

import prompt_ref as ref

pytestmark = pytest.mark.gpu
NEVER, PAGE = ref.NEVER, 16


def normal(seed, *shape, scale=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


def uniform(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.rand(shape, generator=gen, device="cuda")


def starts(lens, gap=0, first=0):
    s = [first]
    for n in lens:
        s.append(s[-1] + n + gap)
    return s


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def qkv(seed, n, hq, h, d, layout="packed"):
    """q, k, v as views of one projection's output, contiguous, or head by head."""
    if layout == "packed":
        x = normal(seed, n, hq + 2 * h, d)
        return x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
    if layout == "heads":
        return tuple(normal(seed + i, m, n, d).transpose(0, 1) for i, m in enumerate((hq, h, h)))
    return tuple(normal(seed + i, n, m, d) for i, m in enumerate((hq, h, h)))


def run_prompt(kvp, q, k, v, start, seq_len=None, **kw):
    n, hq, _ = q.shape
    st, lse = status(), torch.full((hq, n), -7.0, device="cuda")
    out = kvp.kvp_prompt_attn(q, k, v, i32(start), seq_len=None if seq_len is None else i32(seq_len), lse=lse, status=st, **kw)
    return out, lse, int(st)


def check_prompt(kvp, q, k, v, start, seq_len=None, scale=0.0):
    out0 = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse, st = run_prompt(kvp, q, k, v, start, seq_len, scale=scale, out=out0)
    assert st == 0 and out is out0
    seqs = ref.sequences(start, seq_len, q.shape[0])
    want, want_lse, tol, lse_tol = ref.attention(q, k, v, seqs, scale)
    mine = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for a, n in seqs:
        mine[a:a + n] = True
    assert bool((out[~mine] == 3.0).all()) and bool((lse[:, ~mine] == -7.0).all())   # rows of no sequence: as they were
    ref.within(out[mine], want[mine], tol[mine], "out")
    ref.within(lse[:, mine], want_lse[:, mine], lse_tol[:, mine], "lse")
    return out, lse


SHAPES = [(1, 1, 128), (2, 1, 64), (2, 2, 128), (1, 3, 64), (2, 4, 128), (1, 5, 128), (1, 8, 64), (1, 7, 128), (3, 2, 64)]


@pytest.mark.parametrize("h, g, d", SHAPES)
@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [127, 129], [128, 0, 256], [255, 1, 257, 64], [700]])
def test_prompt_attention(kvp, h, g, d, lens):
    start = starts(lens)
    q, k, v = qkv(len(lens) + h, start[-1], h * g, h, d)
    check_prompt(kvp, q, k, v, start)


@pytest.mark.parametrize("layout", ["packed", "heads", "own"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_layouts_padding_and_gaps(kvp, layout, d):
    lens = [100, 300, 0, 129]
    start = starts(lens, gap=37, first=5)
    q, k, v = qkv(3, start[-1] + 50, 6, 2, d, layout)
    check_prompt(kvp, q, k, v, start, lens)
    check_prompt(kvp, q, k, v, start, [0, 0, 0, 0])
    check_prompt(kvp, q, k, v, start)                        # every row between the starts
    out = torch.empty(6, q.shape[0], d + 8, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., :d]
    got, _, st = run_prompt(kvp, q, k, v, start, lens, out=out)
    same, _, _ = run_prompt(kvp, q, k, v, start, lens)
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(start, lens)]).cuda()
    assert st == 0 and torch.equal(got[rows], same[rows])


@pytest.mark.parametrize("h, g, d, n", [(2, 4, 128, 2300), (1, 3, 64, 4111), (4, 1, 128, 1537), (1, 8, 128, 1024)])
def test_prompt_long(kvp, h, g, d, n):
    q, k, v = qkv(11, n, h * g, h, d)
    check_prompt(kvp, q, k, v, [0, n])


def test_prompt_many_sequences(kvp):
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 40, (700,), generator=gen).tolist()
    lens[300], lens[699] = 900, 333
    start = starts(lens)
    q, k, v = qkv(2, start[-1], 4, 2, 64)
    check_prompt(kvp, q, k, v, start)


@pytest.mark.parametrize("d, g", [(128, 2), (64, 3)])
def test_many_sequences_of_many_lengths(kvp, d, g):
    gen = torch.Generator().manual_seed(6)
    lens = (2.0 ** (11 * torch.rand(150, generator=gen))).int().tolist()     # 1 .. 2047, tiles of up to 16 numbers
    lens[40:75] = [0] * 35                                                   # a whole round of lanes without rows
    start = starts(lens)
    q, k, v = qkv(2, start[-1], 2 * g, 2, d)
    _, lse = check_prompt(kvp, q, k, v, start)
    check_weights(kvp, q, k, start, lse=lse)
    check_weights(kvp, q, k, start, lse=lse, n_last=50, by="sequence")


@pytest.mark.parametrize("scale", [1e-3, 0.5, 3.0])
def test_prompt_scales_and_peaks(kvp, scale):
    q, k, v = qkv(21, 500, 4, 2, 128)
    k = k.clone()
    k[77] += 2 * q[400, :2]
    check_prompt(kvp, q, k, v, [0, 500], scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grow", [2.0 ** 6, 2.0 ** 11, 2.0 ** 20, 2.0 ** 40])
def test_prompt_huge_logits(kvp, d, grow):
    """Logits up to 2^80: the softmax is a choice of the largest, and nothing overflows. Rows and columns are powers of
    two of a small pattern, so that every product and sum is exact and ties are ties on both sides."""
    n = 300
    gen = torch.Generator().manual_seed(int(math.log2(grow)))
    q, k = (torch.randint(-1, 2, (n, 2, d), generator=gen).float().cuda() for _ in range(2))
    q, k = (q * grow).bfloat16(), (k * grow).bfloat16()
    v = normal(9, n, 2, d)
    out, lse, st = run_prompt(kvp, q, k, v, [0, n], scale=1.0)
    want, want_lse, tol, _ = ref.attention(q, k, v, [(0, n)], 1.0)
    assert st == 0
    mean = v.double().abs().amax(0)
    assert bool(((out.double() - want).abs() <= 2.0 ** -6 * mean).all())
    assert bool(((lse.double() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs() + 1e-5).all())


def test_prompt_slowly_rising_logits(kvp):
    """Every key beats all before it by a little or by much: the reference moves at every step."""
    n, d = 900, 128
    for step in (0.02, 0.3, 5.0):
        q = torch.zeros(n, 2, d, device="cuda")
        q[..., 0] = 1.0
        k = torch.zeros(n, 1, d, device="cuda")
        k[:, 0, 0] = torch.arange(n, device="cuda") * step
        check_prompt(kvp, q.bfloat16(), k.bfloat16(), normal(4, n, 1, d), [0, n], scale=1.0)


@pytest.mark.parametrize("d, g", [(64, 1), (128, 2), (128, 3)])
def test_prompt_large_and_small_values(kvp, d, g):
    big = torch.finfo(torch.bfloat16).max
    q, k, _ = qkv(31, 700, g, 1, d)
    v = torch.full((700, 1, d), big, dtype=torch.bfloat16, device="cuda")
    v[::2] = -big
    check_prompt(kvp, q, k, v, [0, 700])
    v[:] = big                                               # a mean of the largest number: it, or infinity by rounding
    out, _, st = run_prompt(kvp, q, k, v, [0, 700])
    assert st == 0 and bool((out.double() >= big * (1 - 2.0 ** -6)).all())
    check_prompt(kvp, q, k, normal(7, 700, 1, d, scale=2.0 ** -70), [0, 700])


@pytest.mark.parametrize("d, g", [(128, 4), (64, 3), (128, 1)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 5, 130, 299])
def test_prompt_masked_places_hold_anything(kvp, d, g, bad, at):
    """A key or value that is no number touches the rows that see it, and no other row."""
    lens = [200, 300, 90]
    start = starts(lens, gap=9)
    q, k, v = (x.contiguous() for x in qkv(41, start[-1], 2 * g, 2, d))
    want, lse = check_prompt(kvp, q, k, v, start, lens)
    row = start[1] + at
    mine = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for a, n in zip(start, lens):
        mine[a:a + n] = True
    for x in (q, k, v):                                      # between the sequences
        x[~mine] = bad
    sees = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    sees[row:start[1] + lens[1]] = True
    vv = v.clone()
    vv[row, 1, 3] = bad
    out, lse2, st = run_prompt(kvp, q, k, vv, start, lens)
    hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    hit[row:start[1] + lens[1], g:, 3] = True
    assert st == 0 and torch.equal(out[mine & ~sees], want[mine & ~sees])
    assert not bool(torch.isfinite(out[hit]).any()) and torch.equal(out[mine][~hit[mine]], want[mine][~hit[mine]])
    assert torch.equal(lse2[:, mine], lse[:, mine])
    if bad != bad:
        assert bool(torch.isnan(out[hit]).all())
    kk = k.clone()
    kk[row, 0, 1] = bad
    out, lse2, st = run_prompt(kvp, q, kk, v, start, lens)
    assert st == 0 and torch.equal(out[mine & ~sees], want[mine & ~sees])
    assert torch.equal(out[mine][:, g:], want[mine][:, g:]) and torch.equal(lse2[g:][:, mine], lse[g:][:, mine])
    if bad != bad:
        assert bool(torch.isnan(out[sees][:, :g]).all()) and bool(torch.isnan(lse2[:g][:, sees]).all())


def test_prompt_infinite_values_keep_their_sign(kvp):
    q, k, v = (x.contiguous() for x in qkv(43, 400, 2, 1, 128))
    v[10, 0, 5], v[390, 0, 6], v[391, 0, 6], v[380, 0, 7] = math.inf, -math.inf, math.inf, -math.inf
    out, _, st = run_prompt(kvp, q, k, v, [0, 400])
    assert st == 0
    assert bool((out[380:, :, 7] == -math.inf).all()) and bool(torch.isfinite(out[:380, :, 7]).all())
    assert bool((out[390, :, 6] == -math.inf).all()) and bool(torch.isnan(out[391:, :, 6]).all())
    assert bool((out[10:128, :, 5] == math.inf).all()) and bool((~torch.isfinite(out[128:, :, 5])).all())


def test_prompt_rows_without_a_finite_logit(kvp):
    q, k, v = (x.contiguous() for x in qkv(45, 300, 2, 1, 64))
    q[:], k[:200, 0, 0] = q.abs(), -math.inf
    out, lse, st = run_prompt(kvp, q, k, v, [0, 300])
    assert st == 0 and bool((out[:200] == 0).all()) and bool((lse[:, :200] == -math.inf).all())
    want, want_lse, tol, lse_tol = ref.attention(q[200:], k[200:], v[200:], [(0, 100)])
    ref.within(out[200:], want, tol, "out")
    ref.within(lse[:, 200:], want_lse, lse_tol, "lse")


@pytest.mark.parametrize("start, seq_len, bad", [
    ([0, 50, 40, 100], None, [1]), ([0, 50, 101, 100], None, [1, 2]), ([-1, 50, 60, 100], None, [0]),
    ([0, 50, 60, 100], [50, 11, 40], [1]), ([0, 50, 60, 100], [-1, 10, 40], [0])])
def test_prompt_bad_sequences_are_left_out(kvp, start, seq_len, bad):
    n = 100
    q, k, v = qkv(51, n, 4, 2, 128)
    out0 = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse, st = run_prompt(kvp, q, k, v, start, seq_len, out=out0)
    assert st == kvp.KVP_ERR_BOUNDS
    acc = torch.full((n, 2), -5.0, device="cuda")
    st2 = status()
    kvp.kvp_prompt_weights(q, k, i32(start), torch.zeros(4, n, device="cuda"),
                           seq_len=None if seq_len is None else i32(seq_len), acc=acc, status=st2)
    assert int(st2) == kvp.KVP_ERR_BOUNDS
    seqs = [s for s in ref.sequences(start, seq_len, n) if s is not None]
    assert len(seqs) == 3 - len(bad)
    mine = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, m in seqs:
        mine[a:a + m] = True
    assert bool((out[~mine] == 3.0).all()) and bool((acc[~mine] == -5.0).all())


def test_prompt_without_lse_or_status(kvp):
    q, k, v = qkv(52, 333, 8, 2, 128)
    want, _, _ = run_prompt(kvp, q, k, v, [0, 33, 333])
    assert torch.equal(kvp.kvp_prompt_attn(q, k, v, i32([0, 33, 333])), want)
    empty = kvp.kvp_prompt_attn(q[:0], k[:0], v[:0], i32([0, 0]))
    assert empty.shape == (0, 8, 128)
    kvp.kvp_prompt_attn(q, k, v, i32([0]), out=want)


def test_prompt_another_stream_and_graph(kvp):
    q, k, v = (x.contiguous() for x in qkv(53, 777, 8, 2, 128))
    start = i32([0, 400, 777])
    want, lse, _ = run_prompt(kvp, q, k, v, [0, 400, 777])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvp.kvp_prompt_attn(q, k, v, start, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, lse2, acc = torch.zeros_like(want), torch.zeros_like(lse), torch.zeros(777, 2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvp.kvp_prompt_attn(q, k, v, start, out=out, lse=lse2)
        kvp.kvp_prompt_weights(q, k, start, lse2, acc=acc)
    for turn in range(3):
        q.copy_(normal(60 + turn, 777, 8, 128))
        start.copy_(i32([0, 100 + 200 * turn, 777]))
        graph.replay()
        want, lse, _ = run_prompt(kvp, q, k, v, start.tolist())
        assert torch.equal(out, want) and torch.equal(lse2, lse)
        assert torch.equal(acc, kvp.kvp_prompt_weights(q, k, start, lse))


def test_prompt_is_repeatable_beside_other_work(kvp):
    q, k, v = qkv(54, 1500, 8, 2, 128)
    start = [0, 1, 600, 1500]
    want, lse, _ = run_prompt(kvp, q, k, v, start)
    acc = kvp.kvp_prompt_weights(q, k, i32(start), lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):
        outs.append(kvp.kvp_prompt_attn(q, k, v, i32(start)))
        with torch.cuda.stream(side):
            outs.append(kvp.kvp_prompt_attn(q, k, v, i32(start)))
        assert torch.equal(kvp.kvp_prompt_weights(q, k, i32(start), lse), acc)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)


# ---------------------------------------------------------------------------- weights

def check_weights(kvp, q, k, start, seq_len=None, n_last=0, scale=0.0, by="token", lse=None):
    n, hq, d = q.shape
    h, n_seqs = k.shape[1], len(start) - 1
    seqs = ref.sequences(start, seq_len, n)
    if lse is None:
        lse = ref.attention(q, k, k, seqs, scale)[1].float()
    want, tol = ref.weights(q, k, lse, seqs, scale, n_last)
    most = max(1, max(m for _, m in seqs))
    acc = torch.full((n, h) if by == "token" else (n_seqs, h, most + 3), -5.0, device="cuda")
    if by == "padded":                                       # rows of a larger buffer
        acc = torch.full((n_seqs, h + 1, most + 60), -5.0, device="cuda")[:, :h, :most + 3]
    st = status()
    got = kvp.kvp_prompt_weights(q, k, i32(start), lse, seq_len=None if seq_len is None else i32(seq_len), n_last=n_last,
                                 scale=scale, acc=acc, status=st)
    assert got is acc and int(st) == 0
    left = torch.ones(acc.shape, dtype=torch.bool, device="cuda")
    for i, (a, m) in enumerate(seqs):
        mine = acc[a:a + m] if by == "token" else acc[i, :, :m].T
        ref.within(mine, want[a:a + m], tol[a:a + m], f"sequence {i}")
        (left[a:a + m] if by == "token" else left[i, :, :m])[:] = False
    assert bool((acc[left] == -5.0).all())


@pytest.mark.parametrize("h, g, d", SHAPES)
@pytest.mark.parametrize("lens, n_last", [([1], 0), ([2, 1, 3], 1), ([127, 129], 0), ([128, 0, 256], 32),
                                          ([255, 1, 257, 64], 100), ([700], 0), ([700, 130], 129)])
def test_weights(kvp, h, g, d, lens, n_last):
    start = starts(lens)
    q, k, _ = qkv(len(lens) + h, start[-1], h * g, h, d)
    check_weights(kvp, q, k, start, n_last=n_last, by="sequence" if n_last else "token")


@pytest.mark.parametrize("layout", ["packed", "heads", "own"])
@pytest.mark.parametrize("by", ["token", "sequence", "padded"])
def test_weights_layouts_padding_and_gaps(kvp, layout, by):
    lens = [100, 300, 0, 129]
    start = starts(lens, gap=37, first=5)
    q, k, _ = qkv(3, start[-1] + 50, 6, 2, 128, layout)
    check_weights(kvp, q, k, start, lens, by=by)
    check_weights(kvp, q, k, start, lens, n_last=10**6, by=by, scale=0.3)


@pytest.mark.parametrize("h, g, d, n, n_last", [(2, 4, 128, 2300, 0), (1, 3, 64, 4111, 0), (4, 1, 128, 5000, 32)])
def test_weights_long(kvp, h, g, d, n, n_last):
    q, k, _ = qkv(11, n, h * g, h, d)
    check_weights(kvp, q, k, [0, n], n_last=n_last)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_weights_masked_places_hold_anything(kvp, bad):
    lens = [200, 300, 90]
    start = starts(lens, gap=9)
    q, k, _ = (x.contiguous() for x in qkv(41, start[-1], 4, 2, 128))
    seqs = ref.sequences(start, lens, q.shape[0])
    lse = ref.attention(q, k, k, seqs)[1].float()
    mine = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for a, n in seqs:
        mine[a:a + n] = True
    lse[:, ~mine] = bad
    q[~mine], k[~mine] = bad, bad
    check_weights(kvp, q, k, start, lens, lse=lse)
    want = kvp.kvp_prompt_weights(q, k, i32(start), lse, seq_len=i32(lens))
    q[start[1] + 100, 1] = bad                               # a query that is no number touches the keys that it sees
    got = kvp.kvp_prompt_weights(q, k, i32(start), lse, seq_len=i32(lens))
    other = mine.clone()
    other[start[1]:start[1] + 101] = False
    assert torch.equal(got[other], want[other]) and torch.equal(got[mine][:, 1], want[mine][:, 1])
    if bad != bad:
        assert bool(torch.isnan(got[start[1]:start[1] + 101, 0]).all())
    kk = k.clone()
    kk[start[2] + 7, 1] = bad                                # a key that is no number: its own sum
    got2 = kvp.kvp_prompt_weights(q, kk, i32(start), lse, seq_len=i32(lens))
    same = mine.clone()
    same[start[2] + 7] = False
    assert torch.equal(got2[same][torch.isfinite(got[same])], got[same][torch.isfinite(got[same])])


def test_weights_of_queries_that_pay_nothing(kvp):
    q, k, _ = qkv(46, 300, 2, 1, 64)
    lse = ref.attention(q, k, k, [(0, 300)])[1].float()
    lse[:, 50:200] = -math.inf
    lse[1] = -math.inf
    check_weights(kvp, q, k, [0, 300], lse=lse)


@pytest.mark.parametrize("n_last", [0, 20, 200])
def test_weights_of_rows_that_are_no_number(kvp, n_last):
    """A NaN normaliser touches the keys that its query sees, not those after it."""
    q, k, _ = qkv(48, 500, 4, 2, 128)
    lse = ref.attention(q, k, k, [(0, 500)])[1].float()
    lse[0, 480], lse[2, 490:495] = math.nan, math.nan
    check_weights(kvp, q, k, [0, 500], lse=lse, n_last=n_last)
    got = kvp.kvp_prompt_weights(q, k, i32([0, 500]), lse, n_last=n_last)
    assert bool(torch.isnan(got[:481, 0]).all()) and not bool(torch.isnan(got[481:, 0]).any())
    assert bool(torch.isnan(got[:495, 1]).all()) and not bool(torch.isnan(got[495:, 1]).any())


def test_weights_short_sums_record_bounds(kvp):
    q, k, _ = qkv(47, 300, 2, 1, 64)
    lse = ref.attention(q, k, k, [(0, 300)])[1].float()
    whole = kvp.kvp_prompt_weights(q, k, i32([0, 300]), lse)
    room = torch.full((1, 1, 260), -5.0, device="cuda")
    st = status()
    kvp.kvp_prompt_weights(q, k, i32([0, 300]), lse, acc=room[:, :, :250], status=st)
    assert int(st) == kvp.KVP_ERR_BOUNDS and bool((room[:, :, 250:] == -5.0).all())
    assert torch.equal(room[0, 0, :250], whole[:250, 0])


# ---------------------------------------------------------------------------- decode attention that adds its weights

def cache_of(kvp, seed, counts, max_pages, d, h, t, spare=1, expired=0.2):
    """A cache with counts [B][H] entries: shuffled pages, positions in order, some entries expired."""
    b = len(counts)
    gen = torch.Generator().manual_seed(seed)
    need = [[(n + PAGE - 1) // PAGE for n in row] for row in counts]
    total = sum(map(sum, need)) + spare
    order = torch.randperm(total, generator=gen).tolist()
    table = torch.full((b, h, max_pages), -1, dtype=torch.int32)
    remap = torch.full((b, h, max_pages * PAGE), -1, dtype=torch.int32)
    at = 0
    for i in range(b):
        for j in range(h):
            table[i, j, :need[i][j]] = torch.tensor(order[at:at + need[i][j]], dtype=torch.int32)
            at += need[i][j]
            n = counts[i][j]
            remap[i, j, :n] = torch.randperm(t, generator=gen)[:n].sort().values.int()
    expire = torch.where(torch.rand(total, PAGE, generator=gen) < expired, t - 1, NEVER).int()
    return kvp.PagedKV(normal(seed, total, PAGE, d), normal(seed + 1, total, PAGE, d), expire.cuda(), table.cuda(),
                       remap.cuda(), i32(counts))


DECODE = [(1, 1, 1, 128, [[300]]), (2, 2, 2, 64, [[5, 0], [33, 200]]), (1, 3, 4, 128, [[1, 16, 700]]),
          (2, 1, 8, 64, [[17], [900]]), (1, 2, 4, 64, [[0, 0]]), (3, 1, 1, 64, [[15], [1], [4000]]),
          (1, 1, 8, 128, [[6000]]), (1, 2, 2, 128, [[2500, 1]])]


@pytest.mark.parametrize("b, h, g, d, counts", DECODE)
@pytest.mark.parametrize("grid_limit", [0, 3])
def test_decode_adds_its_weights(kvp, b, h, g, d, counts, grid_limit):
    most = max(max(r) for r in counts)
    t = most + 50
    cache = cache_of(kvp, 7 * b + g, counts, (most + PAGE - 1) // PAGE + 2, d, h, t)
    q = normal(1, b, h * g, d)
    acc = uniform(2, b, h, t + 5)
    before = acc.clone()
    want, tol = ref.decode(q, cache, t - 1, acc)
    ws = torch.zeros(kvp.kvp_decode_attn_acc_workspace_bytes(b, h * g, h, d, cache.max_pages), dtype=torch.uint8,
                     device="cuda")
    for _ in range(2):                                       # the workspace serves the next call
        acc.copy_(before)
        st, lse = status(), torch.empty(b, h * g, device="cuda")
        out = kvp.kvp_decode_attn_acc(q, cache, t - 1, acc, lse=lse, workspace=ws, grid_limit=grid_limit, status=st)
        assert int(st) == 0
        for got, w, e, name in zip((out, lse, acc), want, tol, ("out", "lse", "acc")):
            ref.within(got, w, e, name)
    quiet = want[2] == before.double()
    assert torch.equal(acc[quiet], before[quiet])
    plain = kvp.kvp_decode_attn(q, cache, t - 1, grid_limit=grid_limit)
    assert float((plain - out).abs().max()) <= 2.0 ** -14


def test_decode_sums_in_rows_of_a_larger_buffer(kvp):
    cache = cache_of(kvp, 3, [[90, 200], [40, 64]], 14, 128, 2, 220)
    q, now = normal(4, 2, 8, 128), i32([219])
    whole = torch.zeros(2, 3, 300, device="cuda")
    acc = whole[:, 1:, 20:260]
    want, tol = ref.decode(q, cache, 219, acc)
    out = kvp.kvp_decode_attn_acc_devpos(q, cache, now, acc)
    ref.within(acc, want[2], tol[2], "acc")
    ref.within(out, want[0], tol[0], "out")
    assert bool((whole[:, 0] == 0).all()) and bool((whole[:, :, :20] == 0).all()) and bool((whole[:, :, 260:] == 0).all())


def test_decode_positions_and_pages_out_of_range(kvp):
    cache = cache_of(kvp, 5, [[100, 100]], 8, 64, 2, 120, expired=0.0)
    cache.remap[0, 0, 3], cache.remap[0, 0, 50], cache.remap[0, 1, 99] = -1, 500, 125
    for g in (1, 4):
        q, acc, st = normal(6, 1, 2 * g, 64), torch.zeros(1, 2, 125, device="cuda"), status()
        want, tol = ref.decode(q, cache, 119, acc)
        out = kvp.kvp_decode_attn_acc(q, cache, 119, acc, status=st)
        assert int(st) == kvp.KVP_ERR_BOUNDS
        ref.within(out, want[0], tol[0], "out")
        ref.within(acc, want[2], tol[2], "acc")
    cache.page_table[0, 0, 2], cache.page_table[0, 1, 0] = cache.n_pages_cap, -5
    for g in (2, 8):
        q, acc, st = normal(6, 1, 2 * g, 64), torch.zeros(1, 2, 600, device="cuda"), status()
        want, tol = ref.decode(q, cache, 119, acc)
        out = kvp.kvp_decode_attn_acc(q, cache, 119, acc, status=st)
        assert int(st) == kvp.KVP_ERR_BOUNDS
        ref.within(out, want[0], tol[0], "out")


def test_decode_everything_expired(kvp):
    cache = cache_of(kvp, 8, [[60]], 4, 128, 1, 80, expired=1.1)
    for g in (1, 4):
        acc = torch.full((1, 1, 80), 2.5, device="cuda")
        lse = torch.zeros(1, g, device="cuda")
        out = kvp.kvp_decode_attn_acc(normal(1, 1, g, 128), cache, 79, acc, lse=lse)
        assert bool((out == 0).all()) and bool((acc == 2.5).all()) and bool((lse == -math.inf).all())


# ---------------------------------------------------------------------------- eviction

def heavy(seed, *shape):
    """Weight sums with ties: a few values, zeros of both signs, some large."""
    x = (uniform(seed, *shape) * 6).floor() * 0.25
    y = uniform(seed + 1, *shape)
    return torch.where(y < 0.1, -0.0, torch.where(y > 0.9, uniform(seed + 2, *shape) * 1e3, x))


@pytest.mark.parametrize("b, h, t", [(1, 1, 1), (2, 3, 7), (1, 2, 511), (3, 1, 512), (2, 2, 513), (1, 1, 5000), (1, 3, 2049)])
@pytest.mark.parametrize("budget, recent", [(0, 0), (1, 0), (5, 3), (200, 64), (10**6, 1), (3, 10**6), (400, 0)])
def test_evict_dense(kvp, b, h, t, budget, recent):
    acc = heavy(t, b, h, t)
    want, kept = ref.evict_dense(acc.cpu(), t - 1, budget, recent)
    expire, count = kvp.kvp_evict(acc, t - 1, budget=budget, recent=recent)
    assert torch.equal(count.cpu(), kept) and torch.equal(expire.cpu(), want)
    by_token = acc.permute(0, 2, 1).contiguous().permute(0, 2, 1)
    assert torch.equal(kvp.kvp_evict(by_token, t - 1, budget=budget, recent=recent)[0].cpu(), want)


@pytest.mark.parametrize("t", [40000, 131072, 131071])
def test_evict_dense_long(kvp, t):
    for seed, acc in ((1, heavy(1, 1, 2, t)), (2, torch.exp(2 * torch.randn(1, 2, t, device="cuda"))),
                      (3, torch.full((1, 2, t), 0.5, device="cuda"))):
        budget = t // 4 + seed
        key = acc.clone()
        key[..., t - 128:] = math.inf                        # the recent ones first, then by weight, then by position
        order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
        want = torch.full((1, 2, t), t - 1, dtype=torch.int32, device="cuda")
        want.scatter_(2, order, NEVER)
        expire, count = kvp.kvp_evict(acc, t - 1, budget=budget, recent=128)
        assert bool((count == budget).all()) and torch.equal(expire, want)


def test_evict_no_numbers_and_infinities(kvp):
    acc = heavy(3, 2, 2, 300)
    y = uniform(9, 2, 2, 300)
    acc[y < 0.2], acc[(y > 0.2) & (y < 0.3)], acc[y > 0.9], acc[(y > 0.8) & (y < 0.9)] = math.nan, -math.inf, math.inf, -3.0
    for budget in (10, 60, 100, 200, 250, 280, 299):
        want, kept = ref.evict_dense(acc.cpu(), 299, budget, 20)
        expire, count = kvp.kvp_evict(acc, 299, budget=budget, recent=20)
        assert torch.equal(count.cpu(), kept) and torch.equal(expire.cpu(), want), budget
    expire, count = kvp.kvp_evict(acc[:, :, :0], 299, budget=5)
    assert expire.shape == (2, 2, 0) and bool((count == 0).all())
    expire, _ = kvp.kvp_evict(acc, 1000, budget=50, recent=800)   # a step later than the last position
    assert torch.equal(expire.cpu(), ref.evict_dense(acc.cpu(), 1000, 50, 800)[0])


def test_evict_ranks_every_nan_lowest(kvp):
    # NaN of both signs and of several payloads, one class, below -inf: the first of them go last
    bits = i32([0x7F800001, 0x7FFFFFFF, 0x7FC00000, -1, -0x400000, -0x7FFFFF])   # the last three are negative ones
    for t in (600, 40000):
        acc = heavy(4, 1, 1, t)
        at = torch.arange(7, t - 20, 13, device="cuda")
        acc[0, 0, at] = bits[torch.arange(len(at), device="cuda") % 6].view(torch.float32)
        acc[0, 0, at + 1] = -math.inf
        n = t - 10 - len(at)                                                     # candidates that are numbers
        for budget in (10 + n - 3, 10 + n, 10 + n + 5):
            expire, count = kvp.kvp_evict(acc, t - 1, budget=budget, recent=10)
            kept = at[expire[0, 0, at] == NEVER]
            assert int(count) == budget and int((expire == NEVER).sum()) == budget
            assert torch.equal(kept, at[:max(0, budget - 10 - n)])


@pytest.mark.parametrize("counts", [[[1]], [[0, 40], [700, 16]], [[3000, 5], [17, 2047]], [[9000]], [[70000, 20]]])
@pytest.mark.parametrize("budget, recent", [(0, 0), (30, 10), (500, 64), (10**6, 5), (2, 10**6)])
def test_evict_paged(kvp, counts, budget, recent):
    h, most = len(counts[0]), max(max(r) for r in counts)
    t = most + 100
    cache = cache_of(kvp, most, counts, (most + PAGE - 1) // PAGE + 1, 64, h, t)
    acc = heavy(5, len(counts), h, t + 8)
    pool, kept = ref.evict_paged(cache, acc.cpu(), t - 1, budget, recent)
    first = cache.expire_pool.clone()
    got, st = torch.empty(len(counts), h, dtype=torch.int32, device="cuda"), status()
    kvp.kvp_evict_paged(cache, acc, t - 1, budget=budget, recent=recent, kept=got, status=st)
    assert int(st) == 0 and torch.equal(got.cpu(), kept) and torch.equal(cache.expire_pool.cpu(), pool)
    kvp.kvp_evict_paged(cache, acc, t - 1, budget=budget, recent=recent, kept=got)   # once more: nothing more to go
    assert torch.equal(got.cpu(), kept) and torch.equal(cache.expire_pool.cpu(), pool)
    cache.expire_pool.copy_(first)
    kvp.kvp_evict_paged_devpos(cache, acc, i32([t - 1]), budget=budget, recent=recent)
    assert torch.equal(cache.expire_pool.cpu(), pool)


def test_evict_paged_out_of_range(kvp):
    cache = cache_of(kvp, 4, [[100, 90]], 8, 64, 2, 150, expired=0.1)
    acc = heavy(6, 1, 2, 140)
    cache.page_table[0, 0, 1], cache.page_table[0, 1, 2] = -2, cache.n_pages_cap
    cache.remap[0, 1, 5] = -1
    pool, kept = ref.evict_paged(cache, acc.cpu(), 149, 30, 20)
    st, got = status(), torch.empty(1, 2, dtype=torch.int32, device="cuda")
    kvp.kvp_evict_paged(cache, acc, 149, budget=30, recent=20, kept=got, status=st)
    assert int(st) == kvp.KVP_ERR_BOUNDS
    assert torch.equal(got.cpu(), kept) and torch.equal(cache.expire_pool.cpu(), pool)
    for now in (-1, NEVER):
        st = status()
        kvp.kvp_evict_paged_devpos(cache, acc, i32([now]), budget=0, recent=0, status=st)
        assert int(st) == kvp.KVP_ERR_INVALID and torch.equal(cache.expire_pool.cpu(), pool)


def test_evict_other_caches(kvp):
    """The tables of a latent cache (one head, no head dimension) and of an 8-bit cache."""
    lat = kvp.LatentPagedKV.allocate(2, 12, 5)
    src = cache_of(kvp, 12, [[70], [33]], 5, 64, 1, 90)
    for name in ("expire_pool", "page_table", "remap", "count"):
        t = getattr(lat, name)
        x = getattr(src, name)
        t.view(-1)[:x.numel()] = x.view(-1)
    acc = heavy(8, 2, 1, 90)
    pool, kept = ref.evict_paged(src, acc.cpu(), 89, 25, 8)
    got = torch.empty(2, 1, dtype=torch.int32, device="cuda")
    kvp.kvp_evict_paged(lat, acc, 89, budget=25, recent=8, kept=got)
    assert torch.equal(got.cpu(), kept) and torch.equal(lat.expire_pool[:len(pool)].cpu(), pool)
    b8 = kvp.Block8PagedKV.allocate(2, 1, 64, src.n_pages_cap, 5)
    for name in ("expire_pool", "page_table", "remap", "count"):
        getattr(b8, name).copy_(getattr(src, name))
    kvp.kvp_evict_paged(b8, acc, 89, budget=25, recent=8)
    assert torch.equal(b8.expire_pool.cpu(), pool)


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("h, g, d", [(2, 4, 128), (3, 1, 64)])
def test_a_prompt_and_its_decode_steps(kvp, h, g, d):
    """As they are used: a batch of padded prompts attended, the weights that their keys received, the budget's entries
    compacted, then decode steps that append, attend, add their weights, evict and re-compact, the attention checked
    against 64 bits over what is kept, the sums and the evictions against their restatement."""
    b, t, steps, budget, recent = 2, 300, 40, 96, 16
    hq = h * g
    lens, start = [t, t], [0, t, 2 * t]
    q, k, v = qkv(71, b * t, hq, h, d)
    out, lse = check_prompt(kvp, q, k, v, start)
    acc = torch.zeros(b, h, t + steps, device="cuda")
    kvp.kvp_prompt_weights(q, k, i32(start), lse, acc=acc)
    want, tol = ref.weights(q, k, lse, [(0, t), (t, t)])
    for i in range(b):
        ref.within(acc[i, :, :t].T, want[i * t:(i + 1) * t], tol[i * t:(i + 1) * t], "prompt sums")
    assert bool((acc[:, :, t:] == 0).all())
    expire, count = kvp.kvp_evict(acc[:, :, :t], t - 1, budget=budget, recent=recent)
    assert torch.equal(expire.cpu(), ref.evict_dense(acc[:, :, :t].cpu(), t - 1, budget, recent)[0])
    assert bool((count == budget).all())
    pages = (budget + steps) // PAGE + 2
    caches = [kvp.PagedKV.allocate(b, h, d, b * h * pages, pages) for _ in range(2)]
    st = status()
    kvp.kvp_compact(k.unflatten(0, (b, t)), v.unflatten(0, (b, t)), expire, t - 1, steps, caches[0], status=st)
    cache = caches[0]
    kept = expire == NEVER
    assert torch.equal(cache.count, kept.sum(-1).int())
    tau = torch.full((b, h), -math.inf, device="cuda")
    for step in range(steps):
        now = t + step
        new = normal(500 + step, b, hq + 2 * h, d)
        qn, kn, vn = new[:, :hq].contiguous(), new[:, hq:hq + h].contiguous(), new[:, hq + h:].contiguous()
        kvp.kvp_append(cache, kn, vn, now, mode=kvp.KVP_MASK_KVZAP, score=torch.zeros(b, h, device="cuda"), tau=tau,
                       status=st)
        want, tol = ref.decode(qn, cache, now, acc)
        o = kvp.kvp_decode_attn_acc(qn, cache, now, acc, status=st)
        ref.within(o, want[0], tol[0], f"step {step}: out")
        ref.within(acc, want[2], tol[2], f"step {step}: sums")
        if step % 7 == 6:
            pool, left = ref.evict_paged(cache, acc.cpu(), now, budget, recent)
            kvp.kvp_evict_paged(cache, acc, now, budget=budget, recent=recent, status=st)
            assert torch.equal(cache.expire_pool.cpu(), pool) and bool((left == budget).all())
        if step % 14 == 13:
            dst = caches[1] if cache is caches[0] else caches[0]
            kvp.kvp_compact_paged(cache, now, steps, dst, status=st)
            cache = dst
            assert bool((cache.count == budget).all())
    assert int(st) == 0


def test_a_captured_step(kvp):
    """Append, attention, sums and eviction as one graph, replayed step by step, against the same calls made eagerly."""
    b, h, g, d, t, steps, budget = 2, 2, 4, 128, 200, 24, 60
    two = [cache_of(kvp, 77, [[60, 60], [60, 60]], 8, d, h, t, spare=0, expired=0.0) for _ in range(2)]
    for c in two:                                            # room for the steps: pages of their own for every head
        c.page_table[:, :, :6] = torch.arange(24, dtype=torch.int32, device="cuda").view(b, h, 6)
        for name in ("k_pool", "v_pool", "expire_pool"):
            x = getattr(c, name)
            setattr(c, name, torch.cat([x, torch.zeros(24 - len(x), *x.shape[1:], dtype=x.dtype, device="cuda")]) if len(x) < 24 else x)
    accs = [torch.zeros(b, h, t + steps, device="cuda") for _ in range(2)]
    inputs = normal(78, steps, b, h * g + 2 * h, d)
    x = torch.empty_like(inputs[0])
    q, k, v = x[:, :h * g].contiguous(), x[:, h * g:h * g + h].contiguous(), x[:, h * g + h:].contiguous()
    pos, st, tau = i32([t]), status(), torch.full((b, h), -math.inf, device="cuda")
    score, out = torch.zeros(b, h, device="cuda"), torch.zeros(b, h * g, d, device="cuda")
    ws = torch.zeros(kvp.kvp_decode_attn_acc_workspace_bytes(b, h * g, h, d, 8), dtype=torch.uint8, device="cuda")

    def step(cache, acc):
        kvp.kvp_append_devpos(cache, k, v, pos, mode=kvp.KVP_MASK_KVZAP, score=score, tau=tau, status=st)
        kvp.kvp_decode_attn_acc_devpos(q, cache, pos, acc, out=out, workspace=ws, status=st)
        kvp.kvp_evict_paged_devpos(cache, acc, pos, budget=budget, recent=8, status=st)

    count0 = two[0].count.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(two[0], accs[0])
    torch.cuda.synchronize()
    assert torch.equal(two[0].count, count0)                 # a capture runs nothing
    outs = []
    for which in range(2):
        got = []
        for i in range(steps):
            for dst, src in ((q, inputs[i, :, :h * g]), (k, inputs[i, :, h * g:h * g + h]), (v, inputs[i, :, h * g + h:])):
                dst.copy_(src)
            pos.fill_(t + i)
            graph.replay() if which == 0 else step(two[1], accs[1])
            got.append(out.clone())
        outs.append(torch.stack(got))
    assert int(st) == 0 and torch.equal(outs[0], outs[1]) and torch.equal(accs[0], accs[1])
    assert torch.equal(two[0].expire_pool, two[1].expire_pool) and torch.equal(two[0].count, two[1].count)


# ---------------------------------------------------------------------------- guard bands

def test_nothing_is_written_outside_the_outputs(kvp):
    """Every output between two bands of a sentinel byte, workspaces of exactly the size asked for."""
    bands = []

    def g(shape, dtype, fill=0):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((4096 + n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        x = raw[4096:4096 + n].view(dtype).view(shape)
        x.fill_(fill)
        bands.append((raw, n))
        return x

    for lens, h, gr, d in (([130, 1, 77], 2, 4, 128), ([260], 1, 3, 64)):
        start = starts(lens)
        n, hq = start[-1], h * gr
        q, k, v = qkv(5, n, hq, h, d)
        out, lse, st = g((n, hq, d), torch.bfloat16), g((hq, n), torch.float32), g((1,), torch.int32)
        kvp.kvp_prompt_attn(q, k, v, i32(start), out=out, lse=lse, status=st)
        by_token, by_seq = g((n, h), torch.float32), g((len(lens), h, max(lens)), torch.float32)
        kvp.kvp_prompt_weights(q, k, i32(start), lse, acc=by_token, status=st)
        kvp.kvp_prompt_weights(q, k, i32(start), lse, acc=by_seq, n_last=9, status=st)
        kvp.kvp_evict(by_seq, max(lens) - 1, budget=20, recent=4, expire=g(by_seq.shape, torch.int32),
                      count=g(by_seq.shape[:2], torch.int32))
        for group in (1, 2, 4, 8):
            c = cache_of(kvp, 6, [[100, 60], [16, 0]], 7, d, 2, 120)
            c.expire_pool = g(c.expire_pool.shape, torch.int32, NEVER)
            acc = g((2, 2, 120), torch.float32)
            ws = g((kvp.kvp_decode_attn_acc_workspace_bytes(2, 2 * group, 2, d, 7),), torch.uint8)
            kvp.kvp_decode_attn_acc(normal(7, 2, 2 * group, d), c, 119, acc, out=g((2, 2 * group, d), torch.float32),
                                    lse=g((2, 2 * group), torch.float32), workspace=ws, status=st)
            kvp.kvp_evict_paged(c, acc, 119, budget=30, recent=5, kept=g((2, 2), torch.int32), status=st)
        assert int(st) == 0
    torch.cuda.synchronize()
    for raw, n in bands:
        assert bool((raw[:4096] == 0x5A).all()) and bool((raw[4096 + n:] == 0x5A).all())
