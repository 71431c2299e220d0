"""Prompt attention in each of its ways of work, against the restatement in 64 bits (tests/prompt_ref.py). A call whose query
tiles fit the SMs takes one an item; larger ones take two: of two heads of a kv head, or, where those are odd in number, two
in a row of one head, of which the second may be past the sequence's end. Inputs here repeat their sequences until the calls
are of the way that a test names."""
import math

import pytest
import torch

import prompt_ref as ref
from test_gpu_prompt import check_prompt, i32, normal, qkv, run_prompt, starts

pytestmark = pytest.mark.gpu

ONE_TILE, BY_HEAD, BY_ROW = "one tile", "two heads", "two row tiles"
# kv heads, query heads of each: two heads an item, and two row tiles
EVEN, ODD = [(1, 2), (2, 4), (1, 8)], [(2, 1), (1, 3), (2, 7)]


def way(n_tok, n_seqs, hq, h):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return ONE_TILE if (n_tok // 128 + n_seqs) * hq <= sms else BY_ROW if hq // h % 2 else BY_HEAD


def repeated(lens, h, g):
    """The lengths, as often as it takes for a call to have more query tiles than the SMs take one by one."""
    out = list(lens)
    while way(sum(out), len(out), h * g, h) == ONE_TILE:
        out += lens
    assert way(sum(out), len(out), h * g, h) == (BY_ROW if g % 2 else BY_HEAD)
    return out


LENGTHS = [[1], [2, 1, 3], [127, 129], [128, 0, 256], [255, 1, 257, 64], [700], [385, 384], [513, 511, 120], [1100, 17]]


@pytest.mark.parametrize("h, g", EVEN + ODD)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENGTHS)
def test_lengths(kvp, h, g, d, lens):
    lens = repeated(lens, h, g)
    start = starts(lens)
    check_prompt(kvp, *qkv(len(lens) + h, start[-1], h * g, h, d), start)


@pytest.mark.parametrize("h, g", [(2, 4), (2, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["packed", "heads", "own"])
def test_layouts_padding_and_gaps(kvp, h, g, d, layout):
    lens = repeated([100, 300, 0, 129, 513], h, g)
    start = starts(lens, gap=37, first=5)
    q, k, v = qkv(3, start[-1] + 50, h * g, h, d, layout)
    check_prompt(kvp, q, k, v, start, lens)
    check_prompt(kvp, q, k, v, start)                        # every row between the starts


@pytest.mark.parametrize("h, g", [(2, 4), (2, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shift, step", [(8, 0), (0, 8), (8, 24), (16, 16), (0, 40)])
def test_outputs_that_are_16_bytes_aligned_or_32(kvp, h, g, d, shift, step):
    """Rows of `out` that begin at odd multiples of 16 bytes take another store than those at multiples of 32; both write
    the same rows, and nothing beside them."""
    lens = repeated([100, 0, 129, 401], h, g)
    start = starts(lens)
    n = start[-1]
    q, k, v = qkv(8, n, h * g, h, d)
    want, lse, _ = run_prompt(kvp, q, k, v, start)
    whole = torch.full((n, h * g * (d + step) + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = whole[:, shift:shift + h * g * (d + step)].view(n, h * g, d + step)[..., :d]
    assert (out.data_ptr() | out.stride(0) * 2 | out.stride(1) * 2) % 32 == (16 if (shift | step) % 16 else 0)
    got, lse2, st = run_prompt(kvp, q, k, v, start, out=out)
    assert st == 0 and torch.equal(got, want) and torch.equal(lse2, lse)
    out.fill_(3.0)
    assert bool((whole == 3.0).all())


@pytest.mark.parametrize("h, g", [(1, 2), (2, 4), (2, 1), (1, 3), (1, 5)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_no_number_touch_the_rows_that_see_them(kvp, h, g, d, bad):
    """In every tile of a sequence, the first and the second of an item's, masked for some rows and not for others."""
    lens = repeated([200, 650, 90], h, g)
    start = starts(lens, gap=9)
    n = start[-1]
    q, k, v = (x.contiguous() for x in qkv(41, n, h * g, h, d))
    want, lse, st = run_prompt(kvp, q, k, v, start, lens)
    assert st == 0
    mine = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, m in zip(start, lens):
        mine[a:a + m] = True
    for x in (q, k, v):                                      # between the sequences
        x[~mine] = bad
    places = {s: (0, 5, 127, 128, 130, 255, 256, 383, 384, 500, 511, 512, 640, 649) for s in (1, len(lens) - 2)}
    hit = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    for s, rows in places.items():
        assert lens[s] == 650
        for i, at in enumerate(rows):
            head, col = i % h, (7 * i) % d
            v[start[s] + at, head, col] = bad
            hit[start[s] + at:start[s] + 650, head * g:(head + 1) * g, col] = True
    out, lse2, st = run_prompt(kvp, q, k, v, start, lens)
    assert st == 0 and torch.equal(lse2[:, mine], lse[:, mine])
    assert torch.equal(out[mine][~hit[mine]], want[mine][~hit[mine]])
    assert not bool(torch.isfinite(out[hit]).any())
    if bad != bad:
        assert bool(torch.isnan(out[hit]).all())


@pytest.mark.parametrize("h, g", [(2, 2), (2, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_keep_their_sign(kvp, h, g, d):
    lens = repeated([400], h, g)
    start = starts(lens)
    q, k, v = (x.contiguous() for x in qkv(43, start[-1], h * g, h, d))
    at = torch.arange(start[-1], device="cuda") % 400
    for row, col, x in ((390, 6, -math.inf), (391, 6, math.inf), (388, 7, -math.inf), (300, 8, math.inf)):
        v[at == row, :, col] = x
    out, _, st = run_prompt(kvp, q, k, v, start)
    assert st == 0
    assert bool((out[at >= 388][:, :, 7] == -math.inf).all()) and bool(torch.isfinite(out[at < 388][:, :, 7]).all())
    assert bool((out[at == 390][:, :, 6] == -math.inf).all()) and bool(torch.isnan(out[at > 390][:, :, 6]).all())
    seen = (at >= 300) & (at < 384)                          # their own tile of keys; after it a weight of 0 would make NaN
    assert bool((out[seen][:, :, 8] == math.inf).all()) and bool((~torch.isfinite(out[at >= 384][:, :, 8])).all())


@pytest.mark.parametrize("h, g", [(1, 2), (1, 4), (2, 1), (1, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [0.02, 0.3, 5.0])
def test_references_that_move(kvp, h, g, d, step):
    """Every key beats all before it for some heads and some sequences, and none does for the others: one tile of an item
    rescales its sums while the other's run on."""
    lens = repeated([900, 130, 650], h, g)
    start = starts(lens)
    n = start[-1]
    q = torch.zeros(n, h * g, d, device="cuda")
    q[..., 0] = torch.where(torch.arange(h * g, device="cuda") % 2 == 0, 1.0, -1.0)
    for s in range(1, len(lens), 2):
        q[start[s]:start[s + 1]] *= -1
    k = torch.zeros(n, h, d, device="cuda")
    for a, m in zip(start, lens):
        k[a:a + m, :, 0] = torch.arange(m, device="cuda")[:, None] * step
        k[a + m // 2:a + m, :, 1] = 3.0                      # and a jump that the first tiles' rows do not see
    q[..., 1] = 4.0
    check_prompt(kvp, q.bfloat16(), k.bfloat16(), normal(4, n, h, d), start, scale=1.0)


@pytest.mark.parametrize("h, g", [(1, 2), (1, 3), (2, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grow", [2.0 ** 6, 2.0 ** 11, 2.0 ** 20, 2.0 ** 40])
def test_huge_logits(kvp, h, g, d, grow):
    """Logits up to 2^86, beside sequences of ordinary ones: powers of two of a small pattern, so that every product and sum
    is exact and ties are ties on both sides. The bounds are those of choices: a row of values' bf16 weights and its own
    rounding, relative to the largest value (2^-8 each, twice over), and a logarithm beside a reference of 24 bits."""
    lens = repeated([300, 520], h, g)
    start = starts(lens)
    n = start[-1]
    gen = torch.Generator().manual_seed(int(math.log2(grow)))
    q = torch.randint(-1, 2, (n, h * g, d), generator=gen).float().cuda()
    k = torch.randint(-1, 2, (n, h, d), generator=gen).float().cuda()
    for s in range(0, len(lens), 2):
        q[start[s]:start[s + 1]] *= grow
        k[start[s]:start[s + 1]] *= grow
    q, k, v = q.bfloat16(), k.bfloat16(), normal(9, n, h, d)
    out, lse, st = run_prompt(kvp, q, k, v, start, scale=1.0)
    want, want_lse, _, _ = ref.attention(q, k, v, ref.sequences(start, None, n), 1.0)
    assert st == 0
    assert bool(((out.double() - want).abs() <= 2.0 ** -6 * v.double().abs().max()).all())
    assert bool(((lse.double() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs() + 1e-5).all())


@pytest.mark.parametrize("h, g", [(2, 2), (2, 3), (2, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_large_and_small_values(kvp, h, g, d):
    lens = repeated([700, 129], h, g)
    start = starts(lens)
    n = start[-1]
    big = torch.finfo(torch.bfloat16).max
    q, k, _ = qkv(31, n, h * g, h, d)
    v = torch.full((n, h, d), big, dtype=torch.bfloat16, device="cuda")
    v[::2] = -big
    check_prompt(kvp, q, k, v, start)
    check_prompt(kvp, q, k, normal(7, n, h, d, scale=2.0 ** -70), start)


@pytest.mark.parametrize("h, g", [(2, 2), (2, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_way_of_work_changes_no_row(kvp, h, g, d):
    """A sequence's rows are the same bits alone, one tile an item, and among many, two an item; and each time."""
    lens = repeated([513, 200, 640], h, g)
    start = starts(lens)
    q, k, v = (x.contiguous() for x in qkv(55, start[-1], h * g, h, d))
    want, lse, _ = run_prompt(kvp, q, k, v, start)
    for _ in range(3):
        out, lse2, _ = run_prompt(kvp, q, k, v, start)
        assert torch.equal(out, want) and torch.equal(lse2, lse)
    for a, m in list(zip(start, lens))[:3]:
        assert way(m, 1, h * g, h) == ONE_TILE
        out, lse2, _ = run_prompt(kvp, q[a:a + m], k[a:a + m], v[a:a + m], [0, m])
        assert torch.equal(out, want[a:a + m]) and torch.equal(lse2, lse[:, a:a + m])


def test_rows_far_apart(kvp):
    """Rows 2^23 values apart: offsets of q, k, v and out pass 2^31 elements, and lie in one buffer of 4 heads' columns."""
    n, h, g, d, step = 600, 1, 2, 128, 2 ** 23
    assert (n - 1) * step > 2 ** 31
    room = torch.zeros(n * step, dtype=torch.bfloat16, device="cuda").view(n, step)
    q0, k0, v0 = (x.contiguous() for x in qkv(61, n, h * g, h, d))
    q, k, v = room[:, :h * g * d].view(n, h * g, d), room[:, 1000:1128].view(n, 1, d), room[:, 2000:2128].view(n, 1, d)
    out = room[:, step - 256:].view(n, h * g, d)
    for x, y in ((q, q0), (k, k0), (v, v0)):
        x.copy_(y)
    want, lse, _ = run_prompt(kvp, q0, k0, v0, [0, 250, n])
    got, lse2, st = run_prompt(kvp, q, k, v, [0, 250, n], out=out)
    assert st == 0 and torch.equal(got, want) and torch.equal(lse2, lse)
    sums = kvp.kvp_prompt_weights(q0, k0, i32([0, 250, n]), lse)
    far = torch.zeros(n * (step // 2), device="cuda").view(n, step // 2)[:, 7:8]
    assert torch.equal(kvp.kvp_prompt_weights(q, k, i32([0, 250, n]), lse, acc=far), sums)
