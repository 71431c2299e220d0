"""Prompt attention, the weights it pays, decode attention that adds its weights, and eviction to a budget, restated in
64 bits (torch float64, row by row of the definitions; no code shared with the library), with the error bounds that the
library's number formats allow."""
import math

import torch

NEVER = 2**31 - 1
PAGE = 16


def sequences(seq_start, seq_len, n_tok):
    """(first row, length) of every valid sequence (None: one that breaks the rules)."""
    out = []
    for i in range(len(seq_start) - 1):
        a, b = seq_start[i], seq_start[i + 1]
        n = b - a if seq_len is None else seq_len[i]
        out.append((a, n) if 0 <= a <= b <= n_tok and 0 <= n <= b - a else None)
    return out


def logits(q, k, scale):
    """Scaled logits [Hq, n, n] of one sequence, -inf where the key comes later, and a bound on an fp32 evaluation's
    error: d products of bf16 are exact, each of the d additions rounds (or truncates) to 24 bits of what is at most the
    sum of magnitudes, and the scale's product with log2 e and the subtraction of the reference round once each."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    kk = k.double().repeat_interleave(g, 1).permute(1, 2, 0)
    x = torch.matmul(q.double().permute(1, 0, 2), kk) * scale
    mag = torch.matmul(q.double().abs().permute(1, 0, 2), kk.abs()) * scale
    later = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
    err = (d + 4) * 2.0 ** -23 * torch.where(later | ~torch.isfinite(mag), 0.0, mag).amax(-1) if n else mag.sum(-1)
    return x.masked_fill(later, -math.inf), err


def attention(q, k, v, seqs, scale=None):
    """out [n_tok, Hq, d], lse [Hq, n_tok] in float64, and a bound on each one's error. Rows of no sequence: NaN."""
    n_tok, hq, d = q.shape
    g = hq // k.shape[1]
    scale = 1 / math.sqrt(d) if not scale else scale
    out = torch.full((n_tok, hq, d), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((hq, n_tok), math.nan, dtype=torch.float64, device=q.device)
    out_tol, lse_tol = out.clone(), lse.clone()
    for s in seqs:
        if s is None or s[1] == 0:
            continue
        a, n = s
        x, err = logits(q[a:a + n], k[a:a + n], scale)
        top = x.amax(-1, keepdim=True)
        w = torch.exp(x - top)
        total = w.sum(-1, keepdim=True)
        w = w / total
        vv = v[a:a + n].double().repeat_interleave(g, 1).permute(1, 0, 2)
        o = torch.matmul(w, vv)
        mean = torch.matmul(w, vv.abs())
        out[a:a + n] = o.permute(1, 0, 2)
        lse[:, a:a + n] = (top + torch.log(total))[..., 0]
        # a weight: rounded to bf16 (2^-8), off by its logit's error and the row's (2 err), the exponential and the sums'
        # rounding (2^-20 with n terms of 2^-24 each); then one rounding of the result
        rel = 2.0 ** -8 + 2 * err[..., None] + 2.0 ** -20 + n * 2.0 ** -23
        out_tol[a:a + n] = (rel * mean + 2.0 ** -8 * (o.abs() + rel * mean) + 2.0 ** -98 * n).permute(1, 0, 2)
        lse_tol[:, a:a + n] = err + 2.0 ** -22 * (lse[:, a:a + n].abs() + 1) + n * 2.0 ** -23
    return out, lse, out_tol, lse_tol


def weights(q, k, lse, seqs, scale=None, n_last=0):
    """acc [n_tok, H] in float64 from the given lse, and a bound on its error. Rows of no sequence: NaN."""
    n_tok, hq, d = q.shape
    h = k.shape[1]
    scale = 1 / math.sqrt(d) if not scale else scale
    acc = torch.full((n_tok, h), math.nan, dtype=torch.float64, device=q.device)
    tol = acc.clone()
    for s in seqs:
        if s is None or s[1] == 0:
            continue
        a, n = s
        x, err = logits(q[a:a + n], k[a:a + n], scale)
        ls = lse[:, a:a + n].double()
        later = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)      # whatever their lse is
        w = torch.where(torch.isneginf(ls)[..., None] | later, 0.0, torch.exp(x - ls[..., None]))
        rel = err + 2.0 ** -22 * (torch.where(torch.isfinite(ls), ls.abs(), 0.0) + 1)
        if n_last:
            w, rel = w[:, max(0, n - n_last):], rel[:, max(0, n - n_last):]
        acc[a:a + n] = w.reshape(h, -1, n).sum(1).T
        # partial sums of at most 128 weights, 2^-24 each, and their sum in turn
        tol[a:a + n] = ((w * rel[..., None]).reshape(h, -1, n).sum(1) + w.reshape(h, -1, n).sum(1) *
                        (160 + hq // h * n / 128) * 2.0 ** -24).T + 2.0 ** -120
    return acc, tol


def decode(q, cache, now, acc, scale=None):
    """out, lse, acc after the step (float64) and the bound on their errors: the weights keep at least 16 bits."""
    b, hq, d = q.shape
    h = cache.count.shape[1]
    g = hq // h
    scale = 1 / math.sqrt(d) if not scale else scale
    out = torch.zeros(b, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=q.device)
    acc = acc.double().clone()
    tols = [torch.zeros_like(x) for x in (out, lse, acc)]
    count, table, remap = cache.count.tolist(), cache.page_table.long(), cache.remap.long()
    for i in range(b):
        for j in range(h):
            n = min(max(count[i][j], 0), table.shape[2] * PAGE)
            slot = torch.arange(n, device=q.device)
            page, row = table[i, j, slot // PAGE], slot % PAGE
            fine = (page >= 0) & (page < cache.k_pool.shape[0])
            page = torch.where(fine, page, 0)
            there = fine & (cache.expire_pool[page, row] > now)
            page, row, pos = page[there], row[there], remap[i, j, :n][there]
            if not len(page):
                continue
            heads = slice(j * g, (j + 1) * g)
            k, v, qq = cache.k_pool[page, row].double(), cache.v_pool[page, row].double(), q[i, heads].double()
            x = qq @ k.T * scale
            err = ((d + 4) * 2.0 ** -23 * (qq.abs() @ k.abs().T) * scale).amax(1)
            w = torch.softmax(x, 1)
            out[i, heads], lse[i, heads] = w @ v, torch.logsumexp(x, 1)
            rel = 2 * err[:, None] + 2.0 ** -16 + 2.0 ** -20 + len(page) * 2.0 ** -24
            tols[0][i, heads] = rel * (w @ v.abs()) + 2.0 ** -22 * out[i, heads].abs()
            tols[1][i, heads] = err + 2.0 ** -22 * (lse[i, heads].abs() + 1) + len(page) * 2.0 ** -24
            ok = (pos >= 0) & (pos < acc.shape[2])
            acc[i, j].index_add_(0, pos[ok], w.sum(0)[ok])
            tols[2][i, j].index_add_(0, pos[ok], (w * (rel - 2.0 ** -16)).sum(0)[ok])
    tols[2] += 2.0 ** -23 * acc.abs()
    return (out, lse, acc), tols


def _rank_key(x):
    """Sort key: larger first, NaN below -inf, -0 equal to 0."""
    return (1, 0.0) if x != x else (0, -(x + 0.0))


def evict_dense(acc, now, budget, recent):
    """expire [B, H, T], count [B, H] (int32) by a sort of each (b, h)'s entries."""
    b, h, t = acc.shape
    expire = torch.full((b, h, t), NEVER, dtype=torch.int32)
    count = torch.zeros(b, h, dtype=torch.int32)
    for i in range(b):
        for j in range(h):
            row = acc[i, j].tolist()
            old = [x for x in range(t) if x <= now - recent]
            room = max(0, budget - (t - len(old)))
            gone = sorted(old, key=lambda x: (_rank_key(row[x]), x))[room:]
            expire[i, j, gone] = now
            count[i, j] = t - len(gone)
    return expire, count


def evict_paged(cache, acc, now, budget, recent):
    """expire_pool after the eviction, and kept [B, H]."""
    pool = cache.expire_pool.cpu().clone()
    table, remap, count = (x.cpu().tolist() for x in (cache.page_table, cache.remap, cache.count))
    b, h = len(count), len(count[0])
    kept = torch.zeros(b, h, dtype=torch.int32)
    for i in range(b):
        for j in range(h):
            row = acc[i, j].tolist()
            new, old = [], []
            for s in range(min(max(count[i][j], 0), len(table[i][j]) * PAGE)):
                page, pos = table[i][j][s // PAGE], remap[i][j][s]
                if not 0 <= page < pool.shape[0] or not 0 <= pos < len(row) or pool[page, s % PAGE] <= now:
                    continue
                (new if pos > now - recent else old).append((s, page, pos))
            room = max(0, budget - len(new))
            old.sort(key=lambda e: (_rank_key(row[e[2]]), e[0]))
            for s, page, _ in old[room:]:
                pool[page, s % PAGE] = now
            kept[i, j] = len(new) + min(room, len(old))
    return pool, kept


def within(got, want, tol, what):
    """Every element within its bound (non-finite ones alike)."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities differ"
    if fine.any():
        over = (got[fine] - want[fine]).abs() - tol[fine]
        assert over.max() <= 0, f"{what}: {float(over.max()):.3g} over its bound ({int((over > 0).sum())} elements)"
