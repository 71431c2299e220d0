"""Attention over whole prompts, what it pays to each cached token, and eviction down to a budget by those weights.

Four operators, measured case by case:

  prompt   causal attention over packed prompts of different lengths, with each row's log-sum-exp (kvp_prompt_attn)
  weights  the attention weight that each key of a prompt received, summed over queries and shared heads
           (kvp_prompt_weights)
  decode   single-query attention over the paged cache that adds its weights to such sums (kvp_decode_attn_acc)
  evict    the entries that stay within a budget: the recent ones and the heaviest of the others, over a prompt's
           dense sums (kvp_evict) or a paged cache in use (kvp_evict_paged)

With `own` false, `run` computes them in plain torch operations in 32 bits; with `own` true, it calls the
framework. `exact` restates each operator in 64 bits, apart from both.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
NEVER = 2**31 - 1
ROWS = 1024                                               # queries that the plain forms take at once


# ---------------------------------------------------------------------------- cases

def listed():
    ragged = "1531 37 4099 211 1 907 128 2048 63 1200 640 333 1777 95 512 1024 129 750 17 403 256 88 1111 5"
    return [
        # a short chat turn of one user: latency of one call
        dict(name="prompt_chat", op="prompt", lens="509", kv_heads=8, group=4, dim=128),
        # a Llama-3-8B-shaped layer of a serving batch, its prompts packed
        dict(name="prompt_packed_8b", op="prompt", lens=ragged, kv_heads=8, group=4, dim=128),
        # one long document through the same layer
        dict(name="prompt_long_8b", op="prompt", lens="16384", kv_heads=8, group=4, dim=128),
        # odd head counts and lengths, narrow heads
        dict(name="prompt_odd", op="prompt", lens="1999 65 3001 129 700", kv_heads=5, group=7, dim=64),
        # every query of a prompt counts
        dict(name="weights_8b_layer", op="weights", lens="8192", kv_heads=8, group=4, dim=128, last=0, by="token"),
        # the last 32 queries of each prompt of a batch judge the whole of it
        dict(name="weights_window", op="weights", lens=" ".join(["8192"] * 16), kv_heads=8, group=4, dim=128, last=32,
             by="sequence"),
        # a Llama-65B-shaped layer without shared heads, ragged
        dict(name="weights_65b_odd", op="weights", lens="4099 1 997 37 2048", kv_heads=64, group=1, dim=128, last=0,
             by="sequence"),
        # a decode step of a Llama-3-8B-shaped layer, a quarter of the entries kept
        dict(name="decode_8b_layer", op="decode", batch=16, tokens=8192, kv_heads=8, group=4, dim=128, keep=0.26),
        # a Llama-65B-shaped layer at a long context
        dict(name="decode_65b_long", op="decode", batch=1, tokens=131072, kv_heads=64, group=1, dim=128, keep=0.25),
        # a quarter of a long prompt's entries stays, head by head
        dict(name="evict_prompt_65b", op="evict", form="dense", batch=1, tokens=131072, kv_heads=64, budget=0.25,
             recent=128, by="head"),
        # sums that lie token by token, odd sizes
        dict(name="evict_prompt_odd", op="evict", form="dense", batch=3, tokens=10007, kv_heads=5, budget=0.4, recent=33,
             by="token"),
        # between two decode steps: the 64 entries above the budget go
        dict(name="evict_step", op="evict", form="paged", batch=16, tokens=2112, kv_heads=8, budget=2048, recent=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["prompt", "prompt", "weights", "decode", "evict"])
    dim = rng.choice([64, 128, 128])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 16, 32, 64])
    if op in ("prompt", "weights"):
        group = rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8])
        most = 4e9 if op == "prompt" else 1e9           # pairs of a query and a key, over the query heads
        lens = []
        for _ in range(log(1, 32)):
            left = most / (heads * group) - sum(0.5 * x * x for x in lens)
            if left < 1 or sum(lens) * heads * (group + 2) > 3e6:
                break
            lens.append(log(1, min(16384, math.sqrt(2 * left), 3e6 / (heads * (group + 2)))))
        c = dict(op=op, lens=" ".join(map(str, lens)), kv_heads=heads, group=group, dim=dim)
        return c if op == "prompt" else dict(c, last=rng.choice([0, 0, 1, 32, 100]), by=rng.choice(["token", "sequence"]))
    if op == "decode":
        group = rng.choice([1, 1, 2, 4, 4, 8])
        batch = log(1, 64)
        most = max(1, 2_000_000 // (batch * heads))
        return dict(op=op, batch=batch, tokens=log(1, min(131072, most)), kv_heads=heads, group=group, dim=dim,
                    keep=round(rng.uniform(0.1, 1.0), 3))
    batch = log(1, 32)
    recent = rng.choice([0, 1, 32, 128, 500])
    if rng.random() < 0.5:
        tokens = log(1, min(131072, max(1, 4_000_000 // (batch * heads))))
        return dict(op=op, form="dense", batch=batch, tokens=tokens, kv_heads=heads,
                    budget=round(rng.uniform(0.05, 0.95), 3), recent=recent, by=rng.choice(["head", "token"]))
    tokens = log(1, min(16384, max(1, 2_000_000 // (batch * heads))))
    return dict(op=op, form="paged", batch=batch, tokens=tokens, kv_heads=heads, budget=rng.randint(0, tokens),
                recent=recent)


def _lens(case):
    return [int(x) for x in case["lens"].split()]


def _budget(case):
    b = case["budget"]
    return b if isinstance(b, int) else int(b * case["tokens"])


# ---------------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, heads, dim):
    """Keys have channels that are larger than the others: a factor for each head and channel."""
    return torch.exp(0.3 * _normal(gen, heads, dim))


def _sums(gen, *shape):
    """Accumulated weights: a few entries have most of it, some (never looked at) have none."""
    x = torch.exp(2 * _normal(gen, *shape))
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.03, 0.0, x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    h = c["kv_heads"]
    if c["op"] in ("prompt", "weights"):
        g, d, lens = c["group"], c["dim"], _lens(c)
        n, hq = sum(lens), h * g
        starts = [0]
        for x in lens:
            starts.append(starts[-1] + x)
        s["lens"], s["starts"] = lens, starts
        s["seq_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        qkv = _normal(gen, n, hq + 2 * h, d)              # one projection's output: q, k and v are views of it
        qkv[:, hq:hq + h] *= _keys(gen, h, d)
        common = _normal(gen, h, 1, d)                    # what all queries of a head share, and a prompt's first key
        common /= common.norm(dim=-1, keepdim=True)       # answers: most heads pay it much
        qkv[:, :hq] += (2 * common.expand(h, g, d)).reshape(hq, d)
        qkv[s["seq_start"][:-1].long(), hq:hq + h] += 2.5 * math.sqrt(d) * common[:, 0]
        qkv = qkv.bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        s["lse"] = torch.zeros(hq, n, device="cuda")
        if c["op"] == "prompt":
            s["out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        else:                                             # the attention ran before: its log-sum-exps are there
            for rows, _, at, x in _logits(s):
                s["lse"][:, at:at + rows] = torch.logsumexp(x, -1)
            s["acc"] = torch.zeros(n, h, device="cuda") if c["by"] == "token" else \
                torch.zeros(len(lens), h, max(lens), device="cuda")
        return s
    b, t = c["batch"], c["tokens"]
    s["now"] = t - 1
    if c["op"] == "evict" and c["form"] == "dense":
        s["acc"] = _sums(gen, b, h, t) if c["by"] == "head" else _sums(gen, b, t, h).permute(0, 2, 1)
        s["expire"] = torch.empty(b, h, t, dtype=torch.int32, device="cuda")
        s["count"] = torch.empty(b, h, dtype=torch.int32, device="cuda")
        return s
    # a paged cache in use: pages handed out head after head, a little over what the entries take
    d = c.get("dim", 64)
    if c["op"] == "decode":
        count = ((c["keep"] + 0.03 * _normal(gen, b, h)) * t).round().clamp(min(t, 128), t).long()
    else:
        count = torch.full((b, h), t, device="cuda")
    pages = (count + 32 + PAGE - 1) // PAGE
    first = torch.cumsum(pages.view(-1), 0).view(b, h) - pages
    total, width = int(pages.sum()), int(pages.max())
    index = torch.arange(width, device="cuda")
    slot = torch.arange(width * PAGE, device="cuda")
    live = slot < count[..., None]
    where = torch.div(slot * t, count[..., None], rounding_mode="floor")   # positions: in order, spread over the prompt
    s["page_table"] = torch.where(index < pages[..., None], first[..., None] + index, -1).int()
    s["remap"] = torch.where(live, where, -1).int()
    s["count"] = count.int()
    # most rows stay; some wait for the end of their window, a few are gone since the last compaction
    low = torch.rand(b, h, width * PAGE, generator=gen, device="cuda")
    expire = torch.where(low < 0.02, s["now"], torch.where(low < 0.05, s["now"] + 1 + (low * 2000).int(), NEVER))
    pool = torch.zeros(total, PAGE, dtype=torch.int32, device="cuda")
    there = index < pages[..., None]
    pool[s["page_table"][there].long()] = torch.where(live, expire, 0).int().view(b, h, width, PAGE)[there]
    s["expire0"], s["expire_pool"] = pool, pool.clone()
    s["acc0"] = _sums(gen, b, h, t + 64)
    s["acc"] = s["acc0"].clone()
    if c["op"] == "decode":
        hq = h * c["group"]
        owner = torch.repeat_interleave(torch.arange(b * h, device="cuda"), pages.view(-1)) % h
        s["k_pool"] = (_normal(gen, total, PAGE, d) * _keys(gen, h, d)[owner][:, None]).bfloat16()
        s["v_pool"] = _normal(gen, total, PAGE, d).bfloat16()
        s["q"] = _normal(gen, b, hq, d).bfloat16()
        s["out"] = torch.empty(b, hq, d, device="cuda")
        s["lse"] = torch.empty(b, hq, device="cuda")
    else:
        s["k_pool"] = s["v_pool"] = torch.zeros(total, PAGE, d, dtype=torch.bfloat16, device="cuda")
        s["kept"] = torch.empty(b, h, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

def _logits(s):
    """(queries, keys, first query's row, logits [Hq, queries, keys] with -inf where a key comes later), piece by
    piece; of the last queries alone where only they count."""
    c = s["case"]
    h, g, d = c["kv_heads"], c["group"], c["dim"]
    last = c.get("last", 0)
    for n, at in zip(s["lens"], s["starts"]):
        k = s["k"][at:at + n].float().permute(1, 2, 0)                     # [H, d, n]
        for r in range(max(0, n - last) if last else 0, n, ROWS):
            e = min(n, r + ROWS)
            q = s["q"][at + r:at + e].float().view(e - r, h, g, d).permute(1, 2, 0, 3).reshape(h, g * (e - r), d)
            x = torch.matmul(q, k[:, :, :e]).mul_(1 / math.sqrt(d)).view(h * g, e - r, e)
            later = torch.arange(e, device="cuda") > torch.arange(r, e, device="cuda")[:, None]
            yield e - r, e, at + r, x.masked_fill_(later, -math.inf)


def _plain_prompt(s):
    c = s["case"]
    h, g, d = c["kv_heads"], c["group"], c["dim"]
    for rows, keys, at, x in _logits(s):
        start = max(b for b in s["starts"] if b <= at)
        top = x.amax(-1, keepdim=True)
        w = x.sub_(top).exp_()
        total = w.sum(-1, keepdim=True)
        v = s["v"][start:start + keys].float().permute(1, 0, 2)            # [H, keys, d]
        o = torch.matmul(w.view(h, g * rows, keys), v).view(h * g, rows, d) / total
        s["out"][at:at + rows] = o.permute(1, 0, 2)
        s["lse"][:, at:at + rows] = (top + torch.log(total))[..., 0]
    return s["out"], s["lse"]


def _plain_weights(s):
    c = s["case"]
    h, g = c["kv_heads"], c["group"]
    s["acc"].zero_()
    for rows, keys, at, x in _logits(s):
        i = max(i for i, b in enumerate(s["starts"][:-1]) if b <= at)
        w = x.sub_(s["lse"][:, at:at + rows, None]).exp_().view(h, g * rows, keys).sum(1)
        if c["by"] == "token":
            s["acc"][s["starts"][i]:s["starts"][i] + keys] += w.t()
        else:
            s["acc"][i, :, :keys] += w
    return s["acc"]


def _plain_decode(s):
    c = s["case"]
    b, h, g, d = c["batch"], c["kv_heads"], c["group"], c["dim"]
    s["acc"].copy_(s["acc0"])                             # the step is taken again: what it added is taken back first
    table = s["page_table"].clamp(min=0).long()
    n = table.shape[2] * PAGE
    k = s["k_pool"][table].float().view(b, h, n, d)
    x = torch.matmul(s["q"].float().view(b, h, g, d), k.transpose(2, 3)) * (1 / math.sqrt(d))
    del k
    live = (torch.arange(n, device="cuda") < s["count"][..., None]) & (s["expire_pool"][table].view(b, h, n) > s["now"])
    x = torch.where(live[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    v = s["v_pool"][table].float().view(b, h, n, d)
    w = w / torch.where(total > 0, total, 1)
    s["out"].copy_(torch.matmul(w, v).view(b, h * g, d))
    s["lse"].copy_((top + torch.log(total)).view(b, h * g))
    s["acc"].scatter_add_(2, s["remap"].clamp(min=0).long(), w.sum(2))
    return s["out"], s["lse"], s["acc"]


def _heaviest(acc, candidate, most):
    """The `most` [..., 1] heaviest candidates of each row, the first of equal ones."""
    order = torch.sort(torch.where(candidate, acc, -math.inf), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, torch.arange(acc.shape[-1], device="cuda").expand_as(order))
    return candidate & (rank < most)


def _plain_evict(s):
    c = s["case"]
    now, budget = s["now"], _budget(c)
    if c["form"] == "dense":
        t = torch.arange(c["tokens"], device="cuda")
        recent = (t > now - c["recent"]).expand(s["acc"].shape)
        keep = recent | _heaviest(s["acc"], ~recent, budget - recent.sum(-1, keepdim=True))
        s["expire"].copy_(torch.where(keep, NEVER, now))
        s["count"].copy_(keep.sum(-1))
        return s["expire"], s["count"]
    s["expire_pool"].copy_(s["expire0"])                  # the step is taken again: who went comes back first
    table = s["page_table"].clamp(min=0).long()
    slot = torch.arange(table.shape[2] * PAGE, device="cuda")
    page = table.repeat_interleave(PAGE, 2)
    there = (slot < s["count"][..., None]) & (s["expire_pool"][page, slot % PAGE] > now)
    pos = s["remap"].clamp(min=0).long()
    recent = there & (pos > now - c["recent"])
    keep = recent | _heaviest(s["acc"].gather(2, pos), there & ~recent, budget - recent.sum(-1, keepdim=True))
    gone = there & ~keep
    s["expire_pool"][page[gone], (slot % PAGE).expand(page.shape)[gone]] = now
    s["kept"].copy_(keep.sum(-1))
    return s["expire_pool"], s["kept"]


# ---------------------------------------------------------------------------- the framework's calls

def _own(s):
    import kv_cache_pruning_gb300 as kvp
    c = s["case"]
    if c["op"] == "prompt":
        kvp.kvp_prompt_attn(s["q"], s["k"], s["v"], s["seq_start"], out=s["out"], lse=s["lse"], status=s["status"])
        return s["out"], s["lse"]
    if c["op"] == "weights":
        return kvp.kvp_prompt_weights(s["q"], s["k"], s["seq_start"], s["lse"], n_last=c["last"], acc=s["acc"],
                                      status=s["status"])
    if c["op"] == "evict" and c["form"] == "dense":
        return kvp.kvp_evict(s["acc"], s["now"], budget=_budget(c), recent=c["recent"], expire=s["expire"],
                             count=s["count"])
    if "cache" not in s:                                  # the cache's handle and the workspace that a program keeps
        s["cache"] = kvp.PagedKV(s["k_pool"], s["v_pool"], s["expire_pool"], s["page_table"], s["remap"], s["count"])
        if c["op"] == "decode":
            s["ws"] = torch.zeros(kvp.kvp_decode_attn_acc_workspace_bytes(
                c["batch"], c["kv_heads"] * c["group"], c["kv_heads"], c["dim"], s["page_table"].shape[2]),
                dtype=torch.uint8, device="cuda")
    if c["op"] == "decode":
        s["acc"].copy_(s["acc0"])                         # the step is taken again: what it added is taken back first
        kvp.kvp_decode_attn_acc(s["q"], s["cache"], s["now"], s["acc"], out=s["out"], lse=s["lse"], workspace=s["ws"],
                                status=s["status"])
        return s["out"], s["lse"], s["acc"]
    s["expire_pool"].copy_(s["expire0"])                  # the step is taken again: who went comes back first
    kvp.kvp_evict_paged(s["cache"], s["acc"], s["now"], budget=_budget(c), recent=c["recent"], kept=s["kept"],
                        status=s["status"])
    return s["expire_pool"], s["kept"]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "weights": _plain_weights, "decode": _plain_decode,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    h = c["kv_heads"]
    if c["op"] in ("prompt", "weights"):
        g, d, lens = c["group"], c["dim"], _lens(c)
        n = sum(lens)
        if c["op"] == "prompt":
            pairs = h * g * sum(x * (x + 1) / 2 for x in lens)
            return {"bytes": 4 * n * d * h * (g + 1) + 4 * n * h * g, "flops": 4 * d * pairs}
        seen = [min(x, c["last"] or x) for x in lens]     # queries that count
        pairs = h * g * sum(a * x - a * (a - 1) / 2 for a, x in zip(seen, lens))
        return {"bytes": sum(seen) * h * g * (2 * d + 4) + n * h * (2 * d + 4), "flops": 2 * d * pairs}
    heads = c["batch"] * h
    if c["op"] == "decode":
        kept = heads * min(c["tokens"], max(128, c["tokens"] * c["keep"]))
        return {"bytes": kept * (4 * c["dim"] + 16 + 4 / PAGE) + heads * c["group"] * (6 * c["dim"] + 4),
                "flops": 4 * c["dim"] * kept * c["group"]}
    if c["form"] == "dense":
        return {"bytes": 8 * heads * c["tokens"], "flops": heads * c["tokens"]}
    return {"bytes": heads * c["tokens"] * (12 + 4 / PAGE), "flops": heads * c["tokens"]}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c = case
    h = c["kv_heads"]
    if c["op"] in ("prompt", "weights") and work(c)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if c["op"] in ("prompt", "weights"):
        g, d, lens, last = c["group"], c["dim"], s["lens"], c.get("last", 0)
        out = torch.zeros(sum(lens), h * g, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(h * g, sum(lens), dtype=torch.float64, device="cuda")
        acc = None if c["op"] == "prompt" else torch.zeros(s["acc"].shape, dtype=torch.float64, device="cuda")
        for i, (n, at) in enumerate(zip(lens, s["starts"])):
            tok = torch.arange(n, device="cuda")
            for j in range(h * g):
                k = s["k"][at:at + n, j // g].double()
                for a in range(n - min(n, last or n), n, 4096):
                    b = min(n, a + 4096)
                    x = s["q"][at + a:at + b, j].double() @ k[:b].T / d ** 0.5
                    x[tok[a:b, None] < tok[:b]] = -math.inf
                    if c["op"] == "prompt":
                        lse[j, at + a:at + b] = torch.logsumexp(x, 1)
                        out[at + a:at + b, j] = torch.softmax(x, 1) @ s["v"][at:at + b, j // g].double()
                    else:
                        paid = torch.exp(x - s["lse"][j, at + a:at + b].double()[:, None]).sum(0)
                        (acc[at:at + b, j // g] if c["by"] == "token" else acc[i, j // g, :b]).add_(paid)
        return (out, lse) if c["op"] == "prompt" else acc
    now = s["now"]
    if c["op"] == "decode":
        g, d = c["group"], c["dim"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        acc = s["acc0"].double()
        counts = s["count"].tolist()
        for i in range(c["batch"]):
            for j in range(h):
                n = counts[i][j]
                page = s["page_table"][i, j, :(n + PAGE - 1) // PAGE].long()
                there = (s["expire0"][page].view(-1)[:n] > now).nonzero()[:, 0]
                if not len(there):
                    continue
                heads = slice(j * g, (j + 1) * g)
                x = s["q"][i, heads].double() @ s["k_pool"][page].view(-1, d)[there].double().T / math.sqrt(d)
                w = torch.softmax(x, 1)
                lse[i, heads] = torch.logsumexp(x, 1)
                out[i, heads] = w @ s["v_pool"][page].view(-1, d)[there].double()
                acc[i, j, s["remap"][i, j, :n][there].long()] += w.sum(0)
        return out, lse, acc
    # whole numbers, one head after the other on the host: the heaviest by a sort of (weight, -position)
    acc, budget = s["acc"].cpu().numpy(), _budget(c)
    kept = np.zeros(acc.shape[:2], np.int32)
    if c["form"] == "dense":
        expire = np.full(acc.shape, now, np.int32)
        for i, j in np.ndindex(*kept.shape):
            old = np.arange(max(0, min(c["tokens"], now - c["recent"] + 1)))
            stay = np.lexsort((old, -acc[i, j, old]))[:max(0, budget - (c["tokens"] - len(old)))]
            expire[i, j, len(old):] = NEVER
            expire[i, j, stay] = NEVER
            kept[i, j] = c["tokens"] - len(old) + len(stay)
        return torch.from_numpy(expire), torch.from_numpy(kept)
    pool, table = s["expire0"].cpu().numpy().copy(), s["page_table"].cpu().numpy()
    remap, counts = s["remap"].cpu().numpy(), s["count"].cpu().numpy()
    for i, j in np.ndindex(*kept.shape):
        slot = np.arange(counts[i, j])
        page, row = table[i, j, slot // PAGE], slot % PAGE
        alive = pool[page, row] > now
        new = alive & (remap[i, j, slot] > now - c["recent"])
        old = slot[alive & ~new]
        order = np.lexsort((old, -acc[i, j, remap[i, j, old]]))
        room = max(0, budget - int(new.sum()))
        gone = old[order[room:]]
        pool[page[gone], row[gone]] = now
        kept[i, j] = int(new.sum()) + min(room, len(old))
    return torch.from_numpy(pool), torch.from_numpy(kept)
