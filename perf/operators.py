"""The 8-bit cache with a scale for each block of 16 tokens of a head, and what a decode step runs around it.

Five calls, measured case by case:

  attend   single-query attention over the 8-bit pages (kvp_decode_attn_block8)
  write    a prompt's keys and values, masked, quantised into pages (kvp_compact_block8)
  append   one decoded token into every head's page (kvp_append_block8)
  read     slots of the cache back as bf16 rows (kvp_read_block8)
  rotate   norms of queries and keys for each head and the position rotation (kvp_qk_norm_rope)

With `own` false, `run` computes them in plain torch operations in 32 bits; with `own` true, it calls the
framework. `exact` restates each operator in 64 bits, apart from both.
"""
import math

import torch

own = False

PAGE = 16
NEVER = 2**31 - 1
WINDOW = 128
MODES = {"kvzap": 0, "dms": 1}
FORMATS = {"e4m3": 0, "int8": 1}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # a short chat turn of one user, nothing pruned: latency of one call
        dict(name="attend_chat", op="attend", batch=1, tokens=509, kv_heads=8, group=4, dim=128, fmt="e4m3", keep=1.0),
        # a Llama-3-8B-shaped layer of a serving batch, a quarter kept
        dict(name="attend_llama3_8b_layer", op="attend", batch=16, tokens=8192, kv_heads=8, group=4, dim=128, fmt="e4m3",
             keep=0.26),
        # a Llama-65B-shaped layer without shared heads at a long context, keep rates ~ Beta(2, 5)
        dict(name="attend_llama65b_long", op="attend", batch=1, tokens=131072, kv_heads=64, group=1, dim=128, fmt="int8",
             keep=0.0),
        # odd head counts and lengths, narrow heads
        dict(name="attend_odd", op="attend", batch=3, tokens=5003, kv_heads=5, group=7, dim=64, fmt="int8", keep=0.61),
        # the same two layers' prompts written into the cache
        dict(name="write_llama3_8b_layer", op="write", batch=16, tokens=8192, kv_heads=8, dim=128, fmt="e4m3",
             mode="kvzap", keep=0.26),
        dict(name="write_long_flags", op="write", batch=1, tokens=65521, kv_heads=64, dim=128, fmt="int8", mode="dms",
             keep=0.5),
        # the decoded token of a serving batch; of many short sequences
        dict(name="append_batch16", op="append", batch=16, tokens=2047, kv_heads=8, dim=128, fmt="e4m3", mode="kvzap"),
        dict(name="append_batch128_mha", op="append", batch=128, tokens=203, kv_heads=32, dim=64, fmt="int8", mode="dms"),
        # one sequence moved out; a layer of a batch read back for another pass over its rows
        dict(name="read_one", op="read", batch=1, tokens=1111, kv_heads=8, dim=64, fmt="int8", first=5),
        dict(name="read_layer", op="read", batch=16, tokens=4096, kv_heads=8, dim=128, fmt="e4m3", first=0),
        # queries and keys of a decode step of 16 sequences; of a ragged prompt batch
        dict(name="rotate_decode", op="rotate", tokens=16, q_heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             norm=True),
        dict(name="rotate_prompt", op="rotate", tokens=65521, q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "write", "append", "read", "rotate"])
    dim = rng.choice([64, 128, 128])
    fmt = rng.choice(["e4m3", "int8"])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 16, 32, 64])
    if op == "attend":
        group = rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8, 8])
        batch = log(1, 64)
        most = max(1, 4_000_000 // (batch * heads * group))
        return dict(op=op, batch=batch, tokens=log(1, min(131072, most)), kv_heads=heads, group=group, dim=dim, fmt=fmt,
                    keep=round(rng.uniform(0.1, 1.0), 3))
    if op == "write":
        batch = log(1, 32)
        most = max(1, 4_000_000 // (batch * heads))
        return dict(op=op, batch=batch, tokens=log(1, min(131072, most)), kv_heads=heads, dim=dim, fmt=fmt,
                    mode=rng.choice(["kvzap", "dms"]), keep=round(rng.uniform(0.1, 1.0), 3))
    if op == "append":
        return dict(op=op, batch=log(1, 128), tokens=log(1, 512), kv_heads=heads, dim=dim, fmt=fmt,
                    mode=rng.choice(["kvzap", "dms"]))
    if op == "read":
        batch = log(1, 32)
        tokens = log(1, min(65536, max(1, 1_000_000 // (batch * heads))))
        return dict(op=op, batch=batch, tokens=tokens, kv_heads=heads, dim=dim, fmt=fmt,
                    first=rng.randrange(0, tokens))
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    most = max(1, 2_600_000 // (heads * (group + 1)))
    return dict(op=op, tokens=log(1, min(131072, most)), q_heads=heads * group, kv_heads=heads, dim=dim,
                rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7)


# ---------------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, heads, dim):
    """Keys have channels that are larger than the others: a factor for each head and channel."""
    return torch.exp(0.5 * _normal(gen, heads, dim))


def _block_scale(amax, fmt):
    """The power of two that takes a block whose largest magnitude is `amax` into the format's range (0: 0)."""
    mant, exp = torch.frexp(amax)                        # amax = mant * 2^exp, mant in [0.5, 1)
    e = exp - 9 + (mant > 0.875).int() if fmt == "e4m3" else exp - 7 + (mant > 127 / 128).int()
    power = ((e.clamp(min=-126) + 127) << 23).view(torch.float32)   # 2^e from its bits: exact
    return torch.where(amax > 0, power, torch.zeros_like(amax))


def _codes(x, scale, fmt):
    """x / scale rounded to the format: fp32 values -> the codes' bytes (scale 0: zero codes)."""
    y = x * torch.where(scale > 0, 1 / scale, scale)
    return (y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)).view(torch.uint8)


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _filled(gen, batch, heads, dim, fmt, count, width=None):
    """A cache of `count` [B, H] quantised rows for each head, pages handed out head after head: as many as the
    rows take, or `width` each."""
    pages = (count + PAGE - 1) // PAGE if width is None else torch.full_like(count, width)
    first = torch.cumsum(pages.view(-1), 0).view(batch, heads) - pages
    total, width = int(pages.sum()), int(pages.max())
    index = torch.arange(width, device="cuda", dtype=torch.int64)
    table = torch.where(index < pages[..., None], first[..., None] + index, -1)
    owner = torch.repeat_interleave(torch.arange(batch * heads, device="cuda"), pages.view(-1))
    row = (torch.arange(total, device="cuda") - first.view(-1)[owner])[:, None] * PAGE + \
        torch.arange(PAGE, device="cuda")                # [total, 16]: each row's slot in its head
    live = row < count.view(-1)[owner][:, None]
    pools, scales = [], []
    for chan in (_keys(gen, heads, dim)[owner % heads][:, None], 1.0):
        x = (_normal(gen, total, PAGE, dim) * chan).bfloat16().float() * live[..., None]
        s = _block_scale(x.abs().amax((1, 2)), fmt)
        pools.append(_codes(x, s[:, None, None], fmt))
        scales.append(s)
        del x
    slot = torch.arange(width * PAGE, device="cuda")
    remap = torch.where(slot < count[..., None], slot, -1)   # positions: what is kept, in order
    return dict(kq_pool=pools[0], vq_pool=pools[1], scale_pool=torch.stack(scales, 1).contiguous(), live=live,
                page_table=table.int(), remap=remap.int(), count=count.int())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["op"] == "rotate":
        n, hq, h, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
        qkv = _normal(gen, n, hq + 2 * h, d).bfloat16()   # one projection's output: q, k and v are views of it
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + h]
        start = torch.randint(0, 100_000, (1,), generator=gen, device="cuda")
        s["pos"] = (start + torch.arange(n, device="cuda")).int()
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        s["qw"] = 1 + 0.2 * _normal(gen, d) if c["norm"] else None
        s["kw"] = 1 + 0.2 * _normal(gen, d) if c["norm"] else None
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda")
        return s
    b, t, h, d = c["batch"], c["tokens"], c["kv_heads"], c["dim"]
    if c["op"] == "write":
        s["k"] = (_normal(gen, b, t, h, d) * _keys(gen, h, d)).bfloat16()
        s["v"] = _normal(gen, b, t, h, d).bfloat16()
        if c["mode"] == "kvzap":
            s["scores"] = _normal(gen, b, t, h)
            s["tau"] = torch.full((b, h), math.sqrt(2) * float(torch.erfinv(torch.tensor(1 - 2 * c["keep"]).clamp(-1, 1))),
                                  device="cuda").clamp(-10, 10) + 0.05 * _normal(gen, b, h)
        else:
            age = torch.randint(0, t, (b, h, t), generator=gen, device="cuda")
            gone = torch.rand(b, h, t, generator=gen, device="cuda") >= c["keep"]
            s["flag"] = torch.where(gone, age, -1).int()
        s["now"], s["reserve"] = t - 1, 32
        width = (t + s["reserve"] + PAGE - 1) // PAGE
        cap = b * h * width
        s["cache"] = dict(
            kq_pool=torch.zeros(cap, PAGE, d, dtype=torch.uint8, device="cuda"),
            vq_pool=torch.zeros(cap, PAGE, d, dtype=torch.uint8, device="cuda"),
            scale_pool=torch.zeros(cap, 2, device="cuda"),
            expire_pool=torch.zeros(cap, PAGE, dtype=torch.int32, device="cuda"),
            page_table=torch.full((b, h, width), -1, dtype=torch.int32, device="cuda"),
            remap=torch.full((b, h, width * PAGE), -1, dtype=torch.int32, device="cuda"),
            count=torch.zeros(b, h, dtype=torch.int32, device="cuda"))
        return s
    # a cache in use
    if c["op"] == "attend":
        x = _normal(gen, b, h, 7).square()                # keep 0: rates ~ Beta(2, 5), from gamma variables
        rate = x[..., :2].sum(-1) / x.sum(-1) if c["keep"] == 0 else c["keep"] + 0.03 * _normal(gen, b, h)
        count = (rate * t).round().clamp(min(t, WINDOW), t).long()
    else:                                                 # lengths differ a little from head to head
        count = (t * (1 - 0.2 * torch.rand(b, h, generator=gen, device="cuda"))).ceil().long()
    cache = _filled(gen, b, h, d, c["fmt"], count, t // PAGE + 1 if c["op"] == "append" else None)
    now = t - 1
    low = torch.rand(cache["live"].shape, generator=gen, device="cuda")
    # most rows stay; some wait for the end of their window, a few are gone since the last compaction
    expire = torch.where(low < 0.02, now, torch.where(low < 0.05, now + 1 + (low * 2000).int(), NEVER))
    cache["expire_pool"] = torch.where(cache.pop("live"), expire, 0).int().contiguous()
    s["cache"], s["now"] = cache, now
    if c["op"] == "attend":
        s["q"] = _normal(gen, b, h * c["group"], d).bfloat16()
        s["out"] = torch.empty(b, h * c["group"], d, device="cuda")
        s["lse"] = torch.empty(b, h * c["group"], device="cuda")
    elif c["op"] == "append":
        # the keys of a step are views of its projection; every fourth sequence's token is larger than its page
        grow = torch.where(torch.arange(b, device="cuda") % 4 == 3, 3.0, 1.0)[:, None, None]
        s["k_new"] = (_normal(gen, b, h, d) * grow).bfloat16()
        s["v_new"] = (_normal(gen, b, h, d) * grow).bfloat16()
        if c["mode"] == "kvzap":
            s["score"], s["tau"] = _normal(gen, b, h), torch.zeros(b, h, device="cuda")
        else:
            s["flag"] = torch.where(torch.rand(b, h, generator=gen, device="cuda") < 0.5, now, -1).int()
        s["count0"] = cache["count"].clone()
    else:
        n = t - c["first"]
        s["k_out"] = torch.empty(b, n, h, d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty(b, n, h, d, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms

def _plain_attend(s):
    c, cache = s["case"], s["cache"]
    b, h, g, d = c["batch"], c["kv_heads"], c["group"], c["dim"]
    table = cache["page_table"].clamp(min=0).long()
    n = table.shape[2] * PAGE
    k = (_values(cache["kq_pool"][table], c["fmt"]) * cache["scale_pool"][table][..., 0, None, None]).view(b, h, n, d)
    logits = torch.matmul(s["q"].float().view(b, h, g, d), k.transpose(2, 3)) * (1 / math.sqrt(d))
    del k
    live = (torch.arange(n, device="cuda") < cache["count"][..., None]) & \
        (cache["expire_pool"][table].view(b, h, n) > s["now"])
    logits = torch.where(live[:, :, None], logits, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    w = torch.exp(logits - top)
    total = w.sum(-1, keepdim=True)
    v = (_values(cache["vq_pool"][table], c["fmt"]) * cache["scale_pool"][table][..., 1, None, None]).view(b, h, n, d)
    s["out"].copy_((torch.matmul(w, v) / torch.where(total > 0, total, 1)).view(b, h * g, d))
    s["lse"].copy_((top + torch.log(total)).view(b, h * g))
    return s["out"], s["lse"]


def _shown(cache, fmt):
    """A cache's buffers, the codes as the numbers that they are (a row's values: its codes times its page's scale)."""
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    return dict(cache, kq_pool=cache["kq_pool"].view(kind), vq_pool=cache["vq_pool"].view(kind))


def _plain_write(s):
    c, cache = s["case"], s["cache"]
    b, t, h, d, fmt = c["batch"], c["tokens"], c["kv_heads"], c["dim"], c["fmt"]
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    if c["mode"] == "kvzap":
        expire = torch.where(s["scores"].permute(0, 2, 1) >= s["tau"][..., None], NEVER, pos + WINDOW)
    else:
        expire = torch.where(s["flag"] < 0, NEVER, torch.maximum(s["flag"], pos + WINDOW))
    expire = expire.int().reshape(b * h, t)
    keep = expire > s["now"]
    count = keep.sum(1)
    pages = (count + s["reserve"] + PAGE - 1) // PAGE
    first = torch.cumsum(pages, 0) - pages
    at = torch.nonzero(keep)                              # (head, position), in order
    slot = torch.cumsum(keep, 1)[at[:, 0], at[:, 1]] - 1
    row = first[at[:, 0]] * PAGE + slot
    width = cache["page_table"].shape[2]
    index = torch.arange(width, device="cuda")
    cache["page_table"].copy_(torch.where(index < pages[:, None], first[:, None] + index, -1).view(b, h, width))
    cache["remap"].fill_(-1).view(b * h, -1)[at[:, 0], slot] = at[:, 1].int()
    cache["count"].copy_(count.view(b, h))
    cache["expire_pool"].zero_().view(-1)[row] = expire[keep]
    cap = cache["kq_pool"].shape[0]
    _plain_rows(s["k"], at, row, cap, cache["kq_pool"], cache["scale_pool"][:, 0], b, t, h, d, fmt)
    _plain_rows(s["v"], at, row, cap, cache["vq_pool"], cache["scale_pool"][:, 1], b, t, h, d, fmt)
    return _shown(cache, fmt)


def _plain_rows(src, at, row, cap, pool, scale_out, b, t, h, d, fmt):
    x = src[at[:, 0] // h, at[:, 1], at[:, 0] % h].float()
    amax = torch.zeros(cap, device="cuda").scatter_reduce(0, row // PAGE, x.abs().amax(1), "amax")
    scale = _block_scale(amax, fmt)
    scale_out.copy_(scale)
    pool.zero_().view(cap * PAGE, d)[row] = _codes(x, scale[row // PAGE][:, None], fmt)


def _plain_append(s):
    c, cache = s["case"], s["cache"]
    b, h, d, fmt = c["batch"], c["kv_heads"], c["dim"], c["fmt"]
    cache["count"].copy_(s["count0"])                     # the step is taken again: the slot is given back first
    j = cache["count"].view(-1).long()
    page = cache["page_table"].view(b * h, -1).gather(1, (j // PAGE)[:, None])[:, 0].long()
    r = j % PAGE
    _plain_token(s["k_new"].view(b * h, d), page, r, cache["kq_pool"], cache["scale_pool"][:, 0], fmt)
    _plain_token(s["v_new"].view(b * h, d), page, r, cache["vq_pool"], cache["scale_pool"][:, 1], fmt)
    pos = s["now"] + 1
    if c["mode"] == "kvzap":
        expire = torch.where(s["score"] >= s["tau"], NEVER, pos + WINDOW).view(-1)
    else:
        expire = torch.where(s["flag"] < 0, NEVER, s["flag"].clamp(min=pos + WINDOW)).view(-1)
    cache["expire_pool"][page, r] = expire.int()
    cache["remap"].view(b * h, -1).scatter_(1, j[:, None], pos)
    cache["count"] += 1
    return _shown(cache, fmt)


def _plain_token(x, page, r, pool, scale, fmt):
    x = x.float()
    mine = _block_scale(x.abs().amax(1), fmt)
    old = torch.where(r == 0, 0, scale[page])
    new = torch.maximum(old, mine)
    rows = _values(pool[page], fmt) * (old / torch.where(new > 0, new, 1))[:, None, None]
    one = torch.ones_like(new)[:, None, None]
    before = (torch.arange(PAGE, device="cuda") < r[:, None]) & (new > old)[:, None]
    pool[page] = torch.where(before[..., None], _codes(rows, one, fmt), pool[page])
    pool[page, r] = _codes(x, new[:, None], fmt)
    scale[page] = new


def _plain_read(s):
    c, cache = s["case"], s["cache"]
    b, h, d = c["batch"], c["kv_heads"], c["dim"]
    slot = torch.arange(c["first"], c["tokens"], device="cuda")
    live = slot < cache["count"][..., None]               # [B, H, n]
    index = (slot // PAGE).clamp(max=cache["page_table"].shape[2] - 1)
    page = torch.where(live, cache["page_table"][:, :, index], 0).clamp(min=0).long()
    for pool, out, i in ((cache["kq_pool"], s["k_out"], 0), (cache["vq_pool"], s["v_out"], 1)):
        x = _values(pool[page, slot % PAGE], c["fmt"]) * cache["scale_pool"][page][..., i, None]
        out.copy_(torch.where(live[..., None], x, 0).permute(0, 2, 1, 3))
    return s["k_out"], s["v_out"]


def _plain_rotate(s):
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["inv_freq"]    # far positions: the angle in 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    for x, w, out in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
        rot, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        if c["interleaved"]:
            a, e = rot[..., 0::2], rot[..., 1::2]
            turned = torch.stack((a * cos - e * sin, e * cos + a * sin), -1).flatten(-2)
        else:
            a, e = rot.chunk(2, -1)
            turned = torch.cat((a * cos - e * sin, e * cos + a * sin), -1)
        out.copy_(torch.cat((turned, rest), -1))
    return s["q_out"], s["k_out"]


# ---------------------------------------------------------------------------- the framework's calls

def _own(s):
    import kv_cache_pruning_gb300 as kvp
    c = s["case"]
    if c["op"] == "rotate":
        if "turns" not in s:                              # a model's table, made once
            s["turns"] = kvp.kvp_rope_turns(s["inv_freq"])
        return kvp.kvp_qk_norm_rope(s["q"], s["k"], s["pos"], s["turns"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                    interleaved=c["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    if "handle" not in s:                                 # the cache's handle and the workspace that a program keeps
        s["handle"] = kvp.Block8PagedKV(**s["cache"], fmt=FORMATS[c["fmt"]])
        if c["op"] == "attend":
            s["ws"] = torch.zeros(kvp.kvp_decode_attn_block8_workspace_bytes(
                c["batch"], c["kv_heads"] * c["group"], c["kv_heads"], c["dim"]), dtype=torch.uint8, device="cuda")
        elif c["op"] == "write":
            s["ws"] = torch.empty(kvp.kvp_compact_block8_workspace_bytes(
                c["batch"], c["kv_heads"], c["tokens"], s["cache"]["kq_pool"].shape[0]), dtype=torch.uint8, device="cuda")
        s["shown"] = _shown(s["cache"], c["fmt"])
    cache = s["handle"]
    if c["op"] == "attend":
        kvp.kvp_decode_attn_block8(s["q"], cache, s["now"], out=s["out"], lse=s["lse"], workspace=s["ws"],
                                   status=s["status"])
        return s["out"], s["lse"]
    if c["op"] == "write":
        kvp.kvp_compact_block8(s["k"], s["v"], s["now"], s["reserve"], cache, mode=MODES[c["mode"]],
                               scores=s.get("scores"), tau=s.get("tau"), flag_step=s.get("flag"), window=WINDOW,
                               status=s["status"], workspace=s["ws"])
        return s["shown"]
    if c["op"] == "append":
        cache.count.copy_(s["count0"])                    # the step is taken again: the slot is given back first
        kvp.kvp_append_block8(cache, s["k_new"], s["v_new"], s["now"] + 1, mode=MODES[c["mode"]], score=s.get("score"),
                              tau=s.get("tau"), flag_step=s.get("flag"), window=WINDOW, status=s["status"])
        return s["shown"]
    return kvp.kvp_read_block8(cache, c["first"], c["tokens"] - c["first"], k_out=s["k_out"], v_out=s["v_out"],
                               status=s["status"])


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "write": _plain_write, "append": _plain_append, "read": _plain_read,
            "rotate": _plain_rotate}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    d = c["dim"]
    if c["op"] == "rotate":
        values = c["tokens"] * (c["q_heads"] + c["kv_heads"]) * d
        return {"bytes": 4 * values + 4 * c["tokens"], "flops": 8 * values}
    heads = c["batch"] * c["kv_heads"]
    if c["op"] == "attend":
        kept = heads * c["tokens"] * (c["keep"] or 2 / 7)
        return {"bytes": kept * (2 * d + 4 + 12 / PAGE) + heads * c["group"] * 6 * d,
                "flops": 4 * d * kept * c["group"]}
    if c["op"] == "write":
        kept = heads * min(c["tokens"], c["tokens"] * c["keep"] + min(WINDOW, c["tokens"]) * (1 - c["keep"]))
        return {"bytes": 4 * heads * c["tokens"] + kept * (6 * d + 8 + 12 / PAGE), "flops": 4 * d * kept}
    if c["op"] == "append":
        return {"bytes": heads * (6 * d + 44), "flops": 4 * d * heads}
    slots = heads * (c["tokens"] - c["first"])
    return {"bytes": slots * (6 * d + 12 / PAGE), "flops": 2 * d * slots}


# ---------------------------------------------------------------------------- in 64 bits

def _power64(e):
    """2^e, exactly: from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _numbers64(codes, fmt):
    """The numbers that bytes stand for, from the formats' definitions."""
    byte = torch.arange(256, device="cuda")
    if fmt == "int8":
        table = torch.where(byte < 128, byte, byte - 256).double()
    else:
        field, frac = (byte >> 3) & 15, (byte & 7).double()
        size = torch.where(field > 0, (1 + frac / 8) * _power64(field - 7), frac / 8 * 2.0 ** -6)
        table = torch.where(byte >= 128, -size, size)
    return table[codes.long()]


def _round64(y, fmt):
    """Each value of y (in the format's range) to the nearest number of the format, ties to an even last digit."""
    if fmt == "int8":
        return torch.round(y)
    size = y.abs()
    step = _power64(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(size / step) * step, y)


def _scale64(amax, fmt):
    """The smallest power of two that is at least amax over the format's largest number."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / (448.0 if fmt == "e4m3" else 127.0)) - 1e-12)
    return torch.where(amax > 0, _power64(e.clamp(min=-126)), 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rotate":
        got = []
        for name in ("q", "k"):
            x, w = s[name], s[name + "w"]
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for a in range(0, x.shape[0], 8192):
                y = x[a:a + 8192].double()
                if w is not None:
                    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["dim"] + 1e-6) * w.double()
                turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                   s["pos"][a:a + 8192].double()[:, None] * s["inv_freq"])[:, None]
                half = c["rot"] // 2
                first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else \
                    (slice(0, half), slice(half, c["rot"]))
                z = torch.complex(y[..., first], y[..., second]) * turn
                y[..., first], y[..., second] = z.real, z.imag
                out[a:a + 8192] = y
            got.append(out)
        return tuple(got)
    b, h, d, fmt, cache = c["batch"], c["kv_heads"], c["dim"], c["fmt"], s["cache"]
    if c["op"] == "attend":
        out = torch.zeros(b, h * c["group"], d, dtype=torch.float64, device="cuda")
        lse = torch.full((b, h * c["group"]), -math.inf, dtype=torch.float64, device="cuda")
        counts = cache["count"].tolist()
        for i in range(b):
            for j in range(h):
                n = counts[i][j]
                page = cache["page_table"][i, j, :(n + PAGE - 1) // PAGE].long()
                there = (cache["expire_pool"][page].view(-1)[:n] > s["now"]).nonzero()[:, 0]
                if not len(there):
                    continue
                sc = cache["scale_pool"].double()[page].repeat_interleave(PAGE, 0)[there]
                k = _numbers64(cache["kq_pool"][page].view(-1, d)[there], fmt) * sc[:, :1]
                v = _numbers64(cache["vq_pool"][page].view(-1, d)[there], fmt) * sc[:, 1:]
                heads = slice(j * c["group"], (j + 1) * c["group"])
                x = s["q"][i, heads].double() @ k.T / math.sqrt(d)
                lse[i, heads] = torch.logsumexp(x, 1)
                out[i, heads] = torch.softmax(x, 1) @ v
        return out, lse
    if c["op"] == "read":
        n = c["tokens"] - c["first"]
        outs = torch.zeros(2, b, n, h, d, dtype=torch.float64, device="cuda")
        counts = cache["count"].tolist()
        for i in range(b):
            for j in range(h):
                slots = torch.arange(c["first"], max(c["first"], counts[i][j]), device="cuda")
                page = cache["page_table"][i, j, slots // PAGE].long()
                for w, pool in ((0, "kq_pool"), (1, "vq_pool")):
                    x = _numbers64(cache[pool][page, slots % PAGE], fmt) * cache["scale_pool"][page, w].double()[:, None]
                    outs[w, i, :len(slots), j] = x
        return outs[0], outs[1]
    blank = dict.fromkeys(cache)                          # whole numbers have no value in 64 bits of their own
    scale = torch.zeros(cache["scale_pool"].shape, dtype=torch.float64, device="cuda")
    pools = [_numbers64(cache[n], fmt).float() if c["op"] == "append" else torch.zeros(cache[n].shape, device="cuda")
             for n in ("kq_pool", "vq_pool")]             # numbers of 8 bits: 32 bits hold them
    if c["op"] == "append":
        scale.copy_(cache["scale_pool"])
        counts, table = s["count0"].tolist(), cache["page_table"].tolist()
        for i in range(b):
            for j in range(h):
                r, p = counts[i][j] % PAGE, table[i][j][counts[i][j] // PAGE]
                for w, x in ((0, s["k_new"]), (1, s["v_new"])):
                    x = x[i, j].double()
                    old = scale[p, w].clone() if r else scale.new_zeros(())
                    new = torch.maximum(old, _scale64(x.abs().max(), fmt))
                    if r:
                        pools[w][p, :r] = _round64(pools[w][p, :r].double() * (old / new), fmt).float()
                    pools[w][p, r] = _round64(x / new, fmt).float()
                    scale[p, w] = new
    else:
        page = 0
        for i in range(b):
            for j in range(h):
                pos = torch.arange(c["tokens"], device="cuda")
                if c["mode"] == "kvzap":
                    there = (s["scores"][i, :, j] >= s["tau"][i, j]) | (pos + WINDOW > s["now"])
                else:
                    f = s["flag"][i, j]
                    there = (f < 0) | (f > s["now"]) | (pos + WINDOW > s["now"])
                at = there.nonzero()[:, 0]
                n = (len(at) + PAGE - 1) // PAGE
                for w, x in ((0, s["k"]), (1, s["v"])):
                    rows = torch.zeros(n * PAGE, d, dtype=torch.float64, device="cuda")
                    rows[:len(at)] = x[i, at, j].double()
                    rows = rows.view(n, PAGE, d)
                    sc = _scale64(rows.abs().amax((1, 2)), fmt)
                    scale[page:page + n, w] = sc
                    pools[w][page:page + n] = _round64(rows / torch.where(sc > 0, sc, 1.0)[:, None, None], fmt).float()
                page += (len(at) + s["reserve"] + PAGE - 1) // PAGE
    return dict(blank, kq_pool=pools[0] if fmt == "e4m3" else None, vq_pool=pools[1] if fmt == "e4m3" else None,
                scale_pool=scale)
