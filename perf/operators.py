"""The paged 8-bit latent cache and the calls around it, as a decode loop makes them.

Four operators, each in a plain form of elementary torch operations (`own` false) and
as the library's calls (`own` true):

  pages    block tables and slot maps from the requests' lengths: pages are taken from
           and returned to a free stack on the device
  write    bf16 latent rows (512 + 64 values) quantised to e4m3 into their pages, one
           power-of-two scale for each page of 64 tokens
  attn     tree-verify MLA attention over that cache (one node = a single-token step)
  compact  the accepted rows of the tree block gathered behind the prefix, in place

listed() names the cases that are measured, draw() gives more of the same ranges,
prepare() makes a case's inputs on the GPU from a seed, run() makes one pass, exact()
gives the result in 64 bits from the definition, and work() what a pass has to move and
compute.
"""
import math

import torch

own = False

PAGE = 64            # tokens per page, and so per scale
HEADS, LATENT, ROPE = 64, 512, 64
E4M3_MAX = 448.0
MIN_EXP = -40        # smallest exponent of a page's scale
SCALE = 1.0 / math.sqrt(192.0)
#: the largest listed cases bound what draw() gives
MOST_SCORES = 64 * 65 * (8192 + 65)
MOST_ROWS = 1024 * 128


def listed():
    return [
        # every request's tree block of one decode step, then back to the accepted rows
        {"name": "pages 64 x 33", "op": "pages", "B": 64, "rows_lo": 33, "rows_hi": 33,
         "prefix_lo": 1, "prefix_hi": 8192, "admit": False},
        # a batch of prompts admitted at once, then retired
        {"name": "pages 1000 prompts", "op": "pages", "B": 1000, "rows_lo": 1, "rows_hi": 2048,
         "prefix_lo": 0, "prefix_hi": 0, "admit": True},
        # the tree block of one decode step
        {"name": "write 64 x 33", "op": "write", "B": 64, "rows_lo": 33, "rows_hi": 33,
         "prefix_lo": 256, "prefix_hi": 4096, "ragged": False},
        # prompts of odd lengths, from an empty cache (prefill)
        {"name": "write 24 prompts", "op": "write", "B": 24, "rows_lo": 1, "rows_hi": 4001,
         "prefix_lo": 0, "prefix_hi": 0, "ragged": True},
        # the accepted path of one decode step
        {"name": "compact 64 x 33", "op": "compact", "B": 64, "q_len": 33, "accept": 8,
         "prefix_lo": 256, "prefix_hi": 4096},
        # wide trees on many requests, half of each tree accepted
        {"name": "compact 1024 x 128", "op": "compact", "B": 1024, "q_len": 128, "accept": 64,
         "prefix_lo": 1, "prefix_hi": 500},
        # one small request: latency
        {"name": "attn 1 x 9 x 256", "op": "attn", "B": 1, "q_len": 9, "prefix_lo": 256,
         "prefix_hi": 256, "spread": False, "lse": False},
        # a plain decode step: one token per request, ragged caches
        {"name": "attn 64 x 1 x <=4096", "op": "attn", "B": 64, "q_len": 1, "prefix_lo": 1,
         "prefix_hi": 4096, "spread": False, "lse": True},
        {"name": "attn 8 x 33 x 1024", "op": "attn", "B": 8, "q_len": 33, "prefix_lo": 1024,
         "prefix_hi": 1024, "spread": False, "lse": False},
        # the flagship tree-verify step
        {"name": "attn 64 x 33 x 4096", "op": "attn", "B": 64, "q_len": 33, "prefix_lo": 4096,
         "prefix_hi": 4096, "spread": False, "lse": False},
        # ragged caches, rows of differing magnitude, log-sum-exp wanted
        {"name": "attn 64 x 65 x <=8192", "op": "attn", "B": 64, "q_len": 65, "prefix_lo": 256,
         "prefix_hi": 8192, "spread": True, "lse": True},
        # one long context
        {"name": "attn 1 x 33 x 32768", "op": "attn", "B": 1, "q_len": 33, "prefix_lo": 32768,
         "prefix_hi": 32768, "spread": False, "lse": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["pages", "write", "compact", "attn", "attn", "attn"])
    if op == "pages":
        if rng.random() < 0.5:
            hi = _log_int(rng, 16, 2048)
            return {"op": op, "B": _log_int(rng, 1, 1000), "rows_lo": 1, "rows_hi": hi,
                    "prefix_lo": 0, "prefix_hi": 0, "admit": True}
        q = _log_int(rng, 1, 128)
        return {"op": op, "B": _log_int(rng, 1, 1000), "rows_lo": q, "rows_hi": q,
                "prefix_lo": 1, "prefix_hi": _log_int(rng, 64, 8192), "admit": False}
    if op == "write":
        if rng.random() < 0.5:
            hi = _log_int(rng, 8, 4001)
            return {"op": op, "B": _log_int(rng, 1, 24), "rows_lo": 1, "rows_hi": hi,
                    "prefix_lo": 0, "prefix_hi": rng.choice([0, 100, 1000]), "ragged": True}
        q = _log_int(rng, 1, 128)
        return {"op": op, "B": _log_int(rng, 1, 256), "rows_lo": q, "rows_hi": q,
                "prefix_lo": 0, "prefix_hi": _log_int(rng, 64, 4096), "ragged": False}
    if op == "compact":
        q = _log_int(rng, 2, 128)
        return {"op": op, "B": min(_log_int(rng, 1, 1024), MOST_ROWS // q), "q_len": q,
                "accept": _log_int(rng, 1, q // 2), "prefix_lo": 0,
                "prefix_hi": _log_int(rng, 8, 500)}
    q = _log_int(rng, 1, 128)
    B = _log_int(rng, 1, 64)
    most = min(32768, MOST_SCORES // (B * q) - q, 64 * 8257 // B - q)
    hi = _log_int(rng, 1, most)
    return {"op": op, "B": B, "q_len": q, "prefix_lo": rng.choice([0, hi // 3, hi]),
            "prefix_hi": hi, "spread": rng.random() < 0.5, "lse": rng.random() < 0.5}


# ----------------------------------------------------------------------------- inputs

def _lens(case, g, lo, hi):
    """A request's length each, evenly spread over [lo, hi] and in the seed's order."""
    B = case["B"]
    spread = torch.tensor([hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)])
    return spread[torch.randperm(B, generator=g)]


def _most_pages(case, extra=0):
    """Pages that these lengths can need, whatever their order."""
    B, rows = case["B"], case.get("rows_hi", case.get("q_len"))
    per = [hi if B == 1 else lo + (hi - lo) * i // (B - 1) for i in range(B)
           for lo, hi in ((case["prefix_lo"], case["prefix_hi"]), (case.get("rows_lo", rows), rows))]
    return sum(n // PAGE + 1 for n in per) + extra


def _tables(held, g, pages, width):
    """Block tables whose pages are scattered over the pool, as after long use, and the
    pages that are free."""
    used = int(held.sum())
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((held.numel(), width), -1, dtype=torch.int32)
    col = torch.arange(width)[None, :]
    table[col < held[:, None]] = perm[:used]
    return table, perm[used:]


def _scale_exp(amax):
    """Smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9), at least MIN_EXP."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e.clamp(min=MIN_EXP), torch.full_like(e, MIN_EXP))


def _pow2(e):
    """2^e exactly, for whole exponents of normal floats."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _new_cache(pages, g, spread=False):
    """A cache in use: every row of every page holds what some sequence left there."""
    x = torch.randn((pages, PAGE, LATENT + ROPE), generator=g, device="cuda")
    if spread:
        x *= torch.rand((pages, PAGE, 1), generator=g, device="cuda") * 1.5 + 0.5
    scales = _pow2(_scale_exp(x.abs().amax((1, 2))))
    x = (x / scales[:, None, None]).to(torch.float8_e4m3fn)
    return x[..., :LATENT].contiguous(), x[..., LATENT:].contiguous(), scales


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _tree_masks(B, q, g):
    """Ancestor-or-self words of random trees, int64 [B, q, ceil(q/64)]."""
    vis = torch.zeros((B, q, q), dtype=torch.bool)
    vis[:, 0, 0] = True
    rows = torch.arange(B)
    for i in range(1, q):
        lo = max(0, i - 12)
        parent = torch.randint(lo, i, (B,), generator=g)
        vis[:, i] = vis[rows, parent]
        vis[:, i, i] = True
    words = torch.zeros((B, q, (q + 63) // 64), dtype=torch.int64)
    for a in range(q):
        words[:, :, a // 64] |= vis[:, :, a].long() << (a % 64)
    return words


def prepare(case, seed):
    h = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B = case["op"], case["B"]
    s = {"case": case, "op": op, "B": B}
    pages = _most_pages(case, 7)
    width = (case["prefix_hi"] + case.get("rows_hi", case.get("q_len")) + PAGE - 1) // PAGE
    if op == "pages":
        prefix = _lens(case, h, case["prefix_lo"], case["prefix_hi"])
        rows = _lens(case, h, case["rows_lo"], case["rows_hi"])
        if case["admit"]:
            after = torch.zeros(B, dtype=torch.int64)          # retired again
        else:
            after = prefix + 1 + (torch.rand(B, generator=h) * rows).long().clamp(max=case["rows_lo"] - 1)
        held = (after + PAGE - 1) // PAGE
        need = (prefix + rows + PAGE - 1) // PAGE
        table, free = _tables(held, h, pages, width)
        if case["admit"] and B > 8:
            # a tenth fewer pages than the prompts want: the last requests are refused
            free = free[:int(need.sum()) * 9 // 10]
        start = torch.zeros(B + 1, dtype=torch.int64)
        start[1:] = rows.cumsum(0)
        s["n_rows"], s["q_len"] = int(start[-1]), case["rows_lo"]
        s["ragged"] = case["rows_lo"] != case["rows_hi"]
        pool = torch.full((pages,), -1, dtype=torch.int32)
        pool[:free.numel()] = free
        for k, v in (("prefix", prefix), ("after", after), ("n_blocks", held), ("start", start),
                     ("n_free", torch.tensor([free.numel()]))):
            s[k] = v.to(torch.int32).cuda()
        s["table"], s["pool"] = table.cuda(), pool.cuda()
    elif op == "write":
        prefix = _lens(case, h, case["prefix_lo"], case["prefix_hi"])
        rows = _lens(case, h, case["rows_lo"], case["rows_hi"])
        held = (prefix + rows + PAGE - 1) // PAGE
        table, _ = _tables(held, h, pages, width)
        start = torch.zeros(B + 1, dtype=torch.int64)
        start[1:] = rows.cumsum(0)
        n = int(start[-1])
        s["ckv8"], s["kr8"], s["scales"] = _new_cache(pages, g)
        # rows a little larger than what the cache holds, so that some pages' scales rise
        s["rows"], s["rope_rows"] = _bf16(g, n, LATENT) * 1.25, _bf16(g, n, ROPE) * 2.0
        s["table"], s["prefix"] = table.cuda(), prefix.to(torch.int32).cuda()
        s["start"], s["max_rows"] = start.to(torch.int32).cuda(), int(rows.max())
        s["ragged"], s["q_len"] = case["ragged"], case["rows_lo"]
    elif op == "compact":
        q, alen = case["q_len"], case["accept"]
        prefix = _lens(case, h, case["prefix_lo"], case["prefix_hi"])
        held = (prefix + q + PAGE - 1) // PAGE
        table, _ = _tables(held, h, pages, width)
        s["ckv8"], s["kr8"], s["scales"] = _new_cache(pages, g, spread=True)
        # the root, then nodes in creation order, all behind the accepted length
        pick = torch.rand((B, q - alen), generator=h).argsort(1)[:, :alen - 1].sort(1).values + alen
        path = torch.full((B, q), -1, dtype=torch.int32)
        path[:, 0] = 0
        path[:, 1:alen] = pick.to(torch.int32)
        accept = torch.randint(max(1, alen - 4), alen + 1, (B,), generator=h)
        s["table"], s["prefix"], s["path"] = table.cuda(), prefix.to(torch.int32).cuda(), path.cuda()
        s["accept"] = accept.to(torch.int32).cuda()
    else:
        q = case["q_len"]
        prefix = _lens(case, h, case["prefix_lo"], case["prefix_hi"])
        held = (prefix + q + PAGE - 1) // PAGE
        table, _ = _tables(held, h, pages, width)
        s["ckv8"], s["kr8"], s["scales"] = _new_cache(pages, g, case["spread"])
        s["q_lat"], s["q_rope"] = _bf16(g, B, q, HEADS, LATENT), _bf16(g, B, q, HEADS, ROPE)
        s["table"], s["prefix"] = table.cuda(), prefix.to(torch.int32).cuda()
        s["mask"], s["max_prefix"] = _tree_masks(B, q, h).cuda(), case["prefix_hi"]
    return s


# --------------------------------------------------------------------------- the passes

def _plain_plan(s, prefix, rows, table, n_blocks, pool, n_free):
    """One plan: pages given back first, then taken in the order of the requests; a
    request that the free pages do not reach leaves its state as it was."""
    B, width = table.shape
    need = (prefix + rows + PAGE - 1) // PAGE
    back, want = (n_blocks - need).clamp(min=0), (need - n_blocks).clamp(min=0)
    free = n_free + back.sum()
    # the pages given back lie on the stack so that taking as many again returns them
    col = torch.arange(width, device="cuda")[None, :]
    gone = (col >= need[:, None]) & (col < n_blocks[:, None])
    order = back.cumsum(0)[:, None] - back[:, None] + (col - need[:, None])
    pool[(free - 1 - order)[gone]] = table[gone]
    table[gone] = -1
    upto = want.cumsum(0)
    served = (want == 0) | (upto <= free)
    took = (col >= n_blocks[:, None]) & (col < need[:, None]) & served[:, None]
    order = (upto - want)[:, None] + (col - n_blocks[:, None])
    table[took] = pool[(free - 1 - order)[took]]
    n_blocks.copy_(torch.where(served, need, n_blocks))
    n_free.copy_(free - torch.where(served, want, 0).sum())
    return served


def _plain_pages(s):
    start = s["start"].long()
    rows = start[1:] - start[:-1]
    req = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), rows, output_size=s["n_rows"])
    state = [s[k] for k in ("table", "n_blocks", "pool", "n_free")]
    served = _plain_plan(s, s["prefix"], rows.int(), *state)
    pos = s["prefix"].long()[req] + torch.arange(s["n_rows"], device="cuda") - start[req]
    slots = s["table"].long()[req, (pos // PAGE).clamp(max=s["table"].shape[1] - 1)] * PAGE + pos % PAGE
    slots = torch.where(served[req], slots, -1)
    _plain_plan(s, s["after"], torch.zeros_like(s["after"]), *state)
    return slots, served


def _plain_write(s):
    start = s["start"].long()
    n = s["rows"].shape[0]
    req = torch.repeat_interleave(torch.arange(s["B"], device="cuda"), start[1:] - start[:-1], output_size=n)
    pos = s["prefix"].long()[req] + torch.arange(n, device="cuda") - start[req]
    page, off = s["table"].long()[req, pos // PAGE], pos % PAGE
    x = torch.cat((s["rows"], s["rope_rows"]), 1).float()
    pages = s["scales"].numel()
    amax = torch.zeros(pages, device="cuda").scatter_reduce_(0, page, x.abs().amax(1), "amax")
    first = torch.full((pages,), PAGE, device="cuda").scatter_reduce_(0, page, off, "amin")
    fresh = _pow2(_scale_exp(amax))
    old = s["scales"].clone()
    new = torch.where(first == PAGE, old, torch.where(first == 0, fresh, torch.maximum(old, fresh)))
    # the live rows of the requests' first pages, where a scale rose
    head = s["table"].long().gather(1, s["prefix"].long()[:, None] // PAGE)[:, 0]
    live = torch.arange(PAGE, device="cuda")[None, :] < (s["prefix"] % PAGE)[:, None]
    for t, cols in ((s["ckv8"], slice(0, LATENT)), (s["kr8"], slice(LATENT, None))):
        rows, bytes_ = t.view(torch.uint8)[head], t.view(torch.uint8)
        again = (rows.view(t.dtype).float() * (old / new)[head][:, None, None]).to(t.dtype).view(torch.uint8)
        bytes_[head] = torch.where(live[..., None], again, rows)
        bytes_[page, off] = (x[:, cols] / new[page][:, None]).to(t.dtype).view(torch.uint8)
    s["scales"].copy_(new)
    return s["ckv8"], s["kr8"], s["scales"]


def _plain_compact(s):
    B, q = s["path"].shape
    prefix, accept = s["prefix"].long(), s["accept"].long()
    i = torch.arange(q, device="cuda")[None, :].expand(B, q)
    on = i < accept[:, None]
    b = torch.arange(B, device="cuda")[:, None].expand(B, q)[on]
    to, frm = (prefix[:, None] + i)[on], (prefix[:, None] + s["path"].long())[on]
    table = s["table"].long()
    tp, to = table[b, to // PAGE], to % PAGE
    fp, frm = table[b, frm // PAGE], frm % PAGE
    old = s["scales"].clone()
    new = old.clone().scatter_reduce_(0, tp, old[fp], "amax")
    # the pages that rows move into; a request's last one stands for those it lacks
    block = prefix[:, None] // PAGE + torch.arange(3, device="cuda")
    home = table.gather(1, torch.minimum(block, (prefix + accept - 1)[:, None] // PAGE)).flatten()
    for t in (s["ckv8"], s["kr8"]):
        bytes_ = t.view(torch.uint8)
        moved = (bytes_[fp, frm].view(t.dtype).float() * (old[fp] / new[tp])[:, None]).to(t.dtype)
        bytes_[home] = (bytes_[home].view(t.dtype).float() * (old / new)[home][:, None, None]).to(t.dtype).view(torch.uint8)
        bytes_[tp, to] = moved.view(torch.uint8)
    s["scales"].copy_(new)
    return s["ckv8"], s["kr8"], s["scales"], (prefix + accept).int()


def _plain_attn(s):
    B, q = s["B"], s["q_lat"].shape[1]
    T = s["max_prefix"] + q
    table = s["table"].long().clamp(min=0)
    scales = s["scales"][table][:, :, None, None]
    c = s["ckv8"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scales
    k = s["kr8"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scales
    c, k = c.flatten(1, 2)[:, :T], k.flatten(1, 2)[:, :T]
    scores = torch.bmm(s["q_lat"].float().flatten(1, 2), c.transpose(1, 2))
    scores += torch.bmm(s["q_rope"].float().flatten(1, 2), k.transpose(1, 2))
    scores *= SCALE
    node = torch.arange(T, device="cuda")[None, :] - s["prefix"].long()[:, None]     # [B, T]
    at = node.clamp(0, q - 1)
    words = torch.gather(s["mask"], 2, (at // 64)[:, None, :].expand(B, q, T))
    seen = (((words >> (at % 64)[:, None, :]) & 1) == 1) & (node < q)[:, None, :]
    seen |= (node < 0)[:, None, :]
    scores.view(B, q, HEADS, T).masked_fill_(~seen[:, :, None, :], -math.inf)
    top = scores.amax(2, keepdim=True)
    weights = scores.sub_(top).exp_()
    total = weights.sum(2, keepdim=True)
    out = (torch.bmm(weights, c) / total).view(B, q, HEADS, LATENT).to(torch.bfloat16)
    lse = (top + total.log()).view(B, q, HEADS)
    return (out, lse) if s["case"]["lse"] else out


def run(s):
    op = s["op"]
    if own:
        from tree_speculative_decoding_05_b200 import ddt
    if op == "pages":
        if own:
            rows = {"row_start": s["start"], "n_rows": s["n_rows"]} if s["ragged"] else {"q_len": s["q_len"]}
            slots, status = ddt.kv_pages(s["prefix"], s["table"], s["n_blocks"], s["pool"], s["n_free"], **rows)
            ddt.kv_pages(s["after"], s["table"], s["n_blocks"], s["pool"], s["n_free"], q_len=0)
            served = status == ddt.REQ_OK
        else:
            slots, served = _plain_pages(s)
        return {"slots": slots, "served": served, "table": s["table"], "n_blocks": s["n_blocks"], "n_free": s["n_free"]}
    if op == "write":
        if own:
            if s["ragged"]:
                ddt.kv_write_q8(s["ckv8"], s["kr8"], s["scales"], s["table"], s["prefix"], s["rows"], s["rope_rows"],
                                row_start=s["start"], max_rows=s["max_rows"])
            else:
                ddt.kv_write_q8(s["ckv8"], s["kr8"], s["scales"], s["table"], s["prefix"],
                                s["rows"].view(s["B"], s["q_len"], LATENT), s["rope_rows"].view(s["B"], s["q_len"], ROPE))
            got = s["ckv8"], s["kr8"], s["scales"]
        else:
            got = _plain_write(s)
        return dict(zip(("c_kv", "k_rope", "scales"), got))
    if op == "compact":
        if own:
            prefix, _ = ddt.kv_compact_q8(s["ckv8"], s["kr8"], s["scales"], s["table"], s["prefix"], s["path"], s["accept"])
            got = s["ckv8"], s["kr8"], s["scales"], prefix
        else:
            got = _plain_compact(s)
        return dict(zip(("c_kv", "k_rope", "scales", "prefix"), got))
    if own:
        out, lse = ddt.verify_attn_q8(s["q_lat"], s["q_rope"], s["ckv8"], s["kr8"], s["scales"], s["table"], s["prefix"],
                                      s["mask"], SCALE, max_prefix=s["max_prefix"], want_lse=s["case"]["lse"])
        got = (out, lse) if s["case"]["lse"] else out
    else:
        got = _plain_attn(s)
    return {"out": got[0], "lse": got[1]} if s["case"]["lse"] else {"out": got}


# ----------------------------------------------------------------------- the definition

def _round_e4m3(x):
    """Round to nearest even in e4m3 (three mantissa bits, exponents from -6)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6.0) - 3.0)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _fit(amax):
    """The smallest power of two, at least 2^MIN_EXP, under which amax fits into e4m3."""
    e = MIN_EXP
    if amax > 0:
        e = max(e, math.ceil(math.log2(amax / E4M3_MAX)) - 1)
        while E4M3_MAX * 2.0 ** e < amax:
            e += 1
    return 2.0 ** e


def _exact_write(s):
    cache = torch.cat((s["ckv8"].double(), s["kr8"].double()), 2)
    rows = torch.cat((s["rows"].double(), s["rope_rows"].double()), 1)
    scales = s["scales"].double().tolist()
    start, prefix, table = s["start"].tolist(), s["prefix"].tolist(), s["table"].tolist()
    tops = rows.abs().amax(1).tolist()
    for b in range(s["B"]):
        at = start[b]
        while at < start[b + 1]:
            pos = prefix[b] + at - start[b]
            page, off = table[b][pos // PAGE], pos % PAGE
            n = min(PAGE - off, start[b + 1] - at)
            scale = _fit(max(tops[at:at + n]))
            if off and scales[page] >= scale:
                scale = scales[page]
            elif off:
                cache[page, :off] = _round_e4m3(cache[page, :off] * (scales[page] / scale))
            cache[page, off:off + n] = _round_e4m3(rows[at:at + n] / scale)
            scales[page] = scale
            at += n
    return {"c_kv": cache[..., :LATENT], "k_rope": cache[..., LATENT:],
            "scales": torch.tensor(scales, dtype=torch.float64)}


def _exact_compact(s):
    cache = torch.cat((s["ckv8"].double(), s["kr8"].double()), 2)
    scales = s["scales"].tolist()
    prefix, table, path, accept = (s[k].tolist() for k in ("prefix", "table", "path", "accept"))
    for b in range(s["B"]):
        frm = [divmod(prefix[b] + j, PAGE) for j in path[b][:accept[b]]]
        held = {}
        for i, (p, o) in enumerate(frm):
            held.setdefault((prefix[b] + i) // PAGE, []).append((i, table[b][p], o))
        values = torch.stack([cache[table[b][p], o] * scales[table[b][p]] for p, o in frm])
        before = {block: scales[table[b][block]] for block in held}
        risen = {block: max([before[block]] + [scales[p] for _, p, _ in got]) for block, got in held.items()}
        for block, got in held.items():
            page = table[b][block]
            if risen[block] > before[block]:
                cache[page] = _round_e4m3(cache[page] * (before[block] / risen[block]))
                scales[page] = risen[block]
            i = [x[0] for x in got]
            o = [(prefix[b] + x) % PAGE for x in i]
            cache[page, o] = _round_e4m3(values[i] / risen[block])
    return {"c_kv": cache[..., :LATENT], "k_rope": cache[..., LATENT:],
            "scales": torch.tensor(scales, dtype=torch.float64), "prefix": None}


def _exact_attn(s):
    B, q = s["B"], s["q_lat"].shape[1]
    outs, lses = [], []
    bits = ((s["mask"][..., None] >> torch.arange(64, device="cuda")) & 1).flatten(2)[:, :, :q].bool()
    for b, P in enumerate(s["prefix"].tolist()):
        T = P + q
        pages = s["table"][b, :(T + PAGE - 1) // PAGE].long().tolist()
        scale = s["scales"][pages].double()[:, None, None]
        c = (s["ckv8"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * scale).flatten(0, 1)[:T]
        k = (s["kr8"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * scale).flatten(0, 1)[:T]
        key = torch.cat((c, k), 1)
        query = torch.cat((s["q_lat"][b], s["q_rope"][b]), 2).double().flatten(0, 1)
        x = (query @ key.T * SCALE).view(q, HEADS, T)
        seen = torch.ones((q, T), dtype=torch.bool, device="cuda")
        seen[:, P:] = bits[b]
        x = torch.where(seen[:, None, :], x, -math.inf)
        lse = torch.logsumexp(x, 2)
        outs.append((torch.exp(x - lse[..., None]).flatten(0, 1) @ c).view(q, HEADS, LATENT))
        lses.append(lse)
    got = {"out": torch.stack(outs)}
    if s["case"]["lse"]:
        got["lse"] = torch.stack(lses)
    return got


def exact(case, seed):
    if case["op"] == "pages":
        return None                      # whole numbers only
    return {"write": _exact_write, "compact": _exact_compact, "attn": _exact_attn}[case["op"]](prepare(case, seed))


# ---------------------------------------------------------------------------- its work

def work(case):
    op, B = case["op"], case["B"]
    if op == "pages":
        rows = B * (case["rows_lo"] + case["rows_hi"]) / 2
        pages = rows / PAGE + B
        # lengths, counts and statuses twice; a slot per row; table and stack entries of the pages that move
        return {"bytes": 8 * rows + 4 * 8 * B + 4 * 4 * pages, "flops": 0}
    if op == "write":
        rows = B * (case["rows_lo"] + case["rows_hi"]) / 2
        return {"bytes": rows * (LATENT + ROPE) * 3 + 12 * B, "flops": 3 * rows * (LATENT + ROPE)}
    if op == "compact":
        rows = B * max(1, case["accept"] - 2)
        return {"bytes": rows * (LATENT + ROPE) * 2 + 4 * B * case["q_len"] + 16 * B, "flops": 0}
    q, keys = case["q_len"], (case["prefix_lo"] + case["prefix_hi"]) / 2
    rows, cached = B * q * HEADS, B * (keys + q)
    return {"bytes": rows * 2 * (LATENT + ROPE + LATENT) + cached * (LATENT + ROPE),
            "flops": 2.0 * rows * (keys + min(q, 8)) * (LATENT + ROPE + LATENT)}
