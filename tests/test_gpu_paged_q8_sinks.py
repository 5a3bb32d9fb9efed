"""Attention over the paged 8-bit cache where one key outweighs thousands of others that
together matter: an attention sink.  Its latent values are small, as a sink's are, so the
result hangs on weights of 2^-5 to 2^-24 of the largest (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from test_gpu_paged_q8 import random_parents, tree_mask
from tree_speculative_decoding_05_b200 import ddt

pytestmark = pytest.mark.gpu
PAGE, HEADS = 64, 64
SCALE = float(np.float32(1 / np.sqrt(192.0)))
STEP = 2.0 ** -6     # every page's scale
SINK = 256.0         # e4m3 value of a sink's first rope column


def sink_case(T, sinks, seed, top_share):
    """One request of one node over T rows with the given sinks.  Heads 0-31 score all other
    rows alike, heads 32-63 spread them by one nat; the heads' shares of the sinks run from
    0.3 to top_share.  Latent values have mean 1 (a sink's are a hundredth)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-T // PAGE)
    lat = 1 + 0.5 * torch.randn((pages * PAGE, 512), generator=g, device="cuda")
    rope = torch.randn((pages * PAGE, 64), generator=g, device="cuda")
    rope[:, 0] = 0
    lat[sinks] *= 0.01
    rope[sinks] = 0
    e4 = lambda x: (x / STEP).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    lat, rope = e4(lat), e4(rope)
    rope[sinks, 0] = SINK
    logit = torch.linspace(math.log(0.3 / 0.7), math.log(top_share / (1 - top_share)), 32).repeat(2)
    spread = torch.tensor([0.0] * 32 + [1.0] * 32)
    gap = logit + math.log(T / len(sinks)) + spread ** 2 / 2        # of a sink over the rest, in nats
    q = torch.zeros(HEADS, 576)
    q[:, 512] = gap / (SCALE * STEP * SINK)
    q[:, 513:545] = spread[:, None] / (SCALE * math.sqrt(32))
    q = q.to(torch.bfloat16).cuda()
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    at = table.long().cuda()
    ckv, kr = (torch.empty((pages, PAGE, n), dtype=torch.uint8, device="cuda") for n in (512, 64))
    ckv[at], kr[at] = lat.view(torch.uint8).view(pages, PAGE, 512), rope.view(torch.uint8).view(pages, PAGE, 64)
    f8 = torch.float8_e4m3fn
    cache = (ckv.view(f8), kr.view(f8), torch.full((pages,), STEP, device="cuda"), table[None].cuda())
    return q, torch.cat((lat[:T].double(), rope[:T].double()), 1) * STEP, cache


def bounds(q, raw, step, P, seen):
    """The result in 64 bits and how far the call's may be from it, element for element, for
    rows q [R, 576] of which `seen` [R, T] tells the keys that each sees; raw [T, 576] and step
    [T] are the cache's e4m3 values and scales, P the prefix.

    A weight times its page's scale enters P V as e4m3 hi + e5m2 lo.  A multiple w = 2^k ..
    2^(k+1) of its unit is off by at most 2^(k-8), that is 2^-8 w, while w >= 2^-6 (hi leaves
    less than 2^(k-4), of which lo keeps three bits), and by at most 2^-14 below; the cast to
    fp16 before adds 2^-11.  The unit of a tile of 128 keys is such that its largest weight is
    at least 2^-4 of it; 2^4 if that is the largest of all so far (which a tile of tree rows
    alone leaves as it is); and 2^8.5 if it moved the unit (2^4.75 past the largest before it)
    and stands out by 2^8 from the largest of some 32 keys of its tile.  Scores: 2^-17 of the
    query's largest value in each, 640 fp32 additions, and 2^-20 of their size."""
    R, T = q.shape[0], raw.shape[0]
    qd, key = q.double(), raw * step[:, None]
    s = qd @ key.T * SCALE
    p = torch.softmax(s.masked_fill(~seen, -torch.inf), 1)
    c = key[:, :512]
    out, mean = p @ c, p @ c.abs()
    off = SCALE * (2.0 ** -17 * qd.abs().amax(1) * key.abs().sum(1).max() +
                   640 * 2.0 ** -24 * (qd.abs() @ key.abs().T).amax(1)) + 2.0 ** -20 * (1 + s.abs().amax(1))
    tiles = -(-T // 128)
    at = torch.arange(T, device="cuda")                    # the rows of the last page end its 64 places
    at[T // PAGE * PAGE:] += -T % PAGE
    pad = torch.zeros(R, 128 * tiles, dtype=torch.float64, device="cuda")
    pad[:, at] = p * step
    # a tile's two pages hold the halves of the CTA's columns; 32 keys of a page are a part
    pad = pad.view(R, tiles, 4, 32)
    part = pad.amax(3)
    top, least = part.amax(2), part.amin(2)
    so_far = top.cummax(1).values
    before = torch.cat((torch.zeros(R, 1, device="cuda"), so_far[:, :-1]), 1)
    unit = torch.where(top >= before, top * 2.0 ** -4, top * 2.0 ** 4)     # top >= 2^-4 units
    # only weights below 2^-2 of a tile's largest can be below 2^-6 units
    low = pad < top[:, :, None, None] / 4
    own = -(-P // 128)                                     # first tile of tree rows alone
    unit[:, own:] = so_far[:, own:] * 2.0 ** -4
    low[:, own:] = True
    stands_out = (top > 2.0 ** 8.1 * least) & (top > 2.0 ** 4.85 * before)
    unit = torch.where(stands_out, top * 2.0 ** -8.5, unit)
    each = (2.0 ** -14 * unit[:, :, None] * low.view(R, tiles, 128)).view(R, -1)[:, at]
    quantum = (each * seen) @ raw[:, :512].abs()
    bound = (2.0 ** -8 + 2.0 ** -11 + 2 * off[:, None]) * mean + quantum + 2.0 ** -8 * out.abs()
    return out, torch.logsumexp(s.masked_fill(~seen, -torch.inf), 1), bound, off


def compare(got, lse, out, want_lse, bound, off):
    assert ddt.fault_flags() == 0
    err = (got.double() - out).abs()
    rel = err.norm(dim=1) / out.norm(dim=1)
    assert bool((err <= bound).all()), (float((err / bound).max()), float(rel.max()))
    assert bool(((lse.double() - want_lse).abs() <= off).all())
    # every row, and the library's own limit for a whole output
    assert bool((rel <= bound.norm(dim=1) / out.norm(dim=1)).all())
    assert float(err.norm() / out.norm()) <= 5e-3


def check(q, key, cache, splits):
    T = key.shape[0]
    mask = torch.ones((1, 1, 1), dtype=torch.int64, device="cuda")
    pre = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    got, lse = ddt.verify_attn_q8(q[None, None, :, :512].contiguous(), q[None, None, :, 512:].contiguous(), *cache,
                                  pre, mask, SCALE, max_prefix=T - 1, want_lse=True, num_splits=splits)
    every = torch.ones(HEADS, T, dtype=torch.bool, device="cuda")
    compare(got[0, 0], lse[0, 0], *bounds(q, key / STEP, torch.full((T,), STEP, device="cuda").double(), T - 1, every))


@pytest.mark.parametrize("splits", [0, 1, 16])
@pytest.mark.parametrize("T", [100, 128, 129, 1000, 1024, 4096, 4097, 8192, 32768])
def test_sink_at_the_first_row(T, splits):
    q, key, cache = sink_case(T, [0], T, 0.99)
    check(q, key, cache, splits)


@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("T,sinks", [(1000, [517]), (4096, [4095]), (4096, [0, 1, 2, 3]), (4096, [0, 2100]),
                                     (4100, [3, 64]), (32768, [5, 20000, 32767])])
def test_sinks_elsewhere(T, sinks, splits):
    """A sink in the middle, at the end, several of them: the weights' unit rises and falls."""
    q, key, cache = sink_case(T, sinks, T + len(sinks), 0.95)
    check(q, key, cache, splits)


def test_sink_far_above_everything():
    """Gaps of 20 to 120 nats.  Past 33 nats (2^48) the rest of the keys is allowed to vanish:
    what the sink holds is all that fp32 sums would show."""
    T = 3000
    q, key, cache = sink_case(T, [7], 3, 0.9)
    gap = torch.linspace(20, 120, HEADS)
    q[:, 512] = (gap / (SCALE * STEP * SINK)).to(torch.bfloat16)
    mask = torch.ones((1, 1, 1), dtype=torch.int64, device="cuda")
    pre = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    for splits in (1, 0):
        got, lse = ddt.verify_attn_q8(q[None, None, :, :512].contiguous(), q[None, None, :, 512:].contiguous(), *cache,
                                      pre, mask, SCALE, max_prefix=T - 1, want_lse=True, num_splits=splits)
        s = q.double() @ key.T * SCALE
        out = torch.softmax(s, 1) @ key[:, :512]
        assert ddt.fault_flags() == 0 and bool(torch.isfinite(got).all())
        # the sink's own weight alone: 2^-8, the output's rounding 2^-8; values of the others
        # reach 4, so T of them below 2^-28 of the sink add at most 5e-5
        err = (got[0, 0].double() - out).abs()
        assert bool((err <= 2.0 ** -6.9 * out.abs() + 5e-5).all())
        assert bool(((lse[0, 0].double() - torch.logsumexp(s, 1)).abs() <= 1e-3).all())


@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("Q,prefix", [(5, [3000, 260, 7]), (33, [1000, 2047]), (64, [64, 128, 700]), (128, [1, 129, 900])])
def test_sinks_under_trees_with_uneven_pages(Q, prefix, splits):
    """Trees over caches whose pages have scales of their own, sinks at the first row, in the
    prefix and among the tree's rows; every head weighs them in its own way."""
    rng = np.random.RandomState(Q + len(prefix))
    g = torch.Generator(device="cuda").manual_seed(Q)
    B = len(prefix)
    held = [-(-(P + Q) // PAGE) for P in prefix]
    pages = sum(held)
    table = torch.full((B, max(held)), -1, dtype=torch.int32)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(Q)).int()
    scales = 2.0 ** torch.randint(-9, -5, (pages,), generator=g, device="cuda").float()
    mask, vis = tree_mask(random_parents(rng, B, Q))
    ckv, kr = (torch.zeros((pages, PAGE, n), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for n in (512, 64))
    raws = []
    for b, P in enumerate(prefix):
        own = perm[sum(held[:b]):sum(held[:b + 1])]
        table[b, :held[b]] = own
        own = own.long().cuda()
        step = scales[own].repeat_interleave(PAGE)
        n = held[b] * PAGE
        x = torch.randn((n, 576), generator=g, device="cuda")
        x[:, :512] = 1 + 0.5 * x[:, :512]
        x[:, 512] = 0
        sinks = [0, P // 2, P, P + Q // 2]
        x[sinks, :512] *= 0.01
        x[sinks, 512:] = 0
        x[sinks, 512] = 2.0                                   # fits every page's scale
        f8 = (x / step[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        ckv.view(torch.uint8)[own] = f8[:, :512].view(torch.uint8).reshape(-1, PAGE, 512)
        kr.view(torch.uint8)[own] = f8[:, 512:].contiguous().view(torch.uint8).reshape(-1, PAGE, 64)
        raws.append((f8[:P + Q].double(), step[:P + Q].double()))
    q = torch.zeros(B, Q, HEADS, 576, device="cuda")
    q[..., 512] = torch.rand((B, Q, HEADS), generator=g, device="cuda") * 12 / (SCALE * 2.0)      # 0 .. 12 nats
    q[..., 513:545] = torch.rand((B, Q, HEADS, 1), generator=g, device="cuda") * 1.5 / (SCALE * math.sqrt(32))
    q = q.to(torch.bfloat16)
    out, lse = ddt.verify_attn_q8(q[..., :512].contiguous(), q[..., 512:].contiguous(), ckv, kr, scales, table.cuda(),
                                  torch.tensor(prefix, dtype=torch.int32, device="cuda"), mask, SCALE,
                                  max_prefix=max(prefix), want_lse=True, num_splits=splits)
    for b, P in enumerate(prefix):
        raw, step = raws[b]
        seen = torch.ones((Q, P + Q), dtype=torch.bool, device="cuda")
        seen[:, P:] = torch.from_numpy(vis[b]).cuda()
        seen = seen.repeat_interleave(HEADS, 0)
        compare(out[b].flatten(0, 1), lse[b].flatten(), *bounds(q[b].flatten(0, 1), raw, step, P, seen))
