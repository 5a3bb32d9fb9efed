"""The paged 8-bit latent cache on the GPU against plain references: the page plan, the
quantising write and the compaction value for value, the attention within a bound
derived from its roundings (needs a B200)."""
import numpy as np
import pytest
import torch

import q8_reference as ref
from tree_speculative_decoding_05_b200 import ddt, inputs

pytestmark = pytest.mark.gpu
PAGE = 64
SCALE = float(np.float32(1 / np.sqrt(192.0)))


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def tree_mask(parents):
    """(mask words on the device, bool [B, Q, Q]) of parent arrays [B, Q]."""
    B, Q = parents.shape
    vis = np.zeros((B, Q, Q), bool)
    for i in range(Q):
        if i:
            vis[:, i] = vis[np.arange(B), parents[:, i]]
        vis[:, i, i] = True
    mask, _, status = ddt.build_mask(i32(parents))
    assert int(status.abs().sum()) == 0
    return mask, vis


def random_parents(rng, B, Q):
    p = np.full((B, Q), -1, np.int64)
    for i in range(1, Q):
        p[:, i] = rng.randint(max(0, i - 12), i, B)
    return p


def words(vis):
    """Mask words of a bool [B, Q, Q]."""
    B, Q, _ = vis.shape
    w = np.zeros((B, Q, (Q + 63) // 64), np.uint64)
    for a in range(Q):
        w[:, :, a // 64] |= vis[:, :, a].astype(np.uint64) << np.uint64(a % 64)
    return torch.from_numpy(w.view(np.int64)).cuda()


class Paged:
    """A cache of scattered pages on host and device.  Rows that no request holds, and
    pages in no table, keep the byte 0x7f (NaN) wherever `junk` is true."""

    def __init__(self, rng, lens, *, spare=3, width=None, exps=(-7,), junk=True, layout="split", amp=1.0):
        B = len(lens)
        held = [-(-n // PAGE) for n in lens]
        self.width = width or max(1, max(held, default=1))
        self.pages = sum(held) + spare
        perm = rng.permutation(self.pages)
        self.table = np.full((B, self.width), -1, np.int64)
        self.cache = np.full((self.pages, PAGE, 576), 0x7F if junk else 0, np.uint8)
        self.scales = np.full(self.pages, np.float32(2.0 ** -3))
        at = 0
        for b, n in enumerate(lens):
            for k in range(held[b]):
                page = perm[at]
                at += 1
                self.table[b, k] = page
                m = min(PAGE, n - PAGE * k)
                e = exps[rng.randint(len(exps))]
                self.scales[page] = 2.0 ** e
                self.cache[page, :m] = ref.encode(np.clip(rng.randn(m, 576) * amp * 100, -448, 448))
        self.layout = layout
        self.to_device()

    def to_device(self):
        c = torch.from_numpy(self.cache).cuda()
        if self.layout == "split":
            self.ckv, self.kr = c[..., :512].contiguous(), c[..., 512:].contiguous()
        elif self.layout == "rows":       # one allocation of 576-byte rows
            self.ckv, self.kr = c[..., :512], c[..., 512:]
        else:                             # rows and pages with room between them
            big = torch.full((self.pages, PAGE + 2, 640), 0x7F, dtype=torch.uint8, device="cuda")
            self.ckv, self.kr = big[:, :PAGE, :512], big[:, 1:PAGE + 1, 544:608]
            self.ckv.copy_(c[..., :512])
            self.kr.copy_(c[..., 512:])
            self.big = big
        self.ckv, self.kr = (t.view(torch.float8_e4m3fn) for t in (self.ckv, self.kr))
        self.dscales = torch.from_numpy(self.scales.copy()).cuda()
        self.dtable = i32(self.table)

    def args(self):
        return self.ckv, self.kr, self.dscales, self.dtable

    def bytes(self):
        return torch.cat((self.ckv.view(torch.uint8), self.kr.view(torch.uint8)), 2).cpu().numpy()

    def check(self):
        """Device and reference agree value for value (-0 and +0 are the same value)."""
        torch.cuda.synchronize()
        got, want = ref.DECODE[self.bytes()], ref.DECODE[self.cache]
        assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(self.dscales.cpu().numpy(), self.scales)


# ------------------------------------------------------------------------------ the plan

def plan_state(rng, B, held, num_pages, width):
    perm = rng.permutation(num_pages)
    table = np.full((B, width), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(num_pages, -1, np.int64)
    free[:num_pages - at] = perm[at:]
    return table, list(held), list(free), [num_pages - at]


def run_plan(prefix, rows, state, num_pages, ragged, n_rows=None):
    table, n, free, top = state
    dev = [i32(table), i32(n), i32(free), i32(top)]
    start = np.concatenate([[0], np.cumsum(rows)])
    total = int(start[-1]) if n_rows is None else n_rows
    slots = torch.full((total,), -7, dtype=torch.int64, device="cuda")
    kw = dict(row_start=i32(start)) if ragged else dict(q_len=int(rows[0]))
    _, status = ddt.kv_pages(i32(prefix), *dev, slots=slots, **kw)
    torch.cuda.synchronize()
    want, st = ref.pages(list(map(int, prefix)), list(map(int, rows)), table, n, free, top, num_pages)
    assert status.tolist() == st
    assert np.array_equal(dev[0].cpu().numpy(), table)
    assert dev[1].tolist() == n and dev[3].tolist() == top
    assert dev[2].tolist()[:top[0]] == [int(x) for x in free[:top[0]]]
    flat = [s for w in want for s in w]
    assert slots.tolist()[:len(flat)] == flat and slots.tolist()[len(flat):] == [-7] * (total - len(flat))
    return st


@pytest.mark.parametrize("B,hi,num_pages", [(1, 5, 4), (7, 200, 40), (33, 300, 90), (1024, 130, 2300),
                                            (1025, 64, 1500), (2500, 900, 20000)])
@pytest.mark.parametrize("ragged", [False, True])
def test_pages_random(B, hi, num_pages, ragged):
    rng = np.random.RandomState(B + ragged)
    prefix = rng.randint(0, hi, B)
    rows = rng.randint(0, hi, B) if ragged else np.full(B, rng.randint(1, 128))
    width = -(-2 * (hi + 128) // PAGE)
    held = np.minimum(rng.randint(0, width + 1, B), num_pages // B)
    state = plan_state(rng, B, [int(h) for h in held], num_pages, width)
    run_plan(prefix, rows, state, num_pages, ragged)
    # and on from that state: other lengths, growing and shrinking
    for _ in range(3):
        prefix = np.maximum(0, prefix + rng.randint(-100, 100, B))
        prefix = np.minimum(prefix, width * PAGE - 130)
        rows = rng.randint(0, 128, B) if ragged else rows
        run_plan(prefix, rows, state, num_pages, ragged)


def test_pages_edges():
    rng = np.random.RandomState(5)
    big = 2 ** 31 - 1
    prefix = np.array([0, -1, 63, 64, 128, 10, big, 0, 191, 192])
    rows = np.array([0, 4, 1, 64, 1, 0, 0, 193, 1, 0])
    state = plan_state(rng, 10, [0, 2, 0, 3, 1, 0, 1, 0, 0, 0], 24, 3)
    st = run_plan(prefix, rows, state, 24, True)
    assert st == [0, 4, 0, 0, 0, 0, 4, 4, 0, 0]


def test_pages_refused_state_changes_nothing():
    """A stack height outside the pool, or more pages given back than it has room for."""
    rng = np.random.RandomState(6)
    for n_rows in (8, 6000):       # slots by the planning launch, and by their own
        for top, held in ((-1, [1, 1]), (9, [1, 1]), (7, [3, 3])):
            table, n, free, _ = plan_state(rng, 2, [3, 3], 8, 4)
            state = (table, held, free, [top])
            rows = np.array([2, n_rows - 2]) if n_rows == 8 else np.array([100, 20])
            assert run_plan(np.array([0, 0]), rows, state, 8, True, n_rows=n_rows) == [ref.BAD_INDEX] * 2


def test_pages_bad_counts_and_negative_rows():
    rng = np.random.RandomState(7)
    state = plan_state(rng, 4, [1, 1, 1, 1], 12, 2)
    state[1][1], state[1][2] = 3, -1
    st = run_plan(np.array([60, 5, 5, 5]), np.array([10, 3, 3, 3]), state, 12, True)
    assert st == [0, ref.BAD_INDEX, ref.BAD_INDEX, 0]
    table, n, free, top = plan_state(rng, 3, [1, 1, 1], 12, 2)
    start = i32([0, 5, 2, 9])      # request 1 would have -3 rows
    slots, status = ddt.kv_pages(i32([60, 5, 5]), i32(table), i32(n), i32(free), i32(top), row_start=start, n_rows=9)
    assert status.tolist() == [0, ref.BAD_LENGTH, 0]
    assert all(-1 <= s < 12 * 64 for s in slots.tolist()[5:])


def test_pages_step_taken_back_restores_the_state():
    rng = np.random.RandomState(8)
    B, num_pages, width = 300, 1500, 8
    prefix = rng.randint(1, 64 * 4, B)
    held = [-(-int(p) // PAGE) for p in prefix]
    table, n, free, top = plan_state(rng, B, held, num_pages, width)
    dev = [i32(table), i32(n), i32(free), i32(top)]
    before = [t.clone() for t in dev]
    ddt.kv_pages(i32(prefix), *dev, q_len=128)
    assert int(dev[1].sum()) > sum(held)
    ddt.kv_pages(i32(prefix), *dev, q_len=0)
    for a, b in zip(dev, before):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------- the write

def f64(t):
    return t.double().cpu().numpy()


def rows_of(rng, lens, amp=1.0):
    """Per request bf16 rows [n, 576] as fp64, some rows much larger or smaller."""
    out = []
    for n in lens:
        x = rng.randn(n, 576) * amp * 2.0 ** rng.randint(-9, 4, (n, 1))
        out.append(f64(torch.from_numpy(x).to(torch.bfloat16)))
    return out


def run_write(paged, prefix, rows, uniform, max_rows=None):
    flat = np.concatenate(rows) if rows else np.zeros((0, 576))
    lat = torch.from_numpy(np.ascontiguousarray(flat[:, :512])).to(torch.bfloat16).cuda()
    rope = torch.from_numpy(np.ascontiguousarray(flat[:, 512:])).to(torch.bfloat16).cuda()
    if uniform:
        B, q = len(rows), len(rows[0])
        status = ddt.kv_write_q8(*paged.args(), i32(prefix), lat.view(B, q, 512), rope.view(B, q, 64))
    else:
        start = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
        status = ddt.kv_write_q8(*paged.args(), i32(prefix), lat, rope, row_start=i32(start),
                                 max_rows=max_rows or max(len(r) for r in rows))
    st = ref.write(paged.cache, paged.scales, paged.table, [int(p) for p in prefix], rows)
    assert status.tolist() == st
    paged.check()
    return st


@pytest.mark.parametrize("layout", ["split", "rows", "room"])
@pytest.mark.parametrize("q", [1, 2, 33, 64, 65, 128])
def test_write_tree_blocks(q, layout):
    rng = np.random.RandomState(q)
    prefix = np.array([0, 1, 31, 63, 64, 100, 127, 128, 200])
    paged = Paged(rng, [int(p) + q for p in prefix], exps=(-12, -7, -2), layout=layout)
    # the rows to come hold junk; live rows are those below the prefix
    for b, P in enumerate(prefix):
        for pos in range(int(P), int(P) + q):
            paged.cache[paged.table[b, pos // PAGE], pos % PAGE] = 0x7F
    paged.to_device()
    st = run_write(paged, prefix, rows_of(rng, [q] * len(prefix)), True)
    assert st == [0] * len(prefix)
    if layout == "room":           # nothing beside the rows was written
        big = paged.big.clone()
        big[:, :PAGE, :512] = 0x7F
        big[:, 1:PAGE + 1, 544:608] = 0x7F
        assert bool((big == 0x7F).all())


@pytest.mark.parametrize("lens", [[1], [0, 5, 0, 64, 700], [129, 1, 63, 65, 1000, 2], [0, 0, 0]])
def test_write_ragged(lens):
    rng = np.random.RandomState(sum(lens))
    prefix = np.array([int(p) for p in rng.randint(0, 300, len(lens))])
    paged = Paged(rng, [int(p) + n for p, n in zip(prefix, lens)], exps=(-9, -5))
    run_write(paged, prefix, rows_of(rng, lens), False, max_rows=max(1, max(lens)))


def test_write_zero_tiny_and_huge_rows():
    rng = np.random.RandomState(2)
    x = [np.zeros((5, 576)), np.full((70, 576), 2.0 ** -133), np.full((3, 576), -float(2 ** 127)),
         np.full((9, 576), 2.0 ** -40 * 3)]
    x[0][2, 7] = -0.0
    prefix = np.array([10, 60, 0, 127])
    paged = Paged(rng, [int(p) + len(r) for p, r in zip(prefix, x)], exps=(-40, 3))
    run_write(paged, prefix, x, False)


def test_write_every_bf16_value():
    """All finite bf16 magnitudes of one binade and its neighbours, ties among them."""
    rng = np.random.RandomState(3)
    bits = np.arange(0x3A00, 0x4380, dtype=np.int32)[:64 * 36]
    v = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)
    x = np.zeros((64, 576))
    x[:, :36] = f64(v).reshape(64, 36)
    x[:, 36:72] = -x[:, :36]
    paged = Paged(rng, [64])
    run_write(paged, np.array([0]), [x], True)


def test_write_not_finite():
    rng = np.random.RandomState(4)
    rows = rows_of(rng, [5, 66, 5, 3])
    rows[0][3, 100] = np.nan
    rows[1][65, 575], rows[1][0, 0] = np.inf, -np.inf
    rows[3][:] = np.nan
    prefix = np.array([7, 30, 64, 1])
    paged = Paged(rng, [int(p) + len(r) for p, r in zip(prefix, rows)], exps=(-9,))
    st = run_write(paged, prefix, rows, False)
    assert st == [ref.NOT_FINITE, ref.NOT_FINITE, 0, ref.NOT_FINITE]
    for b, P in enumerate(prefix):  # no row of a request holds NaN
        for pos in range(int(P) + len(rows[b])):
            assert not np.isnan(ref.DECODE[paged.cache[paged.table[b, pos // PAGE], pos % PAGE]]).any()


def test_write_statuses_of_long_prompts():
    """More pages a request than a cluster takes: statuses raised by any page, over whatever
    stood there, eagerly and in a replayed graph."""
    rng = np.random.RandomState(73)
    lens, prefix = [300, 5, 0, 700, 260, 66, 520], np.array([10, 63, 5, 0, 64, 200, 1])
    paged = Paged(rng, [int(p) + max(n, 1) for p, n in zip(prefix, lens)], exps=(-9,))
    paged.table[4, 3] = -1                       # a page that is none
    paged.to_device()
    rows = rows_of(rng, lens)
    rows[0][0, 5], rows[3][699, 575], rows[3][640, 0], rows[5][30, 3] = np.nan, np.inf, -np.inf, np.nan
    flat = torch.from_numpy(np.concatenate(rows)).to(torch.bfloat16).cuda()
    lat, rope = flat[:, :512].contiguous(), flat[:, 512:].contiguous()
    start, pre = i32(np.concatenate([[0], np.cumsum(lens)])), i32(prefix)
    status = i32([99, -7, 8, 3, 0, 1, 55])
    call = lambda: ddt.kv_write_q8(*paged.args(), pre, lat, rope, row_start=start, max_rows=700, status=status)  # noqa: E731
    call()
    want = ref.write(paged.cache, paged.scales, paged.table, [int(p) for p in prefix], rows)
    assert want == [ref.NOT_FINITE, 0, 0, ref.NOT_FINITE, ref.BAD_INDEX, ref.NOT_FINITE, 0]
    assert status.tolist() == want
    paged.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        status.fill_(77)
        graph.replay()
        assert status.tolist() == want
    # the same rows again, at scales that no longer change but for pages written from their start
    ref.write(paged.cache, paged.scales, paged.table, [int(p) for p in prefix], rows)
    paged.check()


def test_write_refused_requests_change_nothing():
    rng = np.random.RandomState(5)
    rows = rows_of(rng, [70, 70, 70, 70])
    prefix = np.array([10, -1, 64 * 3 - 69, 20])
    paged = Paged(rng, [80, 80, 64 * 3, 90], width=3)
    paged.table[0, 1] = paged.pages      # a page that is none, where the rows go
    paged.table[3, 0], paged.table[3, 2] = paged.table[3, 0], -5   # unused entry: not looked at
    paged.to_device()
    assert run_write(paged, prefix, rows, True) == [ref.BAD_INDEX, ref.BAD_PREFIX, ref.BAD_PREFIX, 0]
    # ragged: rows outside what was handed over, or more than max_rows
    lat = torch.zeros(10, 512, dtype=torch.bfloat16, device="cuda")
    rope = torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda")
    before = paged.bytes()
    for start in ([0, 4, 20, 20, 20], [0, 9, 5, 5, 5], [-3, 0, 0, 0, 0], [0, 0, 0, 0, 9]):
        st = ddt.kv_write_q8(*paged.args(), i32([0, 0, 0, 0]), lat, rope, row_start=i32(start), max_rows=3)
        assert all(s in (0, ref.BAD_LENGTH) for s in st.tolist()) and ref.BAD_LENGTH in st.tolist()
    assert np.array_equal(paged.bytes()[paged.table[1, 0]], before[paged.table[1, 0]])


# ------------------------------------------------------------------------ the compaction

def run_compact(paged, prefix, path, accept, in_place=False):
    p = i32(prefix)
    new, status = ddt.kv_compact_q8(*paged.args(), p, i32(path), i32(accept), new_prefix_lens=p if in_place else None)
    want, st = ref.compact(paged.cache, paged.scales, paged.table, [int(x) for x in prefix], path, [int(a) for a in accept])
    assert status.tolist() == st and new.tolist() == want
    paged.check()
    return st


@pytest.mark.parametrize("layout", ["split", "rows", "room"])
@pytest.mark.parametrize("Q", [1, 2, 33, 65, 128])
def test_compact_random_paths(Q, layout):
    rng = np.random.RandomState(Q)
    prefix = np.array([0, 1, 40, 63, 64, 100, 127, 300])
    paged = Paged(rng, [int(p) + Q for p in prefix], exps=(-20, -8, -7, -6, 0), layout=layout)
    path = np.full((len(prefix), Q), -1)
    accept = rng.randint(1, Q + 1, len(prefix))
    for b, a in enumerate(accept):
        path[b, :a] = np.sort(rng.permutation(Q)[:a])
    run_compact(paged, prefix, path, accept, in_place=Q % 2 == 1)


@pytest.mark.parametrize("kind", ["reversed", "same row", "racing", "identity", "shifted back"])
def test_compact_paths(kind):
    rng = np.random.RandomState(1)
    Q = 128
    one = {"reversed": np.arange(Q)[::-1], "same row": np.full(Q, 77), "identity": np.arange(Q),
           "racing": np.minimum(np.arange(Q) + 1, Q - 1), "shifted back": np.maximum(np.arange(Q) - 1, 0)}[kind]
    prefix = np.array([0, 17, 63])
    paged = Paged(rng, [int(p) + Q for p in prefix], exps=(-9, -6, -5))
    run_compact(paged, prefix, np.stack([one] * 3), np.array([Q, Q - 1, Q]))


def test_compact_refused_requests_change_nothing():
    rng = np.random.RandomState(2)
    Q = 9
    prefix = np.array([5, 5, -1, 64 * 2 - 8, 60, 5, 5])
    paged = Paged(rng, [20, 20, 20, 128, 80, 20, 20], width=2, exps=(-9, -6))
    path = np.tile(np.arange(Q)[::-1], (7, 1))
    path[0, 3] = Q
    path[5, 2] = -1
    accept = np.array([5, 0, 3, 3, 3, 2, Q + 1])    # request 5's bad entry lies past its accepted ones
    paged.table[4, 1] = -1
    paged.to_device()
    st = run_compact(paged, prefix, path, accept)
    assert st == [2, 5, 4, 4, 2, 0, 5]


# -------------------------------------------------------------------------- the attention

def queries(rng, B, Q, amp=1.0):
    q = torch.from_numpy(rng.randn(B, Q, 64, 576) * amp).to(torch.bfloat16)
    return q, q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda()


def check_attention(paged, prefix, q, vis, out, lse, scale=SCALE, requests=None, rel_l2=5e-3):
    torch.cuda.synchronize()
    assert ddt.fault_flags() == 0
    got, gl = f64(out), f64(lse)
    num = den = 0.0
    for b in requests if requests is not None else range(len(prefix)):
        o, l, mean, quantum, off = ref.attend(f64(q[b]), paged.cache, paged.scales, paged.table[b], int(prefix[b]), vis[b], scale)
        bound = ref.error_bound(o, mean, quantum, off)
        err = np.abs(got[b] - o)
        assert np.isfinite(got[b]).all()
        assert (err <= bound).all(), (b, float((err / bound).max()))
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(gl[b]), empty)
        assert (np.abs(gl[b][~empty] - l[~empty]) <= off[~empty]).all()
        num, den = num + float(((got[b] - o) ** 2).sum()), den + float((o ** 2).sum())
    # over the whole output the roundings average out: 2^-9 of the result's own plus the
    # weights' (2^-8 at most each)
    assert num <= rel_l2 ** 2 * den, (num / den) ** 0.5


CASES = [
    (1, [0]), (1, [1]), (1, [62]), (1, [63]), (1, [64]), (1, [65, 0, 200, 127]), (2, [126]), (9, [256]),
    (33, [31, 32, 95]), (64, [0, 64]), (65, [63, 191]), (127, [1]), (128, [0, 129]),
]


@pytest.mark.parametrize("Q,prefix", CASES)
def test_attention_shapes(Q, prefix):
    rng = np.random.RandomState(Q * 7 + len(prefix))
    paged = Paged(rng, [p + Q for p in prefix], exps=(-8, -7, -6))
    mask, vis = tree_mask(random_parents(rng, len(prefix), Q))
    q, ql, qr = queries(rng, len(prefix), Q)
    status = torch.full((len(prefix),), -9, dtype=torch.int32, device="cuda")
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=max(prefix),
                                  want_lse=True, status=status)
    check_attention(paged, prefix, q, vis, out, lse)
    assert status.tolist() == [0] * len(prefix)


@pytest.mark.parametrize("splits", [0, 1, 2, 3, 7, 64])
@pytest.mark.parametrize("Q", [1, 5])
def test_attention_splits(Q, splits):
    """Forced splits, more of them than there are tiles among others."""
    rng = np.random.RandomState(splits)
    prefix = [900, 3, 0, 383]
    paged = Paged(rng, [p + Q for p in prefix], exps=(-8, -7))
    mask, vis = tree_mask(random_parents(rng, 4, Q))
    q, ql, qr = queries(rng, 4, Q)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=900,
                                  want_lse=True, num_splits=splits)
    check_attention(paged, prefix, q, vis, out, lse)


@pytest.mark.parametrize("layout", ["split", "rows", "room"])
def test_attention_strides(layout):
    rng = np.random.RandomState(11)
    prefix = [100, 260]
    paged = Paged(rng, [p + 7 for p in prefix], layout=layout)
    mask, vis = tree_mask(random_parents(rng, 2, 7))
    q, ql, qr = queries(rng, 2, 7)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=260, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


@pytest.mark.parametrize("exps", [(-40,), (-30, -7), (-12, -9, -7, -4), (0, 3)])
def test_attention_page_scales(exps):
    """Pages of very different scales in one request.  The queries shrink as the scales
    grow, so that the softmax keeps several keys."""
    rng = np.random.RandomState(13)
    prefix = [500, 120]
    paged = Paged(rng, [p + 3 for p in prefix], exps=exps)
    mask, vis = tree_mask(random_parents(rng, 2, 3))
    q, ql, qr = queries(rng, 2, 3, amp=2.0 ** (-7 - max(exps)))
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=500, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


@pytest.mark.parametrize("amp", [0.0, 1e-3, 8.0, 40.0])
def test_attention_flat_and_peaked(amp):
    """From a uniform softmax to one that a single key wins, with growing maxima."""
    rng = np.random.RandomState(17)
    prefix = [700]
    paged = Paged(rng, [703], exps=(-7,))
    mask, vis = tree_mask(random_parents(rng, 1, 3))
    q, ql, qr = queries(rng, 1, 3, amp=amp)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=700, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


def test_attention_rising_maximum():
    """Keys aligned with the query grow from page to page, so the running maximum rises
    all the way (and its reference with it)."""
    rng = np.random.RandomState(19)
    Q, prefix = 2, [64 * 14 + 5]
    paged = Paged(rng, [prefix[0] + Q], exps=(-7,))
    q, ql, qr = queries(rng, 1, Q)
    d = f64(q)[0, 0, 0] / np.abs(f64(q)[0, 0, 0]).max()
    for k in range(15):
        m = min(PAGE, prefix[0] + Q - PAGE * k)
        paged.cache[paged.table[0, k], :m] = ref.encode(d[None, :] * (4.0 + 8.0 * k) + rng.randn(m, 576) * 2)
    paged.to_device()
    mask, vis = tree_mask(random_parents(rng, 1, Q))
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=prefix[0], want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


def test_attention_rows_that_see_nothing():
    rng = np.random.RandomState(23)
    Q, prefix = 5, [0, 0, 70]
    paged = Paged(rng, [p + Q for p in prefix])
    vis = np.zeros((3, Q, Q), bool)
    vis[0, 2, 1] = vis[1, :, 0] = True           # request 0: node 2 alone sees a row; request 2: prefix only
    q, ql, qr = queries(rng, 3, Q)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), words(vis), SCALE, max_prefix=70, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)
    assert float(out[0, 0].float().abs().max()) == 0.0 and bool(torch.isneginf(lse[0, 0]).all())


def test_attention_mask_bits_past_q_len_are_ignored():
    rng = np.random.RandomState(29)
    Q, prefix = 6, [130, 58]
    paged = Paged(rng, [p + Q for p in prefix])
    mask, vis = tree_mask(random_parents(rng, 2, Q))
    q, ql, qr = queries(rng, 2, Q)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask | (-1 << Q), SCALE, max_prefix=130, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


def test_attention_not_finite_queries_stay_in_their_rows():
    rng = np.random.RandomState(31)
    Q, prefix = 3, [200]
    paged = Paged(rng, [203])
    mask, vis = tree_mask(random_parents(rng, 1, Q))
    q, ql, qr = queries(rng, 1, Q)
    clean, cl = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=200, want_lse=True)
    ql[0, 1, 5, 17], qr[0, 0, 63, 2] = float("nan"), float("inf")
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=200, want_lse=True)
    bad = torch.zeros(1, Q, 64, dtype=torch.bool, device="cuda")
    bad[0, 1, 5] = bad[0, 0, 63] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], cl[~bad])


def test_attention_bad_requests():
    rng = np.random.RandomState(37)
    Q, prefix = 4, [100, -1, 64 * 3 - 3, 100, 100]
    paged = Paged(rng, [104, 10, 64 * 3, 104, 104], width=3)
    mask, vis = tree_mask(random_parents(rng, 5, Q))
    q, ql, qr = queries(rng, 5, Q)
    paged.table[3, 1], paged.table[4, 2] = paged.pages, 10 ** 9      # the second lies past the rows
    paged.dtable = i32(paged.table)
    out = torch.full((5, Q, 64, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, Q, 64), 3.0, device="cuda")
    status = torch.full((5,), -9, dtype=torch.int32, device="cuda")
    for splits in (1, 2):
        ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=100, out=out, lse=lse,
                           status=status, num_splits=splits)
        assert status.tolist() == [0, 4, 4, 2, 0]
        assert bool((out[1:3] == 3.0).all()) and bool((lse[1:3] == 3.0).all())
        check_attention(paged, prefix, q, vis, out, lse, requests=[0, 3, 4])


def test_attention_many_short_requests():
    """More requests than one sorted schedule holds, most of them shorter than a tile."""
    rng = np.random.RandomState(41)
    B, Q = 700, 1
    prefix = [int(x) for x in rng.randint(0, 150, B)]
    paged = Paged(rng, [p + Q for p in prefix])
    vis = np.ones((B, 1, 1), bool)
    q, ql, qr = queries(rng, B, Q)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), words(vis), SCALE, max_prefix=150, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


def test_attention_pages_past_two_gigabytes():
    rng = np.random.RandomState(43)
    Q, prefix = 3, [150, 90]
    small = Paged(rng, [p + Q for p in prefix])
    pages = 70000                                   # 2.3 GB of latent rows
    ckv = torch.zeros((pages, 64, 512), dtype=torch.uint8, device="cuda")
    kr = torch.zeros((pages, 64, 64), dtype=torch.uint8, device="cuda")
    scales = torch.ones(pages, device="cuda")
    far = torch.arange(pages - small.pages, pages, device="cuda")
    ckv[far], kr[far] = small.ckv.view(torch.uint8), small.kr.view(torch.uint8)
    scales[far] = small.dscales
    table = torch.where(small.dtable >= 0, small.dtable + (pages - small.pages), -1).int()
    args = (ckv.view(torch.float8_e4m3fn), kr.view(torch.float8_e4m3fn), scales, table)
    mask, vis = tree_mask(random_parents(rng, 2, Q))
    q, ql, qr = queries(rng, 2, Q)
    rows = rows_of(rng, [Q, Q])
    flat = torch.from_numpy(np.stack(rows)).to(torch.bfloat16).cuda()
    st = ddt.kv_write_q8(*args, i32(prefix), flat[..., :512].contiguous(), flat[..., 512:].contiguous())
    assert st.tolist() == ref.write(small.cache, small.scales, small.table, prefix, rows)
    out, lse = ddt.verify_attn_q8(ql, qr, *args, i32(prefix), mask, SCALE, max_prefix=150, want_lse=True)
    check_attention(small, prefix, q, vis, out, lse)
    path = np.array([[0, 2, -1], [0, 1, 2]])
    new, st = ddt.kv_compact_q8(*args, i32(prefix), i32(path), i32([2, 3]))
    want, _ = ref.compact(small.cache, small.scales, small.table, prefix, path, [2, 3])
    assert new.tolist() == want
    got = torch.cat((args[0].view(torch.uint8)[far], args[1].view(torch.uint8)[far]), 2).cpu().numpy()
    assert np.array_equal(ref.DECODE[got], ref.DECODE[small.cache], equal_nan=True)


# --------------------------------------------------------------------- together, as used

class Loop:
    """A few decode steps over the paged cache: plan, tree, write, attention, accept,
    compaction, with all lengths on the device."""

    def __init__(self, seed, B=6, Q=17, D=8, K=4, steps=4):
        rng = np.random.RandomState(seed)
        self.B, self.Q, self.steps = B, Q, steps
        prompt = [int(x) for x in rng.randint(0, 150, B)]
        width, self.num_pages = 8, 8 * B
        self.table, self.n, self.free, self.top = plan_state(rng, B, [0] * B, self.num_pages, width)
        self.drafts = [inputs.draft_batch(seed * 50 + k, B, D, K) for k in range(steps)]
        self.conts = []
        for d in self.drafts:
            c = np.zeros((B, Q), np.int32)
            for b in range(B):
                for j in range(Q):
                    c[b, j] = d.tok[b, min(j, D - 1), 0] if rng.rand() < 0.7 else 31999
            self.conts.append(c)
        self.prompt = prompt
        self.prompt_rows = rows_of(rng, prompt)
        self.rows = [rows_of(rng, [Q] * B) for _ in range(steps)]
        self.q = [torch.from_numpy(rng.randn(B, Q, 64, 576)).to(torch.bfloat16) for _ in range(steps)]
        self.cache = np.zeros((self.num_pages, PAGE, 576), np.uint8)
        self.scales = np.ones(self.num_pages, np.float32)

    def to_device(self):
        bf = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()  # noqa: E731
        c = torch.from_numpy(self.cache).cuda()
        d = {"ckv": c[..., :512].contiguous().view(torch.float8_e4m3fn),
             "kr": c[..., 512:].contiguous().view(torch.float8_e4m3fn), "scales": torch.from_numpy(self.scales).cuda(),
             "table": i32(self.table), "n": i32(self.n), "free": i32(self.free), "top": i32(self.top),
             "prefix": i32([0] * self.B)}
        flat = np.concatenate(self.prompt_rows)
        d["prompt"] = (bf(flat[:, :512]), bf(flat[:, 512:]), i32(np.concatenate([[0], np.cumsum(self.prompt)])))
        d["steps"] = [{"lp": torch.from_numpy(f.lp).cuda(), "tok": torch.from_numpy(f.tok).cuda(),
                       "root": i32(f.root_token), "cont": i32(c).long(), "ckv": bf(np.stack(r)[..., :512]),
                       "kr": bf(np.stack(r)[..., 512:]), "ql": q[..., :512].contiguous().cuda(),
                       "qr": q[..., 512:].contiguous().cuda()}
                      for f, c, r, q in zip(self.drafts, self.conts, self.rows, self.q)]
        return d

    def admit(self, d):
        state = (d["table"], d["n"], d["free"], d["top"])
        lat, rope, start = d["prompt"]
        _, st = ddt.kv_pages(d["prefix"], *state, row_start=start, n_rows=lat.shape[0])
        w = ddt.kv_write_q8(d["ckv"], d["kr"], d["scales"], d["table"], d["prefix"], lat, rope, row_start=start,
                            max_rows=max(self.prompt))
        d["prefix"] += start[1:] - start[:-1]
        return st, w

    def step(self, d, s):
        state = (d["table"], d["n"], d["free"], d["top"])
        args = (d["ckv"], d["kr"], d["scales"], d["table"])
        slots, st0 = ddt.kv_pages(d["prefix"], *state, q_len=self.Q)
        tree = ddt.tree_build(s["lp"], s["tok"], s["root"], self.Q)
        st1 = ddt.kv_write_q8(*args, d["prefix"], s["ckv"], s["kr"])
        out, lse = ddt.verify_attn_q8(s["ql"], s["qr"], *args, d["prefix"], tree["mask"], SCALE, max_prefix=300, want_lse=True)
        target = torch.gather(s["cont"], 1, tree["depth"].long()).int()
        path, alen, bonus, _ = ddt.tree_accept(tree["node_tokens"], target, tree["next_token"], tree["next_sibling"])
        _, st2 = ddt.kv_compact_q8(*args, d["prefix"], path, alen, new_prefix_lens=d["prefix"])
        return {"slots": slots, "st": st0 + st1 + st2, "out": out, "lse": lse, "path": path, "alen": alen,
                "mask": tree["mask"], "parents": tree["parents"]}

    def check(self, d, got, seen_prefix):
        """One step's outputs against the references, which advance with it."""
        torch.cuda.synchronize()
        prefix = seen_prefix
        slots, st = ref.pages(prefix, [self.Q] * self.B, self.table, self.n, self.free, self.top, self.num_pages)
        assert st == [0] * self.B and got["slots"].tolist() == [x for s in slots for x in s]
        assert int(got["st"].abs().sum()) == 0
        return got["path"].cpu().numpy(), got["alen"].tolist()


def follow(loop, d, results):
    """Checks a run of steps; the references follow the device's accepted paths."""
    prefix = [0] * loop.B
    ref.pages(prefix, loop.prompt, loop.table, loop.n, loop.free, loop.top, loop.num_pages)
    ref.write(loop.cache, loop.scales, loop.table, prefix, loop.prompt_rows)
    prefix = list(loop.prompt)
    moved = 0
    for k, got in enumerate(results):
        path, alen = loop.check(d, got, prefix)
        ref.write(loop.cache, loop.scales, loop.table, prefix, loop.rows[k])
        parents = got["parents"].cpu().numpy()
        vis = np.zeros((loop.B, loop.Q, loop.Q), bool)
        for i in range(loop.Q):
            if i:
                vis[:, i] = vis[np.arange(loop.B), parents[:, i]]
            vis[:, i, i] = True
        check_attention(loop, prefix, loop.q[k], vis, got["out"], got["lse"])
        prefix, _ = ref.compact(loop.cache, loop.scales, loop.table, prefix, path, alen)
        moved += sum(alen)
    assert d["prefix"].tolist() == prefix and moved > loop.B * len(results)
    got = torch.cat((d["ckv"].view(torch.uint8), d["kr"].view(torch.uint8)), 2).cpu().numpy()
    assert np.array_equal(ref.DECODE[got], ref.DECODE[loop.cache], equal_nan=True)
    assert np.array_equal(d["scales"].cpu().numpy(), loop.scales)


def test_decode_loop():
    loop = Loop(1)
    d = loop.to_device()
    st, w = loop.admit(d)
    assert int(st.abs().sum()) == 0 and int(w.abs().sum()) == 0
    follow(loop, d, [loop.step(d, s) for s in d["steps"]])


def test_decode_loop_captured_and_on_another_stream():
    """The same loop with each step captured in a CUDA graph, replayed on a side stream."""
    loop = Loop(2, steps=3)
    d = loop.to_device()
    loop.admit(d)
    warm = loop.to_device()            # first calls outside capture, on state of their own
    loop.admit(warm)
    loop.step(warm, warm["steps"][0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    results, graphs = [], []
    for s in d["steps"]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(loop.step(d, s))
        graphs.append(g)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for g in graphs:
            g.replay()
    torch.cuda.current_stream().wait_stream(side)
    follow(loop, d, results)


def test_attention_long_ragged_whole_output():
    """Long ragged caches, every row of the output, against elementary operations in 64
    bits on the device."""
    rng = np.random.RandomState(47)
    Q, prefix = 33, [6000, 5, 2900, 4100, 640, 63, 1, 3333]
    B, width = len(prefix), 96
    pages = sum(-(-(p + Q) // PAGE) for p in prefix)
    table = np.full((B, width), -1, np.int64)
    perm, at = rng.permutation(pages), 0
    for b, P in enumerate(prefix):
        n = -(-(P + Q) // PAGE)
        table[b, :n] = perm[at:at + n]
        at += n
    g = torch.Generator(device="cuda").manual_seed(5)
    raw = (torch.randn((pages, PAGE, 576), generator=g, device="cuda") * 90).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = 2.0 ** torch.randint(-8, -4, (pages,), generator=g, device="cuda").float()
    mask, vis = tree_mask(random_parents(rng, B, Q))
    q, ql, qr = queries(rng, B, Q)
    status = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    out, lse = ddt.verify_attn_q8(ql, qr, raw[..., :512], raw[..., 512:], scales, i32(table), i32(prefix), mask, SCALE,
                                  max_prefix=6100, want_lse=True, status=status)
    assert status.tolist() == [0] * B and ddt.fault_flags() == 0
    num = den = 0.0
    for b, P in enumerate(prefix):
        n = -(-(P + Q) // PAGE)
        ids = torch.from_numpy(table[b, :n]).cuda()
        key = (raw.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * scales[ids].double()[:, None, None]).flatten(0, 1)[:P + Q]
        s = q[b].cuda().double().flatten(0, 1) @ key.T * SCALE
        seen = torch.ones((Q, P + Q), dtype=torch.bool, device="cuda")
        seen[:, P:] = torch.from_numpy(vis[b]).cuda()
        s = s.view(Q, 64, P + Q).masked_fill(~seen[:, None, :], -torch.inf)
        w = torch.softmax(s, 2).flatten(0, 1)
        o = (w @ key[:, :512]).view(Q, 64, 512)
        err = (out[b].double() - o).abs()
        # the terms of q8_reference.error_bound: scores off by at most 4e-3 (a bound over
        # these inputs: 2^-17 * 5 * 576 * 10 * SCALE and 640 * 2^-24 * 576 * 5 * 10 * SCALE);
        # each weight times its page's scale off by at most 2^-14 of the row's largest, so
        # the sum of weight * value by that times the sum of the values' magnitudes
        mean = (w @ key[:, :512].abs()).view(Q, 64, 512)
        step = scales[ids].double().repeat_interleave(PAGE)[:P + Q]
        quantum = 2.0 ** -14 * (w * step).amax(1).view(Q, 64, 1) * (key[:, :512].abs() / step[:, None]).sum(0)
        assert bool((err <= (2.0 ** -8 + 8e-3) * mean + 2.0 ** -8 * o.abs() + quantum).all())
        assert float((lse[b].double() - torch.logsumexp(s, 2)).abs().max()) <= 4e-3
        num, den = num + float((err ** 2).sum()), den + float((o ** 2).sum())
    assert (num / den) ** 0.5 <= 5e-3


def test_attention_replayed_with_other_lengths():
    """One captured call, replayed as the lengths on the device change: the cut into chunks
    follows them."""
    rng = np.random.RandomState(59)
    Q, most = 2, [1500, 1500, 1500]
    paged = Paged(rng, [p + Q for p in most])
    mask, vis = tree_mask(random_parents(rng, 3, Q))
    q, ql, qr = queries(rng, 3, Q)
    prefix = i32(most)
    args = (ql, qr, *paged.args(), prefix, mask, SCALE)
    ddt.verify_attn_q8(*args, max_prefix=1500)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = ddt.verify_attn_q8(*args, max_prefix=1500, want_lse=True)
    for lens in (most, [3, 1400, 700], [0, 0, 1], [1500, 2, 127]):
        prefix.copy_(i32(lens))
        graph.replay()
        check_attention(paged, lens, q, vis, out, lse)


def test_attention_requests_share_pages():
    """Requests with a common prefix read the same pages."""
    rng = np.random.RandomState(61)
    Q, prefix = 4, [200, 200, 200]
    paged = Paged(rng, [p + Q for p in prefix])
    paged.table[1:, :3] = paged.table[0, :3]
    paged.dtable = i32(paged.table)
    mask, vis = tree_mask(random_parents(rng, 3, Q))
    q, ql, qr = queries(rng, 3, Q)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=200, want_lse=True)
    check_attention(paged, prefix, q, vis, out, lse)


@pytest.mark.parametrize("last", [8191, 9000])
def test_attention_many_chunks(last):
    """As many chunks as may be forced (64 of one tile, or 36 of two), merged, and a request
    of a few of them beside."""
    rng = np.random.RandomState(last)
    prefix = [last, 1300, 100]
    paged = Paged(rng, [p + 1 for p in prefix], exps=(-8, -7))
    q, ql, qr = queries(rng, 3, 1)
    vis = np.ones((3, 1, 1), bool)
    out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), words(vis), SCALE, max_prefix=last,
                                  want_lse=True, num_splits=64)
    check_attention(paged, prefix, q, vis, out, lse)
    plain, _ = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), words(vis), SCALE, max_prefix=last, num_splits=64)
    assert torch.equal(plain, out)


@pytest.mark.parametrize("splits", [0, 3])
def test_attention_prefix_past_the_stated_bound(splits):
    """max_prefix only plans the cut: longer requests are answered all the same."""
    rng = np.random.RandomState(71 + splits)
    Q, prefix = 3, [2500, 700, 5]
    paged = Paged(rng, [p + Q for p in prefix])
    mask, vis = tree_mask(random_parents(rng, 3, Q))
    q, ql, qr = queries(rng, 3, Q)
    for bound in (0, 1100):
        out, lse = ddt.verify_attn_q8(ql, qr, *paged.args(), i32(prefix), mask, SCALE, max_prefix=bound,
                                      want_lse=True, num_splits=splits)
        check_attention(paged, prefix, q, vis, out, lse)


def test_no_requests():
    none = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    bf16 = torch.bfloat16
    cache = (none(4, 64, 512, dtype=torch.float8_e4m3fn), none(4, 64, 64, dtype=torch.float8_e4m3fn),
             torch.ones(4, device="cuda"), none(0, 3))
    free, count = i32([0, 1, 2, 3]), i32([4])
    slots, status = ddt.kv_pages(none(0), none(0, 3), none(0), free, count, q_len=5)
    assert slots.numel() == status.numel() == 0 and count.tolist() == [4]
    assert ddt.kv_write_q8(*cache, none(0), none(0, 5, 512, dtype=bf16), none(0, 5, 64, dtype=bf16)).numel() == 0
    out, lse = ddt.verify_attn_q8(none(0, 5, 64, 512, dtype=bf16), none(0, 5, 64, 64, dtype=bf16), *cache, none(0),
                                  none(0, 5, 1, dtype=torch.int64), SCALE, max_prefix=9, want_lse=True)
    assert out.shape == (0, 5, 64, 512) and lse.shape == (0, 5, 64)
    new, status = ddt.kv_compact_q8(*cache, none(0), none(0, 5), none(0))
    assert new.numel() == status.numel() == 0


def test_calls_on_a_given_stream_keep_their_buffers():
    """Outputs and workspace that a call allocates for a given stream, dropped at once."""
    rng = np.random.RandomState(67)
    Q, prefix = 1, [3000, 2000]
    paged = Paged(rng, [p + Q for p in prefix])
    vis = np.ones((2, 1, 1), bool)
    q, ql, qr = queries(rng, 2, Q)
    side, pre, mask = torch.cuda.Stream(), i32(prefix), words(vis)
    out = torch.empty_like(ql)
    lse = torch.empty((2, Q, 64), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        ddt.verify_attn_q8(ql, qr, *paged.args(), pre, mask, SCALE, max_prefix=3000, out=out, lse=lse, stream=side)
        torch.full((8 << 20,), 1e9, device="cuda")     # would land in a workspace given back too soon
    torch.cuda.current_stream().wait_stream(side)
    check_attention(paged, prefix, q, vis, out, lse)


def test_two_streams_at_once_give_the_same():
    rng = np.random.RandomState(51)
    Q, prefix = 9, [2000, 900, 40]
    paged = Paged(rng, [p + Q for p in prefix])
    mask, _ = tree_mask(random_parents(rng, 3, Q))
    sets = [queries(rng, 3, Q)[1:] for _ in range(2)]
    call = lambda s, stream=None: ddt.verify_attn_q8(*s, *paged.args(), i32(prefix), mask, SCALE, max_prefix=2000,  # noqa: E731
                                                     want_lse=True, stream=stream)
    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    pre, got = i32(prefix), []
    for _ in range(5):
        for x, s in zip(sets, streams):
            with torch.cuda.stream(s):
                got.append(ddt.verify_attn_q8(*x, *paged.args(), pre, mask, SCALE, max_prefix=2000, want_lse=True))
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(got):
        assert torch.equal(o, want[k % 2][0]) and torch.equal(l, want[k % 2][1])


def test_binding_refusals_on_the_device():
    rng = np.random.RandomState(53)
    paged = Paged(rng, [70, 80])
    mask, _ = tree_mask(random_parents(rng, 2, 3))
    _, ql, qr = queries(rng, 2, 3)
    c, k, s, t = paged.args()
    p = i32([60, 70])
    good = lambda **o: ddt.verify_attn_q8(*[o.get(n, v) for n, v in (("ql", ql), ("qr", qr), ("c", c), ("k", k), ("s", s),  # noqa: E731
                                          ("t", t), ("p", p), ("m", mask))], SCALE, max_prefix=70)
    good()
    for bad in ({"ql": ql.float()}, {"qr": qr.transpose(1, 2)}, {"c": c.view(torch.uint8)}, {"k": k[:-1]}, {"s": s[:-1]},
                {"s": s.double()}, {"t": t.long()}, {"t": t[:1]}, {"p": p.long()}, {"p": p.cpu()}, {"m": mask[:, :2]},
                {"c": c.transpose(0, 1)}, {"qr": qr[:, :, :32]}):
        with pytest.raises(ddt.DdtError):
            good(**bad)
    rows = torch.zeros(2, 3, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    for bad in ((rows[0].float(), rows[1]), (rows[0][:, :2], rows[1]), (rows[0].transpose(0, 1), rows[1])):
        with pytest.raises(ddt.DdtError):
            ddt.kv_write_q8(c, k, s, t, p, *bad)
    with pytest.raises(ddt.DdtError):
        ddt.kv_write_q8(c, k, s, t, p, rows[0][0], rows[1][0], row_start=i32([0, 1, 3]))
    for most in (-1, 1 << 31, (1 << 32) + 3):
        with pytest.raises(ddt.DdtError):
            ddt.kv_write_q8(c, k, s, t, p, rows[0][0], rows[1][0], row_start=i32([0, 1, 3]), max_rows=most)
    path = i32([[0, 1, 2], [0, 1, 2]])
    for bad in ((path[:, :2], p), (path.long(), p), (path, p[:1])):
        with pytest.raises(ddt.DdtError):
            ddt.kv_compact_q8(c, k, s, t, p, *bad)
    state = i32([[-1] * 4] * 2), i32([0, 0]), i32(range(8)), i32([8])
    for bad in ({}, {"q_len": 3, "row_start": i32([0, 1, 2])}, {"q_len": -1}, {"row_start": i32([0, 1, 2])},
                {"q_len": 3, "n_rows": 5}, {"q_len": 3, "slots": torch.zeros(5, dtype=torch.int64, device="cuda")}):
        with pytest.raises(ddt.DdtError):
            ddt.kv_pages(p, *state, **bad)
    torch.cuda.synchronize()
