"""Calls of the paged cache on a stream that is given, beside work on the current one that
nothing orders against it (needs a B200)."""
import numpy as np
import pytest
import torch

from test_gpu_paged_q8 import SCALE, Paged, check_attention, i32, queries, random_parents, rows_of, tree_mask
from tree_speculative_decoding_05_b200 import ddt

pytestmark = pytest.mark.gpu


def test_split_calls_on_two_streams_in_turn():
    """Calls of equal workspace size on the current stream and on a side stream, in turn and
    without a wait between them: a workspace given back by one is never the other's while its
    kernels run."""
    rng = np.random.RandomState(83)
    Q, prefix = 5, [6000, 5000]
    paged = Paged(rng, [p + Q for p in prefix])
    mask, _ = tree_mask(random_parents(rng, 2, Q))
    sets = [queries(rng, 2, Q)[1:] for _ in range(2)]
    pre = i32(prefix)
    args = lambda k: (*sets[k], *paged.args(), pre, mask, SCALE)  # noqa: E731
    assert ddt.verify_attn_q8_workspace_size(*args(0), max_prefix=6000)[1] > 1
    want = [ddt.verify_attn_q8(*args(k), max_prefix=6000, want_lse=True) for k in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for k, s in ((0, None), (1, side)):
            got.append((k, ddt.verify_attn_q8(*args(k), max_prefix=6000, want_lse=True, stream=s)))
        # outputs dropped while their kernels run, and memory of the same size written at once
        ddt.verify_attn_q8(*args(1), max_prefix=6000, want_lse=True, stream=side)
        torch.full_like(sets[0][0], 7.0)
    torch.cuda.synchronize()
    assert ddt.fault_flags() == 0
    for k, (o, l) in got:
        assert torch.equal(o, want[k][0]) and torch.equal(l, want[k][1])


def test_cache_calls_on_a_side_stream():
    """Plan, write and compaction on a given stream: statuses and slots that they make."""
    rng = np.random.RandomState(89)
    prefix = [10, 64, 200]
    side = torch.cuda.Stream()
    paged = Paged(rng, [p + 9 for p in prefix], exps=(-9,))
    pre, path, alen = i32(prefix), i32([[0, 2, 3, -1, -1, -1, -1, -1, -1]] * 3), i32([3, 2, 1])
    rows = torch.from_numpy(np.stack(rows_of(rng, [9] * 3))).to(torch.bfloat16).cuda()
    lat, rope = rows[..., :512].contiguous(), rows[..., 512:].contiguous()
    held = i32([1, 1, 4])
    table, free, top = i32(np.arange(15).reshape(3, 5) % 8), i32(range(20)), i32([20])
    torch.cuda.synchronize()
    busy = torch.empty(64 << 20, device="cuda")
    for _ in range(10):
        busy.fill_(1.0)                 # work on the current stream that the side stream passes by
    st0 = ddt.kv_write_q8(*paged.args(), pre, lat, rope, stream=side)
    new, st1 = ddt.kv_compact_q8(*paged.args(), pre, path, alen, stream=side)
    slots, st2 = ddt.kv_pages(pre, table, held, free, top, q_len=9, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert st0.tolist() == st1.tolist() == st2.tolist() == [0, 0, 0]
    assert new.tolist() == [13, 66, 201] and slots.numel() == 27 and int(slots.min()) >= 0


def test_captured_calls_on_a_given_stream():
    """A graph whose capture forks to a side stream that the calls are given, replayed: their
    buffers belong to the graph."""
    rng = np.random.RandomState(97)
    Q, prefix = 3, [4000, 1500]
    paged = Paged(rng, [p + Q for p in prefix])
    mask, vis = tree_mask(random_parents(rng, 2, Q))
    q, ql, qr = queries(rng, 2, Q)
    pre, side = i32(prefix), torch.cuda.Stream()
    rows = torch.zeros(2, Q, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, Q, 64, dtype=torch.bfloat16, device="cuda")
    spare = Paged(rng, [p + Q for p in prefix])
    call = lambda s: (ddt.verify_attn_q8(ql, qr, *paged.args(), pre, mask, SCALE, max_prefix=4000, want_lse=True, stream=s),  # noqa: E731
                      ddt.kv_write_q8(*spare.args(), pre, *rows, stream=s))
    call(None)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            got = call(side)
            torch.cuda.current_stream().wait_stream(side)
        graphs.append((g, got))
    for g, ((out, lse), status) in graphs * 2:
        out.fill_(3.0), lse.fill_(3.0), status.fill_(3)
        g.replay()
        torch.full((32 << 20,), 1e9, device="cuda")
        check_attention(paged, prefix, q, vis, out, lse)
        assert status.tolist() == [0, 0]
