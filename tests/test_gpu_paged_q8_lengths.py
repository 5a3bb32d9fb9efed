"""Attention over the paged 8-bit cache at lengths and batch sizes where the work list
changes its form (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from test_gpu_paged_q8 import Paged, check_attention, i32, queries, words
from tree_speculative_decoding_05_b200 import ddt

pytestmark = pytest.mark.gpu
SCALE = float(np.float32(1 / np.sqrt(192.0)))


def test_cut_of_requests_longer_than_65535_tiles():
    """73 single tokens, one over 270000 tiles of 128 rows and the others over 65600: the cut
    that the schedule's cost favours is chunks of 54000, five for the longest (the longest
    load of 74 CTA pairs by hand: 77 whole chunks, so 108000 tiles; with four chunks of 67500,
    72 others of 65600 make 131200).  All rows are those of one page, over and over, so that the result is
    the attention over that page."""
    tiles = [270000] + [65600] * 72
    B, g = len(tiles), torch.Generator(device="cuda").manual_seed(3)
    prefix = torch.tensor([128 * n - 1 for n in tiles], dtype=torch.int32, device="cuda")
    page = (torch.randn((1, 64, 576), generator=g, device="cuda") * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache = (page[..., :512], page[..., 512:], torch.full((1,), 2.0 ** -6, device="cuda"),
             torch.zeros((B, 2 * max(tiles)), dtype=torch.int32, device="cuda"))
    q = torch.randn((B, 1, 64, 576), generator=g, device="cuda").to(torch.bfloat16)
    call = (q[..., :512].contiguous(), q[..., 512:].contiguous(), *cache, prefix,
            torch.ones((B, 1, 1), dtype=torch.int64, device="cuda"), SCALE)
    size, most = ddt.verify_attn_q8_workspace_size(*call, max_prefix=128 * max(tiles) - 1)
    assert most == 5
    space = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out, lse = ddt.verify_attn_q8(*call, max_prefix=128 * max(tiles) - 1, want_lse=True, workspace=space)
    assert ddt.fault_flags() == 0
    assert int(space[:4].view(torch.int32)) == 54000          # tiles of a chunk, at the workspace's start
    key = page[0].double() * 2.0 ** -6
    s = q[:, 0].double() @ key.T * SCALE
    p = torch.softmax(s, 2)
    # sums over up to 65600 tiles in fp32: a thread's row sum adds one number a tile (half a
    # step, 2^-24), O takes eight products a tile (cut off, 2^-23)
    want = torch.logsumexp(s, 2) + torch.tensor([math.log(2 * n) for n in tiles], device="cuda").double()[:, None]
    assert float((lse[:, 0].double() - want).abs().max()) <= 65600 * 2.0 ** -24 + 1e-3
    bound = (8 * 65600 * 2.0 ** -23 + 65600 * 2.0 ** -24 + 2.0 ** -7) * (p @ key[:, :512].abs())
    assert bool(((out[:, 0].double() - p @ key[:, :512]).abs() <= bound).all())


@pytest.mark.parametrize("B", [512, 513])
@pytest.mark.parametrize("splits", [0, 3])
def test_forced_splits_around_512_requests(B, splits):
    """Past 512 requests none is cut, whatever was asked for, and none is put in order; the
    results are the same."""
    rng = np.random.RandomState(B + splits)
    prefix = [int(x) for x in rng.randint(0, 70, B)]
    prefix[B // 2], prefix[B - 1] = 900, 640
    paged = Paged(rng, [p + 1 for p in prefix])
    q, ql, qr = queries(rng, B, 1)
    args = (ql, qr, *paged.args(), i32(prefix), words(np.ones((B, 1, 1), bool)), SCALE)
    status = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    out, lse = ddt.verify_attn_q8(*args, max_prefix=900, want_lse=True, num_splits=splits, status=status)
    check_attention(paged, prefix, q, np.ones((B, 1, 1), bool), out, lse)
    assert status.tolist() == [0] * B
    assert ddt.verify_attn_q8_workspace_size(*args, max_prefix=900, num_splits=splits)[1] == (3 if splits and B == 512 else 1)
