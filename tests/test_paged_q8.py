"""The paged 8-bit cache on the CPU: struct layouts, what the C entries and the binding
refuse before any launch, and the tests' own reference against closed forms."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import q8_reference as ref
from tree_speculative_decoding_05_b200 import build as ddt_build
from tree_speculative_decoding_05_b200 import ddt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    ddt_build.build()
    return ddt.load()


@pytest.mark.parametrize("cname,pystruct", [("ddt_q8_cache", ddt.Q8Cache),
                                             ("ddt_attn_q8_args", ddt.AttnQ8Args)])
def test_struct_layouts_match_c(tmp_path, cname, pystruct):
    fields = [f for f, _ in pystruct._fields_]
    body = "\n".join(f'  printf("{f} %zu\\n", offsetof({cname}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ddt.h"\nint main(void){\n'
                   f'  printf("sizeof %zu\\n", sizeof({cname}));\n{body}\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got["sizeof"]) == ctypes.sizeof(pystruct)
    for f in fields:
        assert int(got[f]) == getattr(pystruct, f).offset, f


FAKE = 0x10000  # an aligned address that no refused call follows


def good_cache(**over):
    c = ddt.Q8Cache(c_kv=FAKE, k_rope=FAKE, scales=FAKE, block_table=FAKE, ckv_page_stride=64 * 512,
                    ckv_row_stride=512, kr_page_stride=64 * 64, kr_row_stride=64, num_pages=4, max_blocks=3)
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [{"c_kv": None}, {"k_rope": None}, {"scales": None}, {"block_table": None}, {"c_kv": FAKE + 8},
              {"k_rope": FAKE + 4}, {"ckv_row_stride": 496}, {"kr_row_stride": 48}, {"ckv_row_stride": 520},
              {"ckv_page_stride": 64 * 512 - 16}, {"kr_page_stride": 64 * 64 + 8}, {"num_pages": 0},
              {"max_blocks": 0}, {"max_blocks": (1 << 24) + 1}, {"ckv_page_stride": -64 * 512}]


@pytest.mark.parametrize("over", BAD_CACHES)
def test_bad_caches_are_refused(lib, over):
    c = good_cache(**over)
    r = ctypes.byref(c)
    assert lib.ddt_kv_write_q8(r, FAKE, None, 2, 5, 0, 10, FAKE, FAKE, None, None) == ddt.DDT_ERR_INVALID_ARG
    assert lib.ddt_kv_compact_q8(r, FAKE, FAKE, FAKE, 2, 5, None, None, None) == ddt.DDT_ERR_INVALID_ARG
    a = attn_args(cache=c)
    assert lib.ddt_verify_attn_q8(ctypes.byref(a), None) == ddt.DDT_ERR_INVALID_ARG


def attn_args(**over):
    a = ddt.AttnQ8Args(B=2, q_len=9, num_heads=64, d_latent=512, d_rope=64, max_prefix=100,
                       cache=good_cache(), prefix_lens=FAKE, q_lat=FAKE, q_rope=FAKE, mask=FAKE, out=FAKE,
                       softmax_scale=0.07)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    ({"q_len": 0}, ddt.DDT_ERR_UNSUPPORTED), ({"q_len": 129}, ddt.DDT_ERR_UNSUPPORTED),
    ({"num_heads": 32}, ddt.DDT_ERR_UNSUPPORTED), ({"d_latent": 256}, ddt.DDT_ERR_UNSUPPORTED),
    ({"d_rope": 32}, ddt.DDT_ERR_UNSUPPORTED), ({"B": -1}, ddt.DDT_ERR_INVALID_ARG),
    ({"max_prefix": -1}, ddt.DDT_ERR_INVALID_ARG), ({"num_splits": 65}, ddt.DDT_ERR_INVALID_ARG),
    ({"num_splits": -1}, ddt.DDT_ERR_INVALID_ARG), ({"q_lat": None}, ddt.DDT_ERR_INVALID_ARG),
    ({"q_rope": None}, ddt.DDT_ERR_INVALID_ARG), ({"mask": None}, ddt.DDT_ERR_INVALID_ARG),
    ({"out": None}, ddt.DDT_ERR_INVALID_ARG), ({"prefix_lens": None}, ddt.DDT_ERR_INVALID_ARG),
    ({"q_lat": FAKE + 2}, ddt.DDT_ERR_INVALID_ARG), ({"out": FAKE + 16}, ddt.DDT_ERR_INVALID_ARG),
    ({"softmax_scale": 0.0}, ddt.DDT_ERR_INVALID_ARG), ({"softmax_scale": float("nan")}, ddt.DDT_ERR_INVALID_ARG),
    ({"softmax_scale": float("inf")}, ddt.DDT_ERR_INVALID_ARG),
    ({"cache": good_cache(max_blocks=1), "q_len": 65}, ddt.DDT_ERR_INVALID_ARG),
    ({"B": 0}, ddt.DDT_OK)])
def test_attention_refusals(lib, over, want):
    assert lib.ddt_verify_attn_q8(ctypes.byref(attn_args(**over)), None) == want


def test_other_refusals(lib):
    pages = lambda B=2, q=5, n=10, np_=4, mb=3, p=FAKE: lib.ddt_kv_pages(p, None, B, q, n, np_, mb, p, p, p, p, None, None, None)  # noqa: E731
    for bad in (dict(B=-1), dict(q=-1), dict(n=-1), dict(np_=-1), dict(mb=-1), dict(mb=(1 << 24) + 1), dict(p=None)):
        assert pages(**bad) == ddt.DDT_ERR_INVALID_ARG, bad
    assert pages(B=0, p=None) == ddt.DDT_OK
    c = ctypes.byref(good_cache())
    write = lambda B=2, q=5, m=0, n=10, p=FAKE, r=FAKE: lib.ddt_kv_write_q8(c, p, None, B, q, m, n, r, r, None, None)  # noqa: E731
    for bad in (dict(B=-1), dict(q=-1), dict(m=-1), dict(n=-1), dict(p=None), dict(r=None), dict(r=FAKE + 4)):
        assert write(**bad) == ddt.DDT_ERR_INVALID_ARG, bad
    assert lib.ddt_kv_write_q8(None, FAKE, None, 2, 5, 0, 10, FAKE, FAKE, None, None) == ddt.DDT_ERR_INVALID_ARG
    assert write(B=0) == ddt.DDT_OK
    assert write(B=1 << 20, q=1 << 20) == ddt.DDT_ERR_UNSUPPORTED
    compact = lambda B=2, q=5, p=FAKE: lib.ddt_kv_compact_q8(c, p, p, p, B, q, None, None, None)  # noqa: E731
    assert compact(B=-1) == compact(p=None) == ddt.DDT_ERR_INVALID_ARG
    assert compact(q=0) == compact(q=129) == ddt.DDT_ERR_UNSUPPORTED
    assert compact(B=0) == ddt.DDT_OK


def test_split_bound_and_workspace(lib):
    def of(**kw):
        a = ctypes.byref(attn_args(cache=good_cache(max_blocks=600), **kw))
        return lib.ddt_verify_attn_q8_num_splits(a), lib.ddt_verify_attn_q8_workspace_size(a)

    assert of(B=64, q_len=33, max_prefix=4096) == (1, 0)         # enough items without cutting
    for kw in (dict(B=1, q_len=33, max_prefix=32768), dict(B=64, q_len=1, max_prefix=4096), dict(B=1, q_len=9, max_prefix=1000)):
        s, ws = of(**kw)
        tiles = -(-(kw["max_prefix"] + kw["q_len"]) // 128)
        assert 1 < s <= min(32, tiles) and ws == 256 + s * kw["B"] * kw["q_len"] * 64 * 513 * 4
    assert of(B=1, q_len=9, max_prefix=256)[0] == 1              # few tiles
    assert of(B=3, q_len=5, max_prefix=10, num_splits=7) == (7, 256 + 7 * 3 * 5 * 64 * 513 * 4)
    assert of(B=513, q_len=1, max_prefix=4096, num_splits=4) == (1, 0)
    assert of(B=0) == (1, 0) and of(q_len=0) == (1, 0)


def test_binding_refuses_tensors_of_the_host():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f8 = lambda *s: torch.zeros(s, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    cache = (f8(4, 64, 512), f8(4, 64, 64), torch.ones(4), i32(2, 3))
    with pytest.raises(ddt.DdtError):
        ddt.kv_pages(i32(2), i32(2, 3), i32(2), i32(4), i32(1), q_len=5)
    with pytest.raises(ddt.DdtError):
        ddt.kv_write_q8(*cache, i32(2), torch.zeros(2, 5, 512), torch.zeros(2, 5, 64))
    with pytest.raises(ddt.DdtError):
        ddt.kv_compact_q8(*cache, i32(2), i32(2, 5), i32(2))
    with pytest.raises(ddt.DdtError):
        ddt.verify_attn_q8(torch.zeros(2, 5, 64, 512), torch.zeros(2, 5, 64, 64), *cache, i32(2),
                           torch.zeros(2, 5, 1, dtype=torch.int64), 0.07, max_prefix=10)


def test_reference_bytes_against_torch():
    v = ref.DECODE
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    x = np.concatenate([np.random.RandomState(0).randn(20000) * 10.0 ** np.random.RandomState(1).uniform(-4, 2.6, 20000),
                        v[np.isfinite(v)], (v[:126] + v[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]])
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x.astype(np.float32)), want)


def test_reference_fit():
    for e in range(-60, 100):
        for f in (1.0, 1.5, 1.75, 1.7578125, 1.9921875):
            s = ref.fit(f * 2.0 ** e)
            assert f * 2.0 ** e <= 448 * s and (s == 2.0 ** -40 or f * 2.0 ** e > 224 * s)
    assert ref.fit(0.0) == 2.0 ** -40


def test_reference_pages_by_hand():
    table = np.full((3, 4), -1)
    table[0, :2], table[2, :3] = (7, 3), (1, 0, 4)
    n, free, top = [2, 0, 3], [5, 6, 2, -1, -1, -1, -1, -1], [3]
    # request 0 grows by one page, request 1 by two, request 2 gives two back
    slots, st = ref.pages([128, 60, 10], [1, 9, 0], table, n, free, top, 8)
    assert st == [0, 0, 0] and n == [3, 2, 1] and top == [2]
    assert table.tolist() == [[7, 3, 0, -1], [4, 2, -1, -1], [1, -1, -1, -1]]
    assert slots == [[0], [4 * 64 + 60, 4 * 64 + 61, 4 * 64 + 62, 4 * 64 + 63] + [128 + i for i in range(5)], []]
    # taken back: the same pages in the same places
    slots, st = ref.pages([128, 0, 130], [0, 0, 0], table, n, free, top, 8)
    assert st == [0, 0, 0] and table[2].tolist() == [1, 0, 4, -1] and table[0].tolist() == [7, 3, -1, -1]
    assert top == [3] and free[:3] == [5, 6, 2]
    # request 1 wants more than there is: it and those behind it are not served
    slots, st = ref.pages([128, 256, 130], [1, 0, 64], table, n, free, top, 8)
    assert st == [0, ref.NO_PAGES, ref.NO_PAGES] and n == [3, 0, 3] and slots[2] == [-1] * 64
