"""What the binding of the paged calls does around a launch, on the CPU with the launch
itself taken out: where the buffers that a call makes for itself come from."""
import contextlib
import os
import subprocess
import sys

import pytest
import torch

from tree_speculative_decoding_05_b200 import build as ddt_build
from tree_speculative_decoding_05_b200 import ddt


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


CACHE = (torch.zeros(40, 64, 512, dtype=torch.uint8).view(torch.float8_e4m3fn),
         torch.zeros(40, 64, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(40), i32(2, 20))
# every call that makes buffers of its own: outputs, statuses, a workspace (the last)
CALLS = {
    "kv_pages": (lambda stream: ddt.kv_pages(i32(2), i32(2, 20), i32(2), i32(40), i32(1), q_len=5, stream=stream), 2, 0),
    "kv_write_q8": (lambda stream: ddt.kv_write_q8(*CACHE, i32(2), bf16(2, 5, 512), bf16(2, 5, 64), stream=stream), 1, 0),
    "kv_compact_q8": (lambda stream: ddt.kv_compact_q8(*CACHE, i32(2), i32(2, 5), i32(2), stream=stream), 2, 0),
    "verify_attn_q8": (lambda stream: ddt.verify_attn_q8(
        bf16(2, 5, 64, 512), bf16(2, 5, 64, 64), *CACHE, i32(2), torch.ones(2, 5, 1, dtype=torch.int64), 0.07,
        max_prefix=1000, want_lse=True, num_splits=4, stream=stream), 2, 1),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [False, True])
def test_buffers_come_from_the_given_stream(monkeypatch, name, given):
    ddt_build.build()
    ddt.load()
    side, entered, made, recorded = object(), [], [], []

    @contextlib.contextmanager
    def stream_context(s):
        entered.append(s)
        yield
        entered.pop()

    def watch(make):
        def made_here(*args, **kwargs):
            t = make(*args, **kwargs)
            made.append((t, entered[-1] if entered else None))
            return t
        return made_here

    call, returned, scratch = CALLS[name]
    launched = []
    monkeypatch.setattr(ddt, "_device_of", lambda t, name: -1)          # as the tensors say here
    monkeypatch.setattr(ddt, "_launch", lambda *a: launched.append((a, tuple(entered))))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t, s)), raising=False)
    fresh = {n: getattr(torch, n) for n in ("empty", "empty_like")}
    with monkeypatch.context() as m:
        for n, f in fresh.items():
            m.setattr(torch, n, watch(f))
        got = call(side if given else None)
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    assert len(launched) == 1 and launched[0][1] == ()
    assert len(made) == returned + scratch and len(got) == returned
    assert all(s is (side if given else None) for _, s in made)
    # what is handed out lives until the stream that the caller is on is done with it too
    kept = [t.data_ptr() for t, s in recorded if s == "current"]
    assert sorted(kept) == (sorted(t.data_ptr() for t in got) if given else [])


def test_binding_loads_without_the_raw_stream_lookup():
    """A torch that lacks the short way to the current stream still imports the binding, and
    takes the public way."""
    code = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
from tree_speculative_decoding_05_b200 import ddt
class Stream:
    cuda_stream = 42
torch.cuda.current_stream = lambda dev=None: Stream if dev == 3 else None
torch.cuda.current_device = lambda: 3
seen = []
ddt._launch(lambda *a: seen.append(a) or ddt.DDT_OK, "what", 3, None, 7, 8)
assert seen == [(7, 8, 42)], seen
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


def test_workspace_is_sized_on_the_tensors_device(monkeypatch):
    """How far a call may be cut depends on the SMs of the device that it runs on, which need
    not be the current one: the size is asked there, as the launch asks again."""
    ddt_build.build()
    lib, current, asked = ddt.load(), [7], []

    @contextlib.contextmanager
    def device_context(d):
        current.append(d.index if isinstance(d, torch.device) else d)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                asked.append((name, current[-1]))
                return 0 if name == "ddt_verify_attn_q8" else getattr(lib, name)(*args)
            return call

    monkeypatch.setattr(ddt, "_device_of", lambda t, name: -1)      # as the tensors say here
    monkeypatch.setattr(ddt, "load", Lib)
    monkeypatch.setattr(ddt, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device_context)
    args = (bf16(2, 5, 64, 512), bf16(2, 5, 64, 64), *CACHE, i32(2), torch.ones(2, 5, 1, dtype=torch.int64), 0.07)
    ddt.verify_attn_q8(*args, max_prefix=1000)
    size, splits = ddt.verify_attn_q8_workspace_size(*args, max_prefix=1000)
    assert [n for n, _ in asked] == ["ddt_verify_attn_q8_workspace_size", "ddt_verify_attn_q8",
                                     "ddt_verify_attn_q8_workspace_size", "ddt_verify_attn_q8_num_splits"]
    assert all(d == -1 for _, d in asked), asked
    assert size > 0 and splits > 1 and current == [7]
