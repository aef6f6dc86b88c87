"""Memory that the paged cache's calls allocate belongs to the stream that they launch on.

A block of another stream may still be in use there, or be given to the next
tensor of that stream while the call's kernels write it.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def cpu_cache(monkeypatch):
    """A cache over host memory whose library calls do nothing, and a log of allocations with the stream they are made on."""
    c = dfl.PagedCache(1, 4, 16, 2, 64, 2, 2, device="cpu")
    c._lib = SimpleNamespace(dfl_kv4_attn=lambda *a: log.append(("launch", a[-1])) or 0)
    log, on = [], [7]   # 7: the current stream's handle

    @contextlib.contextmanager
    def scope(s):
        on.append(s.cuda_stream)
        yield
        on.pop()

    def logged(f):
        def g(*a, **kw):
            log.append(("alloc", on[-1]))
            return f(*a, **kw)
        return g

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: on[-1], raising=False)
    monkeypatch.setattr(torch.cuda, "stream", scope)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: _Stream(h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0))
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, logged(getattr(torch, f)))
    return c, log


@pytest.mark.parametrize("stream,handle", [(None, 7), (_Stream(9), 9), (11, 11), (0, 0)])
def test_outputs_and_scratch_are_allocated_on_the_stream_of_the_call(cpu_cache, stream, handle):
    c, log = cpu_cache
    Q, K = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)
    c.attn(0, Q, K, K, stream=stream)   # out and scratch
    c.attn(0, Q, K, K, stream=stream)   # out
    assert [x for x, _ in log].count("alloc") == 3 and {s for _, s in log} == {handle}


@pytest.mark.gpu
@pytest.mark.parametrize("by_handle", [False, True])
def test_blocks_of_a_call_on_a_side_stream(by_handle):
    dfl.build()
    torch.cuda.set_device(0)
    c = dfl.PagedCache(1, 4, 16, 2, 64, 2, 2)
    Q, K = (torch.zeros((2, 3, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.attn(0, Q, K, K, stream=s.cuda_stream if by_handle else s)
    s.synchronize()
    own = {out.data_ptr()} | {ws.data_ptr() for ws, _, _ in c._attn_ws.values()}
    found = [seg["stream"] for seg in torch.cuda.memory_snapshot() for p in own
             if seg["address"] <= p < seg["address"] + seg["total_size"]]
    assert len(own) == 2 and found == [s.cuda_stream] * 2
    assert not bool(out.any())
    assert dfl.dfl_get_device_error() == 0


def test_scratch_does_not_grow_with_the_number_of_shapes(cpu_cache):
    c, log = cpu_cache
    for B in range(1, 65):
        for Hq in (2, 4, 8):
            Q, K = torch.zeros((2, B, Hq, 64), dtype=torch.bfloat16), torch.zeros((2, B, 2, 64), dtype=torch.bfloat16)
            c.attn(0, Q, K, K, out=torch.zeros_like(Q))
    held = {ws.data_ptr(): ws.numel() for ws, _, _ in c._attn_ws.values()}
    # a size for up to 8, 16, 64 and more query rows to a K/V head
    assert len(held) == 4 and sum(held.values()) <= 64 << 20
    for (B, Hq), (ws, at, size) in c._attn_ws.items():
        assert size >= dfl.workspace_size(dfl.DFL_OP_KV4_ATTN, N=2, B=B, Hq=Hq, Hkv=2, hd=64) and at == ws.data_ptr()
