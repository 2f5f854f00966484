"""New tensors and workspaces of the calls that take a stream come from the memory of the stream that
the kernels run on, the default stream (handle 0) among them."""
import contextlib

import pytest

import moe_expert_amd as M


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("current", [0, 111])
@pytest.mark.parametrize("given", [None, 0, 111, 222])
def test_allocation_stream(monkeypatch, current, given):
    """On a stand-in for torch's streams.  As torch has it, an external stream of handle 0 is not the
    default stream but some stream of a pool."""
    import torch
    active = [current]

    @contextlib.contextmanager
    def on(stream):
        active.append(stream.cuda_stream)
        yield
        active.pop()

    device = torch.device("cuda:0")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream(h or 999))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(active[-1]))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: (shape, dtype, device, active[-1]))
    monkeypatch.setattr(M, "_CURRENT", (lambda: 0, lambda i: active[-1]))
    want = current if given is None else given
    assert M._empty((3, 4), torch.float32, device, given) == ((3, 4), torch.float32, device, want)
    assert active == [current]


@pytest.mark.gpu
@pytest.mark.parametrize("current", ["default", "side"])
@pytest.mark.parametrize("given", ["none", "default", "side", "other"])
def test_calls_allocate_on_their_stream(monkeypatch, current, given):
    """Every allocation that the calls make, on the real streams; and the results are the same."""
    import torch
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    handle = {"none": None, "default": 0, "side": side.cuda_stream, "other": other.cuda_stream}[given]
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = torch.randn(40, 256, generator=g, device="cuda"), torch.rand(256, generator=g, device="cuda")
    a = torch.randn(2, 16, 256, generator=g, device="cuda").half()
    b = torch.randn(2, 64, 16, generator=g, device="cuda").half()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ranks, scales, off, adapter = i32(16, 9), torch.rand(2, generator=g, device="cuda"), i32(0, 30, 40), i32(1, 0)

    def calls(stream):
        y, yq, _ = M.qmm_rmsnorm(x, w, 1e-6, y=torch.float16, yq=True, stream=stream)
        ids, weights = M.qmm_moe_route(x, 4, stream=stream)
        lists = M.qmm_moe_dispatch(ids, 256, stream=stream)
        values = M.qmm_dequantize_q8_1(yq, 256, stream=stream)
        out = torch.zeros_like(base)
        torch.cuda.synchronize()
        return [y, yq, ids, weights, *lists, values, M.qmm_lora(x, a, b, ranks, scales, off, adapter, out, base=base, stream=stream)]

    base = torch.randn(40, 64, generator=g, device="cuda")
    want = calls(None)
    torch.cuda.synchronize()
    seen, empty = [], torch.empty

    def recorded(*args, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    with torch.cuda.stream(side) if current == "side" else contextlib.nullcontext():
        here = torch.cuda.current_stream().cuda_stream
        monkeypatch.setattr(torch, "empty", recorded)
        got = calls(handle)
        monkeypatch.setattr(torch, "empty", empty)
        torch.cuda.synchronize()
    # the norm's two, the routing's two, the dispatch's five lists and its workspace, the values, the adapters' workspace
    assert len(seen) == 12 and set(seen) == {here if handle is None else handle}
    assert all(torch.equal(p, q) for p, q in zip(got, want))
