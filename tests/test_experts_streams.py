"""The experts' calls on a stream that is not the current one: the results that a call allocates are memory of the
stream it launches on, as under torch.cuda.stream(stream).  Memory of the current stream could still be read by work
queued there, or be handed out again there, while the other stream writes it."""
import contextlib

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
from combine_moe_route_02_gb300 import experts

BF16, U8 = torch.bfloat16, torch.uint8


def calls(dev, R=96, H=256, I=128, E=3):
    """Each call with everything but `out`, as a function of the keyword arguments."""
    def b(*shape):
        return torch.ones(shape, dtype=BF16, device=dev)

    def q(*shape):
        return torch.full(shape, 0x38, dtype=U8, device=dev)        # 1.0

    def s(*shape):
        return torch.ones(shape, device=dev)

    off = torch.tensor([0, R // 2, R // 2, R], dtype=torch.int32, device=dev)
    x8, xs, W1, s1 = q(R, H), s(R, H // 128), q(E, 2 * I, H), s(E, 2 * I // 128, H // 128)
    gu, dA, k8, ks = b(R, 2 * I), b(R, I), q(R, 2 * I), s(R, 2 * I // 128)
    X, Wg, W2, s2, dY, Wb = b(8, H), b(H, E), q(E, H, I), s(E, H // 128, I // 128), b(R, 2 * I), b(E, 2 * I, H)
    return {
        "quantize_weight": lambda **k: moe.quantize_weight(Wb, **k),
        "expert_gemm": lambda **k: moe.expert_gemm(x8, xs, W1, s1, off, **k),
        "expert_wgrad": lambda **k: moe.expert_wgrad(dY, x8, xs, off, **k),
        "swiglu": lambda **k: moe.swiglu(gu, **k),
        "swiglu_backward": lambda **k: moe.swiglu_backward(dA, k8, ks, **k),
        "moe_layer": lambda **k: moe.moe_layer(X, Wg, 2, W1, s1, W2, s2, **k),
    }


NAMES = ["quantize_weight", "expert_gemm", "expert_wgrad", "swiglu", "swiglu_backward", "moe_layer"]


def tensors(r):
    if isinstance(r, torch.Tensor):
        return [r]
    return [t for t in (r if isinstance(r, tuple) else vars(r).values()) if t is not None]


class FakeStream:
    cuda_stream = 0x7700


class FakeLib:
    def __init__(self, real):
        self.moe_layer_workspace_size = real.moe_layer_workspace_size

    def __getattr__(self, name):
        return lambda *a: 0


@pytest.mark.parametrize("name", NAMES)
def test_results_are_allocated_on_the_stream_of_the_call(name, monkeypatch):
    moe.build()
    fake, f = FakeLib(moe.lib()), calls("cpu")[name]
    on, made = [None], {}

    @contextlib.contextmanager
    def stream(s):
        before, on[0] = on[0], s
        yield
        on[0] = before

    def noting(real):
        def make(*a, **k):
            t = real(*a, **k)
            made[t.data_ptr()] = on[0]
            return t
        return make

    monkeypatch.setattr(experts, "lib", lambda: fake)
    monkeypatch.setattr(experts, "_home", lambda t, name: 0)
    monkeypatch.setattr(experts, "_arg", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(experts, "_raw_stream", lambda s, dev: 0)
    monkeypatch.setattr(experts, "_layer_workspaces", {})
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    other = FakeStream()
    got = tensors(f(stream=other))
    assert got and all(made[t.data_ptr()] is other for t in got)
    got = tensors(f())
    assert got and all(made[t.data_ptr()] is None for t in got)


# ------------------------------------------------------------------ on the GPU

@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_work_queued_on_the_current_stream_keeps_its_memory(name):
    """Copies of just freed blocks, of the sizes that the call is about to allocate, wait on the current stream while
    the call runs on another one."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    dev = torch.device("cuda")
    f = calls(dev)[name]
    want = tensors(f())
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    f(stream=other)                                    # (its workspace, its code)
    torch.cuda.synchronize()
    blocks = [torch.full((t.numel() * t.element_size(),), 0x5A, dtype=U8, device=dev) for t in want for _ in range(8)]
    copies = [torch.empty_like(t) for t in blocks]
    torch.cuda._sleep(100_000_000)                     # some 50 ms
    for t, c in zip(blocks, copies):
        c.copy_(t)
    del blocks, t
    got = tensors(f(stream=other))
    other.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(U8), b.view(U8))
    torch.cuda.synchronize()
    assert all(bool((c == 0x5A).all()) for c in copies)
