"""The norms' and the joined products' calls on a stream that is not the current one, as test_experts_streams.py does
for the experts': results and workspaces are memory of the stream that the call launches on."""
import contextlib

import pytest
import torch

import combine_moe_route_02_gb300 as moe
from combine_moe_route_02_gb300 import experts, norms
from test_experts_streams import BF16, U8, FakeStream


def calls(dev, R=96, H=256, I=128, E=3):
    """Each call with everything but `out`, as a function of the keyword arguments, and its results."""
    def b(*shape):
        return torch.ones(shape, dtype=BF16, device=dev)

    def q(*shape):
        return torch.full(shape, 0x38, dtype=U8, device=dev)        # 1.0

    def s(*shape):
        return torch.ones(shape, device=dev)

    off = torch.tensor([0, R // 2, R // 2, R], dtype=torch.int32, device=dev)
    x8, xs, W1, s1, W2, s2 = q(R, H), s(R, H // 128), q(E, 2 * I, H), s(E, 2 * I // 128, H // 128), q(E, H, I), s(E, H // 128, I // 128)
    k8, ks, X, w, rstd = q(R, 2 * I), s(R, 2 * I // 128), b(R, H), s(H), s(R)
    grads = [s(3000), b(500)]
    return {
        "expert_swiglu": lambda **k: vars(moe.expert_swiglu(x8, xs, W1, s1, off, **k)).values(),
        "expert_swiglu_backward": lambda **k: vars(moe.expert_swiglu_backward(x8, xs, W2, s2, k8, ks, off, **k)).values(),
        "rms_norm": lambda **k: vars(moe.rms_norm(X, w, residual=X, fp8=True, **k)).values(),
        "rms_norm_backward": lambda **k: vars(moe.rms_norm_backward(X, X, w, rstd, dS=X, **k)).values(),
        "grad_norm": lambda **k: [moe.grad_norm(grads, **k)],
        "clip_grad_norm": lambda **k: [moe.clip_grad_norm(grads, 1e9, **k)],
    }


NAMES = ["expert_swiglu", "expert_swiglu_backward", "rms_norm", "rms_norm_backward", "grad_norm", "clip_grad_norm"]


class FakeLib:
    def __getattr__(self, name):
        return lambda *a: 64 if name.endswith("_size") else 0


@pytest.mark.parametrize("name", NAMES)
def test_memory_is_of_the_stream_of_the_call(name, monkeypatch):
    moe.build()
    fake, f = FakeLib(), calls("cpu")[name]
    on, made = [None], []

    @contextlib.contextmanager
    def stream(s):
        before, on[0] = on[0], s
        yield
        on[0] = before

    def noting(real):
        def make(*a, **k):
            k.pop("device", None)
            made.append(on[0])
            return real(*a, **k)
        return make

    for m in (experts, norms):
        monkeypatch.setattr(m, "lib", lambda: fake)
        monkeypatch.setattr(m, "_home", lambda t, name: 0)
        monkeypatch.setattr(m, "_arg", lambda t, *a: t.data_ptr())
        monkeypatch.setattr(m, "_raw_stream", lambda s, dev: 0)
    monkeypatch.setattr(norms, "_list", lambda t, name, dev: ([x.data_ptr() for x in t], [x.numel() for x in t], [x.dtype for x in t]))
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noting(torch.empty_like))
    other = FakeStream()
    assert list(f(stream=other)) and made and all(s is other for s in made)
    del made[:]
    assert list(f()) and made and all(s is None for s in made)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_work_queued_on_the_current_stream_keeps_its_memory(name):
    """Copies of just freed blocks, of the sizes that the call is about to allocate, wait on the current stream while
    the call runs on another one."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    f = calls(torch.device("cuda"))[name]
    want = list(f())
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    f(stream=other)
    torch.cuda.synchronize()
    blocks = [torch.full((t.numel() * t.element_size(),), 0x5A, dtype=U8, device="cuda") for t in want for _ in range(8)]
    copies = [torch.empty_like(t) for t in blocks]
    torch.cuda._sleep(100_000_000)                     # some 50 ms
    for t, c in zip(blocks, copies):
        c.copy_(t)
    del blocks, t
    got = list(f(stream=other))
    other.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(U8), b.view(U8))
    torch.cuda.synchronize()
    assert all(bool((c == 0x5A).all()) for c in copies)


@pytest.mark.gpu
def test_calls_at_once_on_two_streams():
    """Nothing is shared between calls: both streams' results are those of a call alone."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    f = calls(torch.device("cuda"), R=3000, H=1024, I=512, E=3)
    want = {n: [t.clone() for t in f[n]()] for n in NAMES}
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for n in NAMES:
            for s in sides:
                got.append((n, list(f[n](stream=s))))
    torch.cuda.synchronize()
    for n, r in got:
        assert all(torch.equal(a.view(U8), b.view(U8)) for a, b in zip(r, want[n])), n
