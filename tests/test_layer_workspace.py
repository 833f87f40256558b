"""moe_layer's own workspace and CUDA graphs.  The kernel wants its counters at zero, so a buffer whose clearing
has only been recorded is fit for that graph alone, and a buffer that a graph holds is not one to be freed or
shared by later calls.  On the CPU the library and the streams are stand-ins."""
import contextlib
import ctypes

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
from combine_moe_route_02_gb300 import experts

DIMS = dict(H=256, I=128, E=8, K=2)


def counters(E, I):
    return 256 + 4 * (E + 128) * (I // 128)


class FakeStream:
    cuda_stream = 0x7700


class FakeLib:
    """Notes the workspace of each moe_layer call, and whether its counters are zero."""

    def __init__(self, real):
        self.moe_layer_workspace_size = real.moe_layer_workspace_size
        self.calls = []

    def moe_layer(self, *a):
        I, E = a[11], a[12]
        ws, size = a[19], a[20]
        ws = getattr(ws, "value", ws)
        clear = not any(ctypes.string_at(ws, counters(E, I)))
        self.calls.append((ws, size, clear))
        return 0


@pytest.fixture
def host(monkeypatch):
    moe.build()
    fake = FakeLib(moe.lib())
    fake.capturing = False
    kept = []                            # every buffer stays allocated, so that addresses tell buffers apart
    real_empty, real_zeros = torch.empty, torch.zeros

    def empty(*a, **k):
        t = real_empty(*a, **k)
        if t.dtype == torch.uint8:
            t.fill_(0xA5)
            kept.append(t)
        return t

    def zeros(*a, **k):
        kept.append(real_zeros(*a, **k))
        return kept[-1]

    monkeypatch.setattr(experts, "lib", lambda: fake)
    monkeypatch.setattr(experts, "_home", lambda t, name: 0)
    monkeypatch.setattr(experts, "_arg", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(experts, "_layer_workspaces", {})
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: fake.capturing)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", zeros)
    return fake


def layer_on_host(fake, N):
    H, I, E, K = DIMS["H"], DIMS["I"], DIMS["E"], DIMS["K"]
    u8 = torch.uint8
    moe.moe_layer(torch.ones((N, H), dtype=torch.bfloat16), torch.ones((H, E), dtype=torch.bfloat16), K,
                  torch.ones((E, 2 * I, H), dtype=u8), torch.ones((E, 2 * I // 128, H // 128)),
                  torch.ones((E, H, I), dtype=u8), torch.ones((E, H // 128, I // 128)), stream=FakeStream())
    return fake.calls[-1]


def test_a_captured_call_has_a_workspace_of_its_own(host):
    host.capturing = True
    first, second = layer_on_host(host, 4), layer_on_host(host, 1)
    assert first[2] and second[2]        # cleared within the capture
    assert first[0] != second[0]
    host.capturing = False
    plain = layer_on_host(host, 1)
    assert plain[2] and plain[0] not in (first[0], second[0])   # what no replay has cleared yet is in no cache
    host.capturing = True
    third = layer_on_host(host, 1)
    assert third[2] and third[0] not in (first[0], second[0], plain[0])
    host.capturing = False
    assert layer_on_host(host, 1)[0] == plain[0]                # calls outside a capture share one


def test_a_workspace_asked_for_within_a_capture_is_not_kept(host):
    a = experts.layer_workspace(4, device="cpu", stream=FakeStream(), **DIMS)
    host.capturing = True
    b = experts.layer_workspace(4, device="cpu", stream=FakeStream(), **DIMS)
    c = experts.layer_workspace(4, device="cpu", stream=FakeStream(), **DIMS)
    assert len({t.data_ptr() for t in (a, b, c)}) == 3
    for t in (b, c):
        assert t.numel() >= experts.layer_workspace_size(4, **DIMS) and not t[:counters(8, 128)].any()
    host.capturing = False
    assert experts.layer_workspace(4, device="cpu", stream=FakeStream(), **DIMS) is a


# ------------------------------------------------------------------ on the GPU

@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    return torch.device("cuda")


def normal(shape, seed, dev, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(dev)


def inputs(dev, N, H, I, E):
    return (normal((N, H), 1, dev), normal((H, E), 2, dev, H ** -0.5),
            *ref.encode_weight(normal((E, 2 * I, H), 3, dev, H ** -0.5), "ue8m0"),
            *ref.encode_weight(normal((E, H, I), 4, dev, I ** -0.5), "ue8m0"))


def capture(t, n, K, st, **where):
    """A graph of one call on the first n tokens, and its outputs."""
    x = t[0][:n].contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, **where):
        r = moe.moe_layer(x, t[1], K, *t[2:], status=st)
    return g, r


def same(r, want):
    return (torch.equal(r.out.view(torch.int16), want.out.view(torch.int16)) and torch.equal(r.topk_idx, want.topk_idx)
            and torch.equal(r.topk_w, want.topk_w) and not r.out.isnan().any())


def spoil(r):
    r.out.fill_(float("nan"))
    r.topk_idx.fill_(-1)
    r.topk_w.fill_(float("nan"))


def wants(t, sizes, K, dev):
    """The same calls, each on a cleared buffer of its own."""
    H, E, I = t[0].shape[1], t[2].shape[0], t[4].shape[2]
    out = {}
    for n in sizes:
        ws = torch.zeros(moe.layer_workspace_size(n, H, I, E, K), dtype=torch.uint8, device=dev)
        out[n] = moe.moe_layer(t[0][:n].contiguous(), t[1], K, *t[2:], workspace=ws)
    torch.cuda.synchronize()
    return out


@pytest.mark.gpu
def test_graphs_of_several_sizes_without_a_call_before(dev, monkeypatch):
    """Captured one after the other on torch's shared capture stream, replayed in another order, with every
    buffer dirty before the replay."""
    H, I, E, K = 384, 256, 24, 4         # (sizes of this test alone: no call has cached a buffer for them)
    t = inputs(dev, 32, H, I, E)
    want = wants(t, (1, 7, 32), K, dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    held, real = [], experts.layer_workspace
    monkeypatch.setattr(experts, "layer_workspace", lambda *a, **k: held.append(real(*a, **k)) or held[-1])
    graphs = {n: capture(t, n, K, st) for n in (7, 1, 32)}
    assert len({ws.data_ptr() for ws in held}) == 3
    for order in ((32, 1, 7), (1, 7, 32), (7, 7, 1)):
        for n in order:
            g, r = graphs[n]
            spoil(r)
            for ws in held:
                ws.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            assert st.item() == 0, moe.status_string(st.item())
            assert same(r, want[n]), n


@pytest.mark.gpu
def test_a_call_on_the_capture_stream_before_the_replay(dev):
    H, I, E, K = 384, 128, 24, 3
    t = inputs(dev, 16, H, I, E)
    want = wants(t, (5, 16), K, dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g, r = capture(t, 5, K, st, stream=s)
    with torch.cuda.stream(s):
        plain = moe.moe_layer(t[0], t[1], K, *t[2:], status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and same(plain, want[16])
    spoil(r)
    g.replay()
    torch.cuda.synchronize()
    assert st.item() == 0 and same(r, want[5])


@pytest.mark.gpu
def test_a_graph_outlives_a_later_call_that_needs_more(dev):
    """Warm-up and capture for one token, then a call for 64 tokens on the same stream, whose buffer is larger;
    what the allocator hands out afterwards is not what the graph writes to."""
    H, I, E, K = 384, 256, 12, 4
    t = inputs(dev, 64, H, I, E)
    want = wants(t, (1, 64), K, dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = t[0][:1].contiguous()
    with torch.cuda.stream(s):
        moe.moe_layer(x, t[1], K, *t[2:], status=st)
    g, r = capture(t, 1, K, st, stream=s)
    with torch.cuda.stream(s):
        big = moe.moe_layer(t[0], t[1], K, *t[2:], status=st)
        over = [torch.full((n,), 0x5A, dtype=torch.uint8, device=dev) for n in (1 << 16, 1 << 18, 1 << 20, 1 << 21) * 8]
    torch.cuda.synchronize()
    assert same(big, want[64])
    for _ in range(3):
        spoil(r)
        g.replay()
        torch.cuda.synchronize()
        assert st.item() == 0, moe.status_string(st.item())
        assert same(r, want[1])
    assert all(bool((o == 0x5A).all()) for o in over)
