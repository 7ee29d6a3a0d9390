"""One MoeLayer called on several streams at once: every stream has a workspace of its own, and so has every
graph that its calls are captured into (a workspace in use by two calls at the same time gives wrong output without an error)."""
import contextlib

import pytest
import torch

from tests.test_binding_operands import BF16, F32, U8, Fake, abi  # noqa: F401  (abi: the fixture)
from tests.test_layer_operands import Tokens, layer

T = 6


@pytest.fixture
def cuda(abi, monkeypatch):  # noqa: F811
    """The current stream's handle, whether it is being captured, and the workspaces the library was called with."""
    from mixture_experts_routing_route_b200 import layer as module
    state = dict(stream=11, capture=0, made=0, init=[], used=[])

    def empty(n, dtype, device):
        state["made"] += 1
        return Fake(U8, n, address=1 << (20 + state["made"]))

    @contextlib.contextmanager
    def under(stream):
        before, state["stream"] = state["stream"], state["stream"] if stream is None else stream
        yield
        state["stream"] = before

    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    monkeypatch.setattr(abi, "_raw_stream", lambda device: state["stream"])
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capture"] != 0)
    monkeypatch.setattr(abi, "_capture_id", lambda handle: state["capture"] if handle == 11 else 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(module.torch, "empty", empty)
    monkeypatch.setattr(abi._lib, "moe_workspace_init", lambda ws, n, s: state["init"].append((ws, s)) or 0)
    monkeypatch.setattr(abi._lib, "moe_forward", lambda *a: state["used"].append((a[5], a[7])) or 0)
    monkeypatch.setattr(abi._lib, "moe_forward_host", lambda *a: state["used"].append((a[5], a[7])) or 0)
    return state


def plain(abi):  # noqa: F811
    m = layer(abi, BF16)
    del m.workspace, m._workspace
    m._ws, m._last, m.w1 = {}, {}, Fake(BF16, 1)
    return m


def forward(m, state, **kw):
    m.forward(Tokens(BF16, T), out=Tokens(BF16, T), aux=Fake(F32, 1), **kw)
    return state["used"][-1]


def test_a_workspace_a_stream(abi, cuda):  # noqa: F811
    m = plain(abi)
    first, on = forward(m, cuda)
    assert on == 11 and cuda["init"] == [(first, 11)]
    assert forward(m, cuda) == (first, 11)
    cuda["stream"] = 22
    second, on = forward(m, cuda)
    assert on == 22 and second != first and cuda["init"][-1] == (second, 22)  # initialised where it is used
    assert m.workspace(T).data_ptr() == second  # the last call's
    assert forward(m, cuda, stream=11) == (first, 11)
    assert m.workspace(T).data_ptr() == first
    third, on = forward(m, cuda, stream=33)
    assert on == 33 and third not in (first, second) and cuda["init"][-1] == (third, 33) and cuda["stream"] == 22
    assert forward(m, cuda) == (second, 22)
    assert m.workspace(T, stream=33).data_ptr() == third and m.workspace(T).data_ptr() == second
    assert forward(m, cuda, stream=0)[1] == 0 and len(cuda["init"]) == 4


def test_host_buffers_and_slots(abi, cuda):  # noqa: F811
    m = plain(abi)

    def host(**kw):
        m.forward_host(Tokens(BF16, T, device=-1), Tokens(BF16, T, device=-1), None, **kw)
        return cuda["used"][-1]

    seen = {host(slot=s, stream=st)[0] for s in (0, 1) for st in (11, 22)} | {forward(m, cuda)[0]}
    assert len(seen) == 5
    assert m.workspace(T, host_io=True, slot=1).data_ptr() == host(slot=1, stream=22)[0]


def test_a_workspace_a_graph(abi, cuda):  # noqa: F811
    m = plain(abi)
    warm, _ = forward(m, cuda)
    seen = [warm]
    for capture in (7, 8):
        cuda["capture"] = capture
        # in stream order within a graph: one for both calls
        one, two = forward(m, cuda)[0], forward(m, cuda, stream=11)[0]
        assert one == two and one not in seen and cuda["init"][-1] == (one, 11)
        seen.append(one)
        # a stream that is not part of the capture
        away, _ = forward(m, cuda, stream=22)
        assert away not in seen and (away, 22) in cuda["init"]
        forward(m, cuda)
        assert m.workspace(T).data_ptr() == one
    assert len(cuda["init"]) == 4
    cuda["capture"] = 0
    assert forward(m, cuda) == (warm, 11) and forward(m, cuda, stream=22) == (away, 22)
    # captured before any other call: what the graph initialises is not for later calls
    n = plain(abi)
    cuda["capture"] = 9
    captured, _ = forward(n, cuda)
    cuda["capture"] = 0
    after, _ = forward(n, cuda)
    assert after != captured and (after, 11) in cuda["init"]


# ------------------------------------------------------------------------- GPU
def gpu_layer(F_, act="swiglu", mxfp4=True, d=512):
    from mixture_experts_routing_route_b200 import MoeLayer
    from tests.test_gpu_mxfp4_layer import weights
    ws = weights(8, d, F_, act, F_)
    return MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=2, act=act, mxfp4=mxfp4)


def gpu_tokens(n, seed, d=512):
    from tests.test_gpu_mxfp4_layer import tokens
    return tokens(n, d, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("mxfp4", [True, False])
@pytest.mark.parametrize("T_", [2, 16, 300])
def test_one_layer_on_two_streams(T_, mxfp4):
    m = gpu_layer(2048, mxfp4=mxfp4)
    xs = [gpu_tokens(T_, s) for s in (3, 4)]
    alone = [m.forward(x)[0].clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for i in range(20):
        for j, (x, st) in enumerate(zip(xs, streams)):
            if i % 2:
                with torch.cuda.stream(st):
                    got[j].append(m.forward(x)[0])
            else:
                out = torch.empty_like(alone[j])
                got[j].append(m.forward(x, out=out, stream=st if i % 4 else st.cuda_stream)[0])
    torch.cuda.synchronize()
    for j, st in enumerate(streams):
        assert m.device_error(T_, stream=st) == 0
        assert all(torch.equal(o, alone[j]) for o in got[j])
        assert m.workspace(T_, stream=st).data_ptr() == m.workspace(T_, stream=st.cuda_stream).data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("warm", [False, True])
@pytest.mark.parametrize("T_", [3, 200])
def test_two_graphs_of_one_layer_at_once(T_, warm):
    """Captured on the same stream, replayed on two, beside a call on a third."""
    m = gpu_layer(1024)
    xs = [gpu_tokens(T_, s) for s in (5, 6, 7)]
    other = gpu_layer(1024)
    alone = [other.forward(x)[0].clone() for x in xs]
    torch.cuda.synchronize()
    if warm:
        m.forward(xs[0])
        torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs[:2]:
        outs.append(torch.zeros_like(alone[0]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            m.forward(x, out=outs[-1])
            m.forward(x, out=outs[-1])
    torch.cuda.synchronize()
    graphs[1].replay()
    torch.cuda.synchronize()
    # what the last captured call left can be read
    assert int(m.views(T_)["seg_offsets"][-1]) == 2 * T_ and m.device_error(T_) == 0
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [m.forward(xs[2])[0] for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, a) for o, a in zip(outs, alone))
        assert all(torch.equal(o, alone[2]) for o in eager)
        assert m.device_error(T_) == 0
