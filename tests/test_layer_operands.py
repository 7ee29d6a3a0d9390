"""What MoeLayer and the binding's whole-layer calls refuse: tokens, outputs and weights of another type, shape or
device than the layer reads. Without a GPU (stand-ins for tensors, the library's functions record their arguments);
the weights' checks need CUDA tensors and are marked."""
import pytest
import torch

from tests.test_binding_operands import BF16, F32, U8, Fake, abi  # noqa: F401  (abi: the fixture)

T, D, E, F = 6, 256, 4, 384


class Tokens(Fake):
    def __init__(self, dtype, rows, cols=D, **kw):
        super().__init__(dtype, rows * cols, **kw)
        self.shape = (rows, cols)


@pytest.fixture
def reached(abi, monkeypatch):  # noqa: F811
    got = []
    for name in ("moe_forward", "moe_forward_host"):
        monkeypatch.setattr(abi._lib, name, lambda *a: got.append(a) or 0)
    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    return got


def layer(abi, dtype):  # noqa: F811
    """A layer whose weights and workspaces are already there."""
    from mixture_experts_routing_route_b200 import MoeLayer
    m = MoeLayer.__new__(MoeLayer)
    m.E, m.d, m.F, m.k, m.dtype = E, D, F, 2, dtype
    m.c = abi.MoeLayerC(D, E, 2, F, abi.dtype_code(dtype))
    m.workspace = m._workspace = lambda *a, **k: Fake(U8, 1 << 20)
    m._last = {}
    return m


def forward(m, dtype, **over):
    args = dict(x=Tokens(dtype, T), out=Tokens(dtype, T, address=8192), aux=Fake(F32, 1), stream=99)
    args.update(over)
    return m.forward(args.pop("x"), **args)


def forward_host(m, dtype, **over):
    args = dict(x=Tokens(dtype, T, device=-1), out=Tokens(dtype, T, device=-1), aux=Fake(F32, 1, device=-1))
    args.update(over)
    return m.forward_host(args["x"], args["out"], args["aux"], stream=99)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward(abi, reached, dtype):  # noqa: F811
    m = layer(abi, dtype)
    forward(m, dtype, x_router=Tokens(dtype, T, address=512), logit_noise=Tokens(F32, T, E, address=768))
    forward(m, dtype)
    assert len(reached) == 2 and reached[1][1] == 4096 and reached[1][3] == 8192
    structs = [args[0]._obj for args in reached]
    assert (structs[0].x_router, structs[0].logit_noise) == (512, 768) and structs[0].d == D
    assert structs[1].x_router is None and structs[1].logit_noise is None
    other = F32 if dtype is BF16 else BF16
    for wrong in (dict(x=Tokens(other, T)), dict(x=Tokens(dtype, T, D - 128)), dict(x=Tokens(dtype, 2, 3 * D)),
                  dict(x=Tokens(dtype, T, device=-1)), dict(x=Tokens(dtype, T, contiguous=False)),
                  dict(out=Tokens(other, T)), dict(out=Tokens(dtype, T - 1)), dict(out=Tokens(dtype, T, device=1)),
                  dict(aux=Fake(BF16, 1)), dict(aux=Fake(F32, 0)), dict(x_router=Tokens(other, T)),
                  dict(x_router=Tokens(dtype, T - 1)), dict(logit_noise=Tokens(BF16, T, E)),
                  dict(logit_noise=Tokens(F32, T, E - 1)), dict(logit_noise=Tokens(F32, T, E, device=-1))):
        with pytest.raises(ValueError):
            forward(m, dtype, **wrong)
    assert len(reached) == 2


def test_two_calls_at_once(abi, reached, monkeypatch):  # noqa: F811
    """A forward that begins while another one is in the library leaves it its router input."""
    m = layer(abi, BF16)
    seen = []

    def library(c, *rest):
        if not seen:
            seen.append("in")
            forward(m, BF16)
        seen.append((c._obj.x_router, c._obj.logit_noise))
        return 0

    monkeypatch.setattr(abi._lib, "moe_forward", library)
    forward(m, BF16, x_router=Tokens(BF16, T, address=512), logit_noise=Tokens(F32, T, E, address=768))
    assert seen == ["in", (None, None), (512, 768)]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_host(abi, reached, dtype):  # noqa: F811
    m = layer(abi, dtype)
    forward_host(m, dtype)
    forward_host(m, dtype, aux=None)
    assert len(reached) == 2 and reached[1][4] is None
    other = F32 if dtype is BF16 else BF16
    for wrong in (dict(x=Tokens(other, T, device=-1)), dict(x=Tokens(dtype, 2, 3 * D, device=-1)),
                  dict(x=Tokens(dtype, T, device=-1, contiguous=False)), dict(out=Tokens(other, T, device=-1)),
                  dict(out=Tokens(dtype, T - 1, device=-1)), dict(aux=Fake(torch.float64, 1, device=-1))):
        with pytest.raises(ValueError):
            forward_host(m, dtype, **wrong)
    assert len(reached) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("mxfp4", [False, True])
def test_weights_that_do_not_fit(mxfp4):
    from mixture_experts_routing_route_b200 import MoeLayer
    mk = lambda *s, dt=BF16, dev="cuda": torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
    right = dict(w_router=mk(D, E), w1=mk(E, D, F), w2=mk(E, F, D), w3=mk(E, D, F))
    MoeLayer(**right, mxfp4=mxfp4)
    wrong = [dict(w_router=mk(D, E + 1)), dict(w_router=mk(E, D)), dict(w2=mk(E, D, F)), dict(w2=mk(E - 1, F, D)),
             dict(w3=mk(E, D, F - 128)), dict(w2=mk(E, F, D, dev="cpu")), dict(w_router=mk(D, E, dt=F32))]
    if not mxfp4:
        wrong += [dict(w2=mk(E, F, D, dt=F32)), dict(w3=mk(E, D, F, dt=F32))]
    for w in wrong:
        with pytest.raises(ValueError):
            MoeLayer(**dict(right, **w), mxfp4=mxfp4)
    MoeLayer(**dict(right, w3=None), act="gelu", mxfp4=mxfp4)


@pytest.mark.gpu
@pytest.mark.parametrize("mxfp4", [False, True])
def test_calls_that_do_not_fit(mxfp4):
    """fp32 weights of a 4-bit layer: its tokens are bf16 all the same."""
    from mixture_experts_routing_route_b200 import MoeLayer
    dt = F32 if mxfp4 else BF16
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g).mul_(0.05).cuda()  # noqa: E731
    m = MoeLayer(mk(D, E).to(BF16), mk(E, D, F).to(dt), mk(E, F, D).to(dt), act="gelu", mxfp4=mxfp4)
    x = mk(T, D)
    for bad in (x, x.cpu().to(BF16), x.to(BF16).t().contiguous().t(), x.to(BF16)[:, :128].contiguous(),
                x.to(BF16).view(2, 3, D)):
        with pytest.raises(ValueError):
            m.forward(bad)
    with pytest.raises(ValueError):
        m.forward(x.to(BF16), out=torch.empty_like(x))
    with pytest.raises(ValueError):
        m.forward_host(x.cpu(), torch.empty(T, D, dtype=BF16), torch.empty(1))
    out, _ = m.forward(x.to(BF16))
    assert torch.equal(m.forward(x.to(BF16).view(T, 1, D))[0], out) and m.device_error(T) == 0
