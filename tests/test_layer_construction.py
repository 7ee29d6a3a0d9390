"""A layer with 4-bit experts is complete when it is made: its first forward may run on another stream than the one
that made it, without waiting for that one."""
import pytest
import torch

from tests.test_binding_operands import abi  # noqa: F401  (the fixture)


def test_everything_is_converted_before_the_wait(abi, monkeypatch):  # noqa: F811
    from mixture_experts_routing_route_b200 import MoeLayer
    order = []

    class Gpu(torch.Tensor):
        is_cuda = True

        def to(self, *a, **k):
            order.append("to")
            return super().to(*a, **k)

        def contiguous(self):
            order.append("contiguous")
            return super().contiguous()

    class Stream:
        def synchronize(self):
            order.append("wait")

    monkeypatch.setattr(abi, "quantize_expert_weights", lambda w: order.append("quantise") or (w, w))
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    mk = lambda *s: torch.zeros(*s, dtype=torch.bfloat16).as_subclass(Gpu)  # noqa: E731
    MoeLayer(mk(128, 4), mk(4, 128, 256), mk(4, 256, 128), bias=mk(4), act="gelu", mxfp4=True)
    assert order.count("wait") == 1 and order[-1] == "wait"
    assert order.count("quantise") == 2 and "to" in order and order.count("contiguous") >= 2


@pytest.mark.gpu
def test_first_forward_on_another_stream():
    from mixture_experts_routing_route_b200 import MoeLayer
    from tests.test_gpu_mxfp4_layer import tokens, weights
    T, d, E, F = 40, 256, 8, 256
    ws = weights(E, d, F, "gelu", 1)
    bias = torch.randn(2 * E, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    x = tokens(T, d, 3)
    make = lambda: MoeLayer(ws[0], ws[1], ws[2], bias=bias[::2], k=2, act="gelu", mxfp4=True)  # noqa: E731
    alone = make().forward(x)[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        make().forward(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # the constructor's work waits behind this
    layer = make()
    with torch.cuda.stream(side):
        out = layer.forward(x)[0]
    torch.cuda.synchronize()
    assert torch.equal(out, alone)
