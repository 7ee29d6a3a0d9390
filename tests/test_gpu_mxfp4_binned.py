"""MXFP4 layers in the binned layout: the same kernels, and the same bits, as in the dense layout."""
import pytest
import torch

from mixture_experts_routing_route_b200 import MoeLayer
from mixture_experts_routing_route_b200 import _abi as abi
from tests.test_gpu_mxfp4_layer import tokens, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d,E,k,F,act,cf", [
    (1, 512, 8, 2, 768, "swiglu", 0.0),       # decode steps: 32 rows at most, however long the bins may get
    (16, 512, 8, 2, 768, "swiglu", 0.0),
    (32, 256, 64, 1, 384, "gelu", 0.0),
    (16, 4096, 4, 2, 2048, "swiglu", 2.0),    # fixed bins, more of them than slots
    (17, 256, 8, 2, 384, "gelu", 0.0),        # 34 rows: tiles
    (300, 2048, 8, 2, 512, "swiglu", 0.0),    # few rows an expert, bins of up to 600
    (300, 2048, 2, 2, 2048, "gelu", 0.0),     # CTA pairs
    (200, 256, 8, 2, 256, "swiglu", 1.0),     # drops
])
def test_binned_is_dense(T, d, E, k, F, act, cf):
    ws = weights(E, d, F, act, T + d)
    x = tokens(T, d, F)
    outs, launches = [], []
    for binned in (False, True):
        layer = MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=k, act=act, capacity_factor=cf, binned=binned, mxfp4=True)
        n = abi.moe_kernel_launches()
        out, aux = layer.forward(x)
        launches.append(abi.moe_kernel_launches() - n)
        assert layer.device_error(T) == 0
        outs.append((out, aux))
        assert torch.equal(layer.forward(x)[0], out)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert launches[0] == launches[1]
