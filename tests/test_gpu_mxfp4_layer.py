"""MoeLayer with MXFP4 experts: the whole forward against float64 on the values
the codes stand for, in the dense and the binned layout, with drops, at decode
and at prefill sizes; and its stages one by one give the same bits."""
import numpy as np
import pytest
import torch

from mixture_experts_routing_route_b200 import MoeLayer
from mixture_experts_routing_route_b200 import _abi as abi
from tests import mx_reference as R
from tests.gpu_helpers import new_ws, np32, npi

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weights(E, d, F, act, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: (0.05 * torch.randn(*s, generator=g)).to(torch.bfloat16).to(DEV)  # noqa: E731
    return mk(d, E), mk(E, d, F), mk(E, F, d), mk(E, d, F) if act == "swiglu" else None


def tokens(T, d, seed):
    return torch.randn(T, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def reference(x, layer, ws, views):
    """The layer's output in float64 from its own routing, every quantisation as the format defines it."""
    wg, w1, w2, w3 = ws
    deq = lambda w: R.values(*R.quantise(np32(w).transpose(0, 2, 1))).transpose(0, 2, 1)  # noqa: E731
    q1, q2, q3 = deq(w1), deq(w2), None if w3 is None else deq(w3)
    T, k = x.shape[0], layer.k
    idx, tw = npi(views["topk_idx"]), np32(views["topk_w"]).astype(np.float64)
    kept = npi(views["slot_to_row"]).reshape(T, k) >= 0
    xq = R.values(*R.quantise(np32(x)))
    out = np.zeros((T, layer.d))
    for e in range(layer.E):
        t, j = np.nonzero((idx == e) & kept)
        if len(t) == 0:
            continue
        g = xq[t] @ q1[e]
        h = R.gelu(g) if w3 is None else R.silu(g) * (xq[t] @ q3[e])
        y = R.values(*R.quantise(h)) @ q2[e]
        np.add.at(out, t, tw[t, j][:, None] * y)
    return out


CASES = [
    (1, 512, 8, 2, 768, "swiglu", 0.0, False),      # a decode step: the weight stream
    (13, 256, 16, 2, 384, "gelu", 0.0, False),
    (16, 1024, 4, 2, 512, "swiglu", 0.0, True),     # binned, dynamic capacity: more than 32 rows of bins
    (3, 256, 2, 1, 256, "swiglu", 1.0, True),       # binned, few rows
    (300, 384, 8, 2, 640, "gelu", 1.0, False),      # drops
    (700, 256, 5, 3, 512, "swiglu", 0.0, False),
    (257, 512, 64, 4, 256, "swiglu", 1.25, True),
    (1100, 2048, 2, 2, 512, "swiglu", 0.0, False),  # CTA pairs up, single CTAs down
    (600, 2048, 4, 2, 2048, "gelu", 2.0, True),     # CTA pairs, bins partly full
]


@pytest.mark.parametrize("T,d,E,k,F,act,cf,binned", CASES)
def test_layer(T, d, E, k, F, act, cf, binned):
    ws = weights(E, d, F, act, d + F)
    layer = MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=k, act=act, capacity_factor=cf, binned=binned, mxfp4=True)
    x = tokens(T, d, T)
    out, aux = layer.forward(x)
    torch.cuda.synchronize()
    assert layer.device_error(T) == 0
    views = layer.views(T)
    ref = reference(x, layer, ws, views)
    err = np32(out) - ref
    # y is rounded to bf16 and so is the sum of k of them (2^-8 each, the second of a sum of up to k rows);
    # fp32 sums move a few codes of h by a step, which the third 2^-8 stands for
    assert np.linalg.norm(err) <= 3 * 2.0 ** -8 * np.linalg.norm(ref)
    dropped = (npi(views["slot_to_row"]).reshape(T, k) < 0).all(1)
    assert np.all(np32(out)[dropped] == 0.0)
    # the same call again, on the same workspace: the same bits
    again, _ = layer.forward(x)
    assert torch.equal(again, out)


@pytest.mark.parametrize("T", [1, 200])
def test_layer_is_its_stages(T):
    d, E, k, F = 512, 8, 2, 640
    ws = weights(E, d, F, "swiglu", 3)
    layer = MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=k, act="swiglu", mxfp4=True)
    x = tokens(T, d, 4)
    out, _ = layer.forward(x)
    v = layer.views(T)
    rows = T * k
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    w = new_ws(abi.moe_expert_ffn_mxfp4_workspace_size(rows, d, F, E))
    xc, xs = u8(rows * d // 2), u8(abi.moe_mxfp4_row_scales_size(rows, E, d))
    hc, hs = u8(rows * F // 2), u8(abi.moe_mxfp4_row_scales_size(rows, E, F))
    y, o = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV), torch.empty_like(out)
    abi.moe_gather_mxfp4(x, T, d, k, v["slot_to_row"], v["seg_offsets"], E, rows, xc, xs, w)
    abi.moe_expert_ffn_mxfp4(xc, xs, layer.w1, layer.scales[0], layer.w3, layer.scales[1], layer.w2, layer.scales[2],
                             abi.MOE_ACT_SWIGLU, rows, d, F, E, v["seg_offsets"], hc, hs, y, w)
    abi.moe_combine(y, v["topk_w"], v["slot_to_row"], T, d, k, rows, o, w)
    assert abi.moe_get_device_error(w) == 0
    assert torch.equal(v["x_perm"].reshape(-1), xc) and torch.equal(v["h"].reshape(-1), hc)
    assert torch.equal(v["y_perm"], y) and torch.equal(o, out)
    # the views read back as values: what the stages' own buffers hold
    for name, K, codes, scales in (("x_perm", d, xc, xs), ("h", F, hc, hs)):
        got, ref = torch.empty(rows, K, device=DEV), torch.empty(rows, K, device=DEV)
        abi.moe_mxfp4_dequantize_rows(v[name], v[name + "_scales"], v["seg_offsets"], E, rows, K, got, w)
        abi.moe_mxfp4_dequantize_rows(codes, scales, v["seg_offsets"], E, rows, K, ref, w)
        assert torch.equal(got, ref) and torch.isfinite(ref).all()


def test_layer_in_a_graph_beside_the_bf16_layer():
    """One graph with both layers on two workspaces, replayed with new tokens."""
    T, d, E, k, F = 24, 256, 8, 2, 256
    ws = weights(E, d, F, "swiglu", 5)
    q = MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=k, mxfp4=True)
    b = MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=k)
    x = tokens(T, d, 6)
    outs = [torch.empty(T, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for layer, o in zip((q, b), outs):
        layer.forward(x, out=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer, o in zip((q, b), outs):
            layer.forward(x, out=o)
    x.copy_(tokens(T, d, 7))
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for layer, g in zip((q, b), got):
        assert torch.equal(layer.forward(x)[0], g)
        assert layer.device_error(T) == 0


@pytest.mark.parametrize("T", [2, 300])
def test_two_layers_on_two_streams(T):
    d, E, k, F = 1024, 8, 2, 1024
    layers = []
    for seed in (1, 2):
        ws = weights(E, d, F, "swiglu", seed)
        layers.append(MoeLayer(ws[0], ws[1], ws[2], w3=ws[3], k=k, mxfp4=True))
    xs = [tokens(T, d, s) for s in (3, 4)]
    alone = [layer.forward(x)[0].clone() for layer, x in zip(layers, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(20):
        for i, (layer, x, st) in enumerate(zip(layers, xs, streams)):
            with torch.cuda.stream(st):
                got[i].append(layer.forward(x)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert layers[i].device_error(T) == 0
        assert all(torch.equal(o, alone[i]) for o in got[i])


@pytest.mark.parametrize("T", [5, 150])
def test_host_buffers(T):
    d, E, k, F = 256, 8, 2, 384
    ws = weights(E, d, F, "gelu", 9)
    layer = MoeLayer(ws[0], ws[1], ws[2], k=k, act="gelu", mxfp4=True)
    x = tokens(T, d, 2)
    out, aux = layer.forward(x)
    xh, oh, ah = x.cpu().pin_memory(), torch.empty(T, d, dtype=torch.bfloat16).pin_memory(), torch.empty(1).pin_memory()
    layer.forward_host(xh, oh, ah)
    torch.cuda.synchronize()
    assert torch.equal(oh, out.cpu()) and torch.equal(ah, aux.cpu())


def test_no_tokens():
    ws = weights(4, 128, 128, "gelu", 1)
    layer = MoeLayer(ws[0], ws[1], ws[2], k=2, act="gelu", mxfp4=True)
    out, _ = layer.forward(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV))
    assert out.shape == (0, 128) and layer.device_error(0) == 0


def test_mxfp4_needs_a_bf16_router():
    ws = weights(4, 128, 128, "gelu", 1)
    with pytest.raises(ValueError):
        MoeLayer(ws[0].float(), ws[1], ws[2], k=1, act="gelu", mxfp4=True)
