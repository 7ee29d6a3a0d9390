"""Refusals and size arithmetic of the row movement's backward passes and of the
MXFP4 entry points, without a GPU: every call here fails a host check, so
nothing is launched."""
import ctypes

import numpy as np
import pytest

import __graft_entry__
from tests import mx_reference as R

OK_PTR, BIG = 16, 1 << 40
NULL, INVALID, UNSUPPORTED, WORKSPACE, ALIGN = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def abi():
    __graft_entry__.build()
    from mixture_experts_routing_route_b200 import _abi
    return _abi


@pytest.fixture(autouse=True)
def nothing_launched(abi):
    n0 = abi.moe_kernel_launches()
    yield
    assert abi.moe_kernel_launches() == n0


def call(fn, names, defaults, **over):
    assert set(over) <= set(names), over
    return fn(*[over.get(n, defaults[n]) for n in names])


def ptrs(names):
    return {n: OK_PTR for n in names}


def combine_backward(abi, **over):
    names = ["d_out", "y", "w", "s2r", "dt", "T", "d", "k", "rows", "dy", "dw", "ws", "bytes", "stream"]
    return call(abi._lib.moe_combine_backward, names, dict(ptrs(names), dt=abi.MOE_BF16, T=8, d=128, k=2, rows=16,
                                                           bytes=256, stream=None), **over)


def gather_backward(abi, **over):
    names = ["dxp", "s2r", "dx_in", "dt", "T", "d", "k", "rows", "dx", "ws", "bytes", "stream"]
    return call(abi._lib.moe_gather_backward, names, dict(ptrs(names), dt=abi.MOE_BF16, T=8, d=128, k=2, rows=16,
                                                          bytes=256, stream=None), **over)


@pytest.mark.parametrize("f", [combine_backward, gather_backward])
def test_backward_refusals(abi, f):
    assert f(abi, ws=None) == NULL
    assert f(abi, s2r=None) == NULL
    assert f(abi, ws=8) == ALIGN
    assert f(abi, s2r=20) == ALIGN
    assert f(abi, bytes=255) == WORKSPACE
    assert f(abi, T=-1) == INVALID and f(abi, d=0) == INVALID
    assert f(abi, k=0) == INVALID and f(abi, k=9) == INVALID
    assert f(abi, dt=7) == INVALID
    assert f(abi, rows=-1) == INVALID and f(abi, rows=1 << 31) == INVALID
    assert f(abi, T=1 << 30, k=4) == INVALID              # T * k past 31 bits
    assert f(abi, d=96) == UNSUPPORTED and f(abi, dt=abi.MOE_F32, d=66) == UNSUPPORTED


def test_combine_backward_refusals(abi):
    assert combine_backward(abi, d_out=None) == NULL
    assert combine_backward(abi, w=None) == NULL           # d_y_perm wants the weights
    assert combine_backward(abi, y=None) == NULL           # d_topk_w wants the rows
    for p in ("d_out", "y", "w", "dy", "dw"):
        assert combine_backward(abi, **{p: 24}) == ALIGN


def test_gather_backward_refusals(abi):
    assert gather_backward(abi, dxp=None) == NULL and gather_backward(abi, dx=None) == NULL
    for p in ("dxp", "dx_in", "dx"):
        assert gather_backward(abi, **{p: 24}) == ALIGN


def weights_call(abi, back, **over):
    names = ["w", "dt", "E", "K", "N", "codes", "scales", "stream"]
    d = dict(ptrs(names), dt=abi.MOE_BF16, E=2, K=128, N=256, stream=None)
    d.update(over)
    if back:
        return abi._lib.moe_mxfp4_dequantize_weights(d["codes"], d["scales"], d["dt"], d["E"], d["K"], d["N"], d["w"], None)
    return abi._lib.moe_mxfp4_quantize_weights(*[d[n] for n in names])


@pytest.mark.parametrize("back", [False, True])
def test_weight_refusals(abi, back):
    for p in ("w", "codes", "scales"):
        assert weights_call(abi, back, **{p: None}) == NULL
        assert weights_call(abi, back, **{p: 8}) == ALIGN
    assert weights_call(abi, back, E=0) == INVALID and weights_call(abi, back, E=257) == INVALID
    assert weights_call(abi, back, K=0) == INVALID and weights_call(abi, back, N=-128) == INVALID
    assert weights_call(abi, back, dt=3) == INVALID
    assert weights_call(abi, back, K=96) == UNSUPPORTED and weights_call(abi, back, N=192) == UNSUPPORTED
    assert weights_call(abi, back, K=128 * 65536) == UNSUPPORTED


def gather_mxfp4(abi, **over):
    names = ["x", "dt", "T", "d", "k", "s2r", "seg", "E", "rows", "codes", "scales", "ws", "bytes", "stream"]
    return call(abi._lib.moe_gather_mxfp4, names, dict(ptrs(names), dt=abi.MOE_BF16, T=8, d=128, k=2, E=4, rows=16,
                                                       bytes=256, stream=None), **over)


def dequantize_rows(abi, **over):
    names = ["codes", "scales", "seg", "E", "rows", "d", "dt", "out", "ws", "bytes", "stream"]
    return call(abi._lib.moe_mxfp4_dequantize_rows, names, dict(ptrs(names), dt=abi.MOE_F32, d=128, E=4, rows=16,
                                                                bytes=256, stream=None), **over)


def test_row_refusals(abi):
    for f, pointers in ((gather_mxfp4, ("x", "s2r", "seg", "codes", "scales", "ws")),
                        (dequantize_rows, ("codes", "scales", "seg", "out", "ws"))):
        for p in pointers:
            assert f(abi, **{p: None}) == NULL
            assert f(abi, **{p: 4}) == ALIGN
        assert f(abi, bytes=0) == WORKSPACE
        assert f(abi, E=0) == INVALID and f(abi, E=300) == INVALID
        assert f(abi, rows=-1) == INVALID and f(abi, rows=1 << 31) == INVALID
        assert f(abi, d=64) == UNSUPPORTED and f(abi, dt=abi.MOE_F32, d=132) == UNSUPPORTED
        assert f(abi, dt=2) == INVALID
    assert gather_mxfp4(abi, k=5) == INVALID  # k > E


def ffn(abi, **over):
    names = ["xc", "xs", "w1", "s1", "w3", "s3", "w2", "s2", "act", "rows", "d", "F", "E", "seg", "hc", "hs", "y", "ws",
             "bytes", "stream"]
    return call(abi._lib.moe_expert_ffn_mxfp4, names,
                dict(ptrs(names), act=abi.MOE_ACT_SWIGLU, rows=64, d=128, F=256, E=4, bytes=BIG, stream=None), **over)


def test_ffn_refusals(abi):
    for p in ("xc", "xs", "w1", "s1", "w3", "s3", "w2", "s2", "seg", "hc", "hs", "y", "ws"):
        assert ffn(abi, **{p: None}) == NULL
        assert ffn(abi, **{p: 8}) == ALIGN
    assert ffn(abi, act=2) == INVALID and ffn(abi, E=0) == INVALID and ffn(abi, E=257) == INVALID
    assert ffn(abi, rows=-1) == INVALID and ffn(abi, rows=1 << 31) == INVALID
    assert ffn(abi, d=64) == UNSUPPORTED and ffn(abi, F=200) == UNSUPPORTED
    assert ffn(abi, d=1 << 21) == UNSUPPORTED               # counts past 32 bits
    assert ffn(abi, rows=(1 << 31) - 2, d=1 << 20) == UNSUPPORTED
    n = abi.moe_expert_ffn_mxfp4_workspace_size(64, 128, 256, 4)
    few = abi.moe_expert_ffn_mxfp4_workspace_size(32, 128, 256, 4)
    assert n == 256 and few > 1 << 20                       # a decode step keeps partial sums
    assert ffn(abi, bytes=n - 1) == WORKSPACE
    assert ffn(abi, rows=32, bytes=few - 1) == WORKSPACE


def layer(abi, **over):
    d = dict(d=256, E=8, k=2, F=128, dtype=abi.MOE_BF16, act=abi.MOE_ACT_SWIGLU, cf=0.0, flags=abi.MOE_LAYER_MXFP4,
             w1=16, w3=16, w2=16, s1=16, s3=16, s2=16)
    d.update(over)
    L = abi.MoeLayerC(d["d"], d["E"], d["k"], d["F"], d["dtype"], d["act"], d["cf"], 16, None, d["w1"], d["w3"], d["w2"],
                      d["flags"], None, None, 1.0, d["s1"], d["s3"], d["s2"])
    return L, abi._lib.moe_forward(ctypes.byref(L), 16, 4, 16, None, 16, over.get("bytes", 0), None, None)


def test_layer_refusals(abi):
    assert layer(abi)[1] == WORKSPACE                        # everything else is right
    for p in ("s1", "s3", "s2"):
        assert layer(abi, **{p: None})[1] == NULL
        assert layer(abi, **{p: 8})[1] == ALIGN
    assert layer(abi, s3=None, w3=None, act=abi.MOE_ACT_GELU)[1] == WORKSPACE
    assert layer(abi, dtype=abi.MOE_F32)[1] == UNSUPPORTED
    assert layer(abi, flags=abi.MOE_LAYER_MXFP4 | abi.MOE_LAYER_GATHER_IN_GEMM)[1] == UNSUPPORTED
    assert layer(abi, k=1, flags=abi.MOE_LAYER_MXFP4 | abi.MOE_LAYER_COMBINE_IN_GEMM)[1] == UNSUPPORTED
    assert layer(abi, flags=64)[1] == INVALID
    # without the flag the scales are not looked at
    assert layer(abi, flags=0, s1=None, s3=None, s2=None)[1] == WORKSPACE
    # codes are a quarter of bf16
    plain, _ = layer(abi, d=4096, F=14336, flags=0)
    quant, _ = layer(abi, d=4096, F=14336)
    assert abi.moe_forward_workspace_size(quant, 4096) < abi.moe_forward_workspace_size(plain, 4096) / 2


def test_scale_sizes(abi):
    assert abi.moe_mxfp4_weight_scales_size(3, 256, 384) == 3 * 256 * 384 // 32
    assert abi.moe_mxfp4_row_scales_size(0, 4, 256) == 4 * 2 * 512
    assert abi.moe_mxfp4_row_scales_size(300, 4, 256) == (2 + 4) * 2 * 512
    assert abi.moe_mxfp4_row_scales_size(-1, 4, 256) == 0 and abi.moe_mxfp4_weight_scales_size(0, 1, 1) == 0


@pytest.mark.parametrize("seed", range(20))
def test_every_row_has_a_scale_of_its_own(abi, seed):
    """Row groups of any segments lie inside the buffer and never share a byte."""
    rng = np.random.default_rng(seed)
    E = int(rng.integers(1, 257))
    counts = rng.integers(0, 4, E) * rng.integers(0, 300, E)
    seg = np.concatenate(([0], np.cumsum(counts)))
    K = 128 * int(rng.integers(1, 4))
    group, row = R.row_groups(seg)
    at = R.scale_at(group[:, None], K // 128, row[:, None], np.arange(K // 32)[None, :]).reshape(-1)
    assert len(np.unique(at)) == at.size
    assert at.size == 0 or at.max() < abi.moe_mxfp4_row_scales_size(int(seg[-1]), E, K)


def test_reference_quantisation():
    """The definition on values worked out by hand."""
    v = np.zeros((1, 32))
    v[0, :12] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, -5.01, 7.9, -0.0]
    codes, scales = R.quantise(v)
    assert scales[0, 0] == 127
    assert codes[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 15, 7, 8]
    assert R.values(codes, scales)[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    for top, byte in ((0.0, 0), (8.0, 128), (1.0, 125), (2.0 ** -126, 0), (2.0 ** -149, 0), (3.4e38, 252), (np.inf, 255),
                      (np.nan, 255)):
        v = np.zeros((1, 32))
        v[0, 3] = top
        assert R.quantise(v)[1][0, 0] == byte
    assert np.array_equal(R.unpack(R.pack(codes)), codes)


def test_binding_refuses_host_tensors(abi):
    """A host address would fault on the GPU: the binding refuses it before the library is called."""
    import torch
    f, i, u = torch.zeros(8, 128), torch.zeros(16, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    w = torch.zeros(1, 128, 128)
    for call_ in (
        lambda: abi.moe_combine_backward(f, f, f, i, 8, 128, 2, 16, f, f, u),
        lambda: abi.moe_gather_backward(f, i, None, 8, 128, 2, 16, f, u),
        lambda: abi.moe_mxfp4_quantize_weights(w, 1, 128, 128, u, u),
        lambda: abi.moe_mxfp4_dequantize_weights(u, u, 1, 128, 128, w),
        lambda: abi.quantize_expert_weights(w),
        lambda: abi.moe_gather_mxfp4(f, 8, 128, 2, i, i, 4, 16, u, u, u),
        lambda: abi.moe_mxfp4_dequantize_rows(u, u, i, 4, 16, 128, f, u),
        lambda: abi.moe_expert_ffn_mxfp4(u, u, u, u, u, u, u, u, 1, 16, 128, 128, 4, i, u, u, u, u),
    ):
        with pytest.raises(ValueError, match="not on the current CUDA device"):
            call_()


def test_binding_refuses_other_devices_and_strides(abi, monkeypatch):
    class Fake:
        def __init__(self, device, contiguous=True):
            self.device, self.ok, self.shape = device, contiguous, (2, 2)

        def get_device(self):
            return self.device

        def is_contiguous(self):
            return self.ok

        def stride(self):
            return (1, 2)

        def data_ptr(self):
            return 256 + self.device

    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    assert abi._on_gpu(Fake(0), None, Fake(0)) == [256, None, 256]
    for others in ((Fake(0), Fake(1)), (Fake(1),), (Fake(0), Fake(-1)), (Fake(-1), Fake(0)), (None, Fake(-1))):
        with pytest.raises(ValueError, match="current CUDA device"):
            abi._on_gpu(*others)
    with pytest.raises(ValueError, match="not contiguous"):
        abi._on_gpu(Fake(0), Fake(0, contiguous=False))
