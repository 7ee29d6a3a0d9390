"""The binding's checks of the operands of the rows' gradients and of the MXFP4 entry points: a tensor of another
type, or one too short for what the library reads or writes, is refused before the library is called. No GPU: the
tensors are stand-ins that say they are on the current device, and the library's functions record their arguments."""
import functools

import pytest
import torch

import __graft_entry__

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
T, D, K, E, F, ROWS = 6, 256, 2, 4, 384, 150


@pytest.fixture(scope="module")
def abi():
    __graft_entry__.build()
    from mixture_experts_routing_route_b200 import _abi
    return _abi


class Fake:
    """A tensor on device 0 as far as the binding looks."""

    def __init__(self, dtype, n, address=4096, device=0, contiguous=True):
        self.dtype, self.n, self.address, self.device, self.ok = dtype, n, address, device, contiguous
        self.shape = (n,)

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.ok

    def stride(self):
        return (2,)

    def numel(self):
        return self.n

    def data_ptr(self):
        return self.address


def row_scales(k):
    return (ROWS // 128 + E) * (k // 128) * 512


def weight_scales():
    return E * (F // 128) * (D // 128) * 512


# entry point: (arguments by name in order, of which the operands are (dtype, elements))
def calls(abi, dt):
    codes, wcodes = (U8, ROWS * D // 2), (U8, E * F * D // 2)
    return {
        "moe_combine_backward": [("d_out", (dt, T * D)), ("y_perm", (dt, ROWS * D)), ("topk_w", (F32, T * K)),
                                 ("slot_to_row", (I32, T * K)), T, D, K, ROWS, ("d_y_perm", (dt, ROWS * D)),
                                 ("d_topk_w", (F32, T * K)), ("ws", (U8, 256))],
        "moe_gather_backward": [("d_x_perm", (dt, ROWS * D)), ("slot_to_row", (I32, T * K)), ("dx_in", (dt, T * D)),
                                T, D, K, ROWS, ("dx", (dt, T * D)), ("ws", (U8, 256))],
        "moe_mxfp4_quantize_weights": [("w", (dt, E * D * F)), E, D, F, ("codes", wcodes),
                                       ("scales", (U8, weight_scales()))],
        "moe_mxfp4_dequantize_weights": [("codes", wcodes), ("scales", (U8, weight_scales())), E, D, F,
                                         ("w", (dt, E * D * F))],
        "moe_gather_mxfp4": [("x", (dt, T * D)), T, D, K, ("slot_to_row", (I32, T * K)), ("seg", (I32, E + 1)), E, ROWS,
                             ("codes", codes), ("scales", (U8, row_scales(D))), ("ws", (U8, 256))],
        "moe_mxfp4_dequantize_rows": [("codes", codes), ("scales", (U8, row_scales(D))), ("seg", (I32, E + 1)), E, ROWS,
                                      D, ("out", (dt, ROWS * D)), ("ws", (U8, 256))],
        "moe_expert_ffn_mxfp4": [("x", codes), ("xs", (U8, row_scales(D))), ("w1", wcodes), ("s1", (U8, weight_scales())),
                                 ("w3", wcodes), ("s3", (U8, weight_scales())), ("w2", wcodes),
                                 ("s2", (U8, weight_scales())), abi.MOE_ACT_SWIGLU, ROWS, D, F, E, ("seg", (I32, E + 1)),
                                 ("h", (U8, ROWS * F // 2)), ("hs", (U8, row_scales(F))), ("y", (BF16, ROWS * D)),
                                 ("ws", (U8, 256))],
    }


NAMES = ["moe_combine_backward", "moe_gather_backward", "moe_mxfp4_quantize_weights", "moe_mxfp4_dequantize_weights",
         "moe_gather_mxfp4", "moe_mxfp4_dequantize_rows", "moe_expert_ffn_mxfp4"]


@pytest.fixture
def reached(abi, monkeypatch):
    """What the library is called with."""
    got = []
    for name in NAMES:
        monkeypatch.setattr(abi._lib, name, lambda *a: got.append(a) or 0)
    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    monkeypatch.setattr(abi, "_raw_stream", lambda device: 7000 + device)
    return got


def arguments(abi, name, dt, **over):
    out = []
    for i, a in enumerate(calls(abi, dt)[name]):
        if isinstance(a, tuple):
            dtype, n = a[1]
            a = over.get(a[0], Fake(dtype, n, address=4096 * (i + 1)))
        out.append(a)
    return out


def operands(abi, name, dt):
    return [a for a in calls(abi, dt)[name] if isinstance(a, tuple)]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dt", [BF16, F32])
def test_right_operands_reach_the_library(abi, reached, name, dt):
    getattr(abi, name)(*arguments(abi, name, dt))
    (args,) = reached
    assert args[-1] == 7000  # the current stream of the current device
    for i, a in enumerate(calls(abi, dt)[name]):
        if isinstance(a, tuple):
            assert 4096 * (i + 1) in args
    # a longer buffer, and another stream
    op, (dtype, n) = operands(abi, name, dt)[0]
    getattr(abi, name)(*arguments(abi, name, dt, **{op: Fake(dtype, n + 5)}), stream=99)
    assert reached[1][-1] == 99


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dt", [BF16, F32])
def test_wrong_operands_do_not(abi, reached, name, dt):
    call = functools.partial(getattr(abi, name), stream=99)
    for op, (dtype, n) in operands(abi, name, dt):
        if op != "ws":  # the library checks its size
            with pytest.raises(ValueError, match="values are read or written"):
                call(*arguments(abi, name, dt, **{op: Fake(dtype, n - 1)}))
        for other in (F32, BF16, I32, torch.int64, U8, torch.float16):
            # the one tensor of values in the call may have either type
            # and a workspace any: the library counts its elements as bytes
            if other is dtype or op == "ws" or (name.startswith(("moe_mxfp4", "moe_gather_mxfp4")) and {dtype, other} == {F32, BF16}):
                continue
            with pytest.raises(ValueError, match="is read or written|values are|unsupported dtype"):
                # long enough in bytes of any of them
                call(*arguments(abi, name, dt, **{op: Fake(other, n)}))
        with pytest.raises(ValueError, match="current CUDA device"):
            call(*arguments(abi, name, dt, **{op: Fake(dtype, n, device=1)}))
        with pytest.raises(ValueError, match="current CUDA device"):
            call(*arguments(abi, name, dt, **{op: Fake(dtype, n, device=-1)}))
        with pytest.raises(ValueError, match="not contiguous"):
            call(*arguments(abi, name, dt, **{op: Fake(dtype, n, contiguous=False)}))
    assert reached == []


def test_optional_operands(abi, reached):
    for op in ("y_perm", "d_topk_w"):
        abi.moe_combine_backward(*arguments(abi, "moe_combine_backward", BF16, **{op: None}))
        assert None in reached.pop()
    abi.moe_gather_backward(*arguments(abi, "moe_gather_backward", BF16, dx_in=None))
    assert None in reached.pop()
    # codes and scales in a type of one byte that says what they are
    abi.moe_mxfp4_quantize_weights(*arguments(abi, "moe_mxfp4_quantize_weights", BF16,
                                              scales=Fake(torch.float8_e8m0fnu, weight_scales())))
    assert len(reached) == 1


def test_gelu_takes_no_w3(abi, reached):
    args = arguments(abi, "moe_expert_ffn_mxfp4", BF16, w3=None, s3=None)
    args[8] = abi.MOE_ACT_GELU
    abi.moe_expert_ffn_mxfp4(*args)
    assert reached[0][4:6] == (None, None)
