"""The activations of the MXFP4 up projection over [-9, 9], in relative terms: a block of 32 columns of h has a
scale of its own, so a block whose values all lie in the tail of GELU is as precise as any other.

The products' sums are exact. Column n of the weights makes z = (n - F / 2) / 64 of ones in x (an integer part in
one block of K, a fraction of 64 in the next), and row r adds m[r] / 1024: every partial sum is a multiple of 2^-10
below 16 (14 bits). What is left is the activation, then one rounding to E2M1.

The bound on the activation, relative to its value, a = |z|: what mxfp4_gemm.cuh states for its polynomials in fp32.
Blocks in the tail (no value of 0.3, some below -2.5) and every block of a decode step: 1.7e-6 for a <= 3, 5.5e-6 to 6,
1.2e-5 to 8, 3.5e-5 to 10. Other blocks: 8e-6 for a <= 2, 3e-5 to 2.5, 6e-5 to 3, 6.5e-3 to 4, 6e-2 to 5, all of it
beyond (such values have the code 0 there). The hardware's exponential (2 ulp), the last product and the sum (half an
ulp each) add 2^-22 + 2^-24 + 2^-24 < 2^-21. silu adds 2^-18 (hardware exponential and reciprocal, |z| below 26)."""
import numpy as np
import pytest
import torch

from mixture_experts_routing_route_b200 import _abi as abi
from tests import mx_reference as R
from tests.gpu_helpers import new_ws, npi

pytestmark = pytest.mark.gpu
DEV = "cuda"
OFFSETS = np.array([0, 1, 2, 3, 4, 6])  # of the rows, in 1 / 1024


def codes_of(total):
    """At most 32 E2M1 codes whose values add up to a whole number."""
    sign, left, out = 8 * (total < 0), abs(total), []
    for value, code in ((6, 7), (4, 6), (3, 5), (2, 4), (1, 2)):
        while left >= value:
            out.append(code + sign)
            left -= value
    return np.pad(np.array(out, np.uint8), (0, 32 - len(out)))


def packed_weights(codes, scales):
    """Codes [N, K] and scale bytes [N, K / 32] of one expert as the library holds them."""
    N, K = codes.shape
    tiled = np.zeros(N * K // 32, np.uint8)
    n, b = np.arange(N)[:, None], np.arange(K // 32)[None, :]
    tiled[R.scale_at(n // 128, K // 128, n % 128, b)] = scales
    return torch.from_numpy(R.pack(codes)[None]).to(DEV), torch.from_numpy(tiled).to(DEV)


# z of the columns, in 1 / 64
ORDERS = {
    "ascending": lambda F: np.arange(F) - F // 2,
    # every block spans the range
    "mixed": lambda F: (np.arange(F) * (F // 32 + 1)) % F - F // 2,
    # a tiny value, or one on either side of 0.3, in every block of the tail
    "zero": lambda F: np.where(np.arange(F) % 32 == 5, 0, np.arange(F) - F // 2),
    "edge": lambda F: np.where(np.arange(F) % 32 == 5, 19, np.arange(F) - F // 2),
}


def inputs(d, F, rows, order):
    q = ORDERS[order](F)
    w, ws = np.zeros((F, d), np.uint8), np.full((F, d // 32), 127, np.uint8)
    for n in range(F):
        w[n, :32], w[n, 32:64] = codes_of(int(q[n] // 64)), codes_of(int(q[n] % 64))
    ws[:, 1] = 127 - 6
    w[:, 64] = 2                          # 1.0
    up = np.zeros_like(w)
    up[:, 96] = 2
    m = OFFSETS[np.arange(rows) % len(OFFSETS)]
    x, xs = np.zeros((rows, d), np.uint8), np.full((rows, d // 32), 127, np.uint8)
    x[:, :64] = 2
    x[:, 64] = np.array([0, 2, 4, 5, 6, 0, 7], np.uint8)[m]
    xs[:, 2] = 127 - 10
    x[:, 96] = 2                          # u = 1
    scales = np.full(abi.moe_mxfp4_row_scales_size(rows, 1, d), 0xFF, np.uint8)
    g, r = R.row_groups([0, rows])
    scales[R.scale_at(g[:, None], d // 128, r[:, None], np.arange(d // 32)[None, :])] = xs
    z = q[None, :] / 64 + m[:, None] / 1024
    return z, torch.from_numpy(R.pack(x)).to(DEV), torch.from_numpy(scales).to(DEV), packed_weights(w, ws), \
        packed_weights(up, np.full_like(ws, 127))


def gelu_bound(z, all_tail):
    """z [rows, blocks, 32]."""
    a = np.abs(z)
    tail = np.select([a <= 3, a <= 6, a <= 8], [1.7e-6, 5.5e-6, 1.2e-5], 3.5e-5)
    rest = np.select([a <= 2, a <= 2.5, a <= 3, a <= 4, a <= 5], [8e-6, 3e-5, 6e-5, 6.5e-3, 6e-2], 1.0)
    deep = (z.min(-1, keepdims=True) < -2.5) & (z.max(-1, keepdims=True) < 0.3)
    return np.where(deep | all_tail, tail, rest) + 2.0 ** -21


def nearest(m):
    """Magnitudes to E2M1, ties to the even code, saturating at 6."""
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    return np.minimum(np.round(m / step) * step, 6.0)


@pytest.mark.parametrize("act,order", [("gelu", o) for o in ORDERS] + [("swiglu", "ascending"), ("swiglu", "mixed")])
@pytest.mark.parametrize("d,F,rows", [
    (128, 1152, 6),      # the weight stream of a decode step
    (128, 1024, 40),     # single CTAs, 256 columns of the MMA
    (128, 1152, 40),     # 128 columns (GELU)
    (2048, 1024, 300),   # CTA pairs
    (2048, 1152, 300),
])
def test_activation(act, order, d, F, rows):
    from scipy.special import erfc
    z, x, xs, (w1, s1), (w3, s3) = inputs(d, F, rows, order)
    z = z.reshape(rows, F // 32, 32)
    w2 = torch.zeros(1, d, F // 2, dtype=torch.uint8, device=DEV)
    s2 = torch.full((d * F // 32,), 127, dtype=torch.uint8, device=DEV)
    seg = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    h = torch.zeros(rows, F // 2, dtype=torch.uint8, device=DEV)
    hs = torch.zeros(abi.moe_mxfp4_row_scales_size(rows, 1, F), dtype=torch.uint8, device=DEV)
    y = torch.full((rows, d), 77.0, dtype=torch.bfloat16, device=DEV)
    ws = new_ws(abi.moe_expert_ffn_mxfp4_workspace_size(rows, d, F, 1))
    gelu = act == "gelu"
    abi.moe_expert_ffn_mxfp4(x, xs, w1, s1, None if gelu else w3, None if gelu else s3, w2, s2,
                             abi.MOE_ACT_GELU if gelu else abi.MOE_ACT_SWIGLU, rows, d, F, 1, seg, h, hs, y, ws)
    assert abi.moe_get_device_error(ws) == 0
    assert torch.all(y == 0)
    if gelu:
        ref, delta = z * 0.5 * erfc(-z / np.sqrt(2.0)), gelu_bound(z, all_tail=rows <= 32)
    else:
        ref, delta = z / (1.0 + np.exp(-z)), np.full_like(z, 2.0 ** -18)
    scale = R.row_scales(npi(hs), [0, rows], F)
    low, high = np.abs(ref * (1 - delta)), np.abs(ref * (1 + delta))
    assert not np.any(np.floor(np.log2(low.max(-1))) - 2 + 127 > scale)
    assert not np.any(np.floor(np.log2(high.max(-1))) - 2 + 127 < scale)
    X = np.ldexp(1.0, scale.astype(np.int64) - 127)[..., None]
    codes = R.unpack(npi(h)).reshape(z.shape)
    got = R.MAGNITUDES[codes & 7]
    bad = (got < nearest(low / X)) | (got > nearest(high / X))
    assert not bad.any(), np.unique(np.floor(z[bad]), return_counts=True)
    assert np.all((np.where(codes & 8, -1.0, 1.0) == np.sign(ref)) | (codes & 7 == 0))
