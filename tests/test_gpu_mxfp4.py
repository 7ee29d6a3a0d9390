"""MXFP4: quantising and reading back bit for bit against the format's
definition, and the experts' FFN on 4-bit rows and weights against float64.

The FFN is checked in two steps, because h is quantised in between and a sum
that is off by one part in 10^6 may fall on the other side of a rounding step:
the kernel's own h (read back) has to be a correct quantisation of a value
within delta of the exact h, and y has to be the product of the kernel's own h.
Sums on the tensor cores: every product of two codes is exact in fp32, and each
of the K additions loses at most 2^-23 of the sum of magnitudes M so far
(truncation), so |error| <= K 2^-23 M. silu and gelu add 2^-18 of their value
(hardware exponential: 2 + |1.16 g| ulp, under 32 ulp for |g| < 26)."""
import numpy as np
import pytest
import torch

from mixture_experts_routing_route_b200 import _abi as abi
from tests import mx_reference as R
from tests.gpu_helpers import new_ws, np32, npi
from tests.test_gpu_dispatch_backward import routing

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def u8(n, fill=0xFF):
    """A byte buffer full of NaN scales (and of -6 codes): what is not written must not matter."""
    return torch.full((max(int(n), 16),), fill, dtype=torch.uint8, device=DEV)


def quantise_weights(w):
    E, K, N = w.shape
    codes, scales = u8(E * N * K // 2), u8(abi.moe_mxfp4_weight_scales_size(E, K, N))
    abi.moe_mxfp4_quantize_weights(w, E, K, N, codes, scales)
    return codes, scales


def awkward(shape, dt, seed):
    """Values with what quantising can get wrong: blocks of zeros, of signed
    zeros, exact ties, values that saturate, powers of two, tiny and huge
    magnitudes, Inf and NaN (blocks are 32 consecutive values of the last axis)."""
    g = np.random.default_rng(seed)
    v = g.standard_normal(shape).astype(np.float32)
    b = v.reshape(-1, 32)
    n = len(b)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, 0.2499, 0.7501, 4.0, 0.0, -0.0, -5.0],
                    np.float32)
    pick = lambda i: b[i % n]  # noqa: E731
    pick(1)[:] = 0.0
    pick(2)[:] = -0.0
    pick(3)[:16], pick(3)[16:] = ties, -ties
    pick(4)[:16], pick(4)[16:] = ties * 2.0 ** -20, ties * 2.0 ** -20
    pick(5)[:] = 2.0 ** -140 * g.integers(-9, 10, 32)   # fp32 subnormals
    pick(6)[:] = 3.3e38 * g.uniform(-1, 1, 32)
    pick(7)[3] = np.inf
    pick(8)[30] = np.nan
    pick(9)[0] = -np.inf
    pick(10)[:] = 2.0 ** g.integers(-3, 4, 32)
    pick(11)[:] = 1e-30
    return torch.from_numpy(v).to(DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("E,K,N", [(1, 128, 128), (3, 384, 256), (2, 1024, 640), (5, 128, 1152)])
def test_weights(E, K, N, dt):
    wt = awkward((E, N, K), dt, E + K)               # blocks along K
    w = wt.transpose(1, 2).contiguous().to(DEV)
    codes, scales = quantise_weights(w)
    rc, rs = R.quantise(wt.float().numpy())
    assert np.array_equal(R.weight_scales(npi(scales), E, K, N), rs)
    got = R.unpack(npi(codes).reshape(E, N, K // 2))
    assert np.array_equal(got, rc)
    back = torch.empty_like(w)
    abi.moe_mxfp4_dequantize_weights(codes, scales, E, K, N, back)
    ref = R.values(rc, rs).transpose(0, 2, 1)
    assert np.array_equal(np32(back).astype(np.float64), ref, equal_nan=True)


def test_nearest_code_of_every_bf16_magnitude():
    """Every finite bf16 magnitude against a block maximum of 6 (scale 1)."""
    v = torch.arange(0, 0x40C1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # 0 .. 6
    n = -(-len(v) // 31)
    blocks = torch.zeros(n * 32, dtype=torch.bfloat16).reshape(n, 32)
    blocks[:, 0] = 6.0
    flat = torch.zeros(n * 31, dtype=torch.bfloat16)
    flat[:len(v)] = v
    blocks[:, 1:] = flat.reshape(n, 31)
    rows = -(-n // 512) * 128
    wt = torch.zeros(rows * 4, 32, dtype=torch.bfloat16)
    wt[:n] = blocks
    wt = wt.reshape(1, rows, 128)
    codes, scales = quantise_weights(wt.transpose(1, 2).contiguous().to(DEV))
    rc, _ = R.quantise(wt.float().numpy())
    assert np.array_equal(R.unpack(npi(codes).reshape(1, rows, 64)), rc)


ROWS = [
    (1, 128, 1, 1, "bf16", 0.0),
    (1, 4096, 8, 2, "bf16", 0.0),         # (binned: a capacity of no row)
    (130, 384, 4, 2, "f32", 1.0),
    (77, 1152, 16, 8, "bf16", 0.0),       # a row of one chunk and a bit
    (1000, 256, 256, 3, "f32", 0.5),
    (2049, 2176, 3, 1, "bf16", 1.25),
]


@pytest.mark.parametrize("T,d,E,k,dt,cf", ROWS)
@pytest.mark.parametrize("binned", [False, True])
def test_gather(T, d, E, k, dt, cf, binned):
    _, _, p, rows = routing(T, E, k, cf if not binned else max(cf, 1.0), T + d, binned)
    x = awkward((T, d), dt, T).to(DEV)
    codes, scales = u8(rows * d // 2), u8(abi.moe_mxfp4_row_scales_size(rows, E, d))
    out = torch.full((rows, d), 77.0, dtype=DT[dt], device=DEV)
    ws = new_ws(256)
    abi.moe_gather_mxfp4(x, T, d, k, p["slot_to_row"], p["seg_offsets"], E, rows, codes, scales, ws)
    abi.moe_mxfp4_dequantize_rows(codes, scales, p["seg_offsets"], E, rows, d, out, ws)
    assert abi.moe_get_device_error(ws) == 0
    s2r, seg = npi(p["slot_to_row"])[:T * k], npi(p["seg_offsets"])[:E + 1]
    kept = np.nonzero(s2r >= 0)[0]
    row, token = s2r[kept], kept // k
    rc, rs = R.quantise(np32(x))
    gc = R.unpack(npi(codes)[:rows * d // 2].reshape(rows, d // 2))
    assert np.array_equal(gc[row], rc[token])
    assert np.array_equal(R.row_scales(npi(scales), seg, d)[row], rs[token])
    empty = np.ones(rows, bool)
    empty[row] = False
    assert np.all(gc[empty] == 15)  # rows that hold no slot: as they were
    got = np32(out).astype(np.float64)
    assert np.array_equal(got[row], R.values(rc, rs)[token], equal_nan=True)
    assert np.all(got[seg[E]:] == 77.0)


def test_weights_are_quantised_on_the_stream_given():
    """A transposed matrix has to be copied first: on the same stream, behind
    what fills it there."""
    side = torch.cuda.Stream()
    wt = awkward((2, 512, 256), "bf16", 3).to(DEV)
    rc, rs = R.quantise(wt.float().cpu().numpy())
    w = torch.zeros_like(wt)
    abi.quantize_expert_weights(w.transpose(1, 2))  # loads every kernel (a first launch waits for the device)
    with torch.cuda.stream(side):
        w.copy_(wt)
    for stream in (side, side.cuda_stream):
        w.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
            w.copy_(wt)
        codes, scales = abi.quantize_expert_weights(w.transpose(1, 2), stream)
        torch.full_like(w, 9.0)  # may take memory that the current stream freed
        torch.cuda.synchronize()
        assert np.array_equal(R.unpack(npi(codes).reshape(2, 512, 128)), rc)
        assert np.array_equal(R.weight_scales(npi(scales), 2, 256, 512), rs)


def test_gather_reports_rows_out_of_range():
    T, d, E, k = 4, 128, 2, 2
    s2r = torch.tensor([0, 4, 1, 9, 2, 5, 3, -1], dtype=torch.int32, device=DEV)
    seg = torch.tensor([0, 4, 6], dtype=torch.int32, device=DEV)
    x = torch.randn(T, d, device=DEV)
    codes, scales = u8(6 * 64), u8(abi.moe_mxfp4_row_scales_size(6, E, d))
    ws = new_ws(256)
    abi.moe_gather_mxfp4(x, T, d, k, s2r, seg, E, 6, codes, scales, ws)
    assert abi.moe_get_device_error(ws) == abi.DEVERR_ROW_RANGE
    rc, _ = R.quantise(np32(x))
    assert np.array_equal(R.unpack(npi(codes)[:6 * 64].reshape(6, 64)), rc[[0, 1, 2, 3, 0, 2]])


# ------------------------------------------------------------------- FFN
class Experts:
    def __init__(self, E, d, F, act, seed, scale=0.05):
        g = torch.Generator().manual_seed(seed)
        mk = lambda K, N: (scale * torch.randn(E, K, N, generator=g)).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.E, self.d, self.F, self.act = E, d, F, act
        self.w1, self.w2 = quantise_weights(mk(d, F)), quantise_weights(mk(F, d))
        self.w3 = quantise_weights(mk(d, F)) if act == "swiglu" else (None, None)

    def values(self, w, K, N):
        out = torch.empty(self.E, K, N, device=DEV)
        abi.moe_mxfp4_dequantize_weights(w[0], w[1], self.E, K, N, out)
        return out.double()


def run_ffn(ex, xc, xs, rows, seg, stream=None, ws=None):
    hc, hs = u8(rows * ex.F // 2), u8(abi.moe_mxfp4_row_scales_size(rows, ex.E, ex.F))
    y = torch.full((rows, ex.d), 77.0, dtype=torch.bfloat16, device=DEV)
    if ws is None:
        ws = new_ws(abi.moe_expert_ffn_mxfp4_workspace_size(rows, ex.d, ex.F, ex.E))
    act = abi.MOE_ACT_SWIGLU if ex.act == "swiglu" else abi.MOE_ACT_GELU
    abi.moe_expert_ffn_mxfp4(xc, xs, *ex.w1, *ex.w3, *ex.w2, act, rows, ex.d, ex.F, ex.E, seg, hc, hs, y, ws, stream)
    return hc, hs, y, ws


def rows_of(ex, counts, extra, seed):
    """Rows with the given counts per expert, quantised; codes and scales of
    what holds no row stay NaN."""
    seg = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    n = int(seg[-1])
    rows = n + extra
    x = np.random.default_rng(seed).standard_normal((n, ex.d))
    rc, rs = R.quantise(x)
    codes = np.full((rows, ex.d // 2), 0xFF, np.uint8)
    codes[:n] = R.pack(rc)
    scales = np.full(abi.moe_mxfp4_row_scales_size(rows, ex.E, ex.d), 0xFF, np.uint8)
    g, r = R.row_groups(seg)
    scales[R.scale_at(g[:, None], ex.d // 128, r[:, None], np.arange(ex.d // 32)[None, :])] = rs
    return rows, torch.from_numpy(seg).to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)


def check_ffn(ex, rows, seg, xc, xs, hc, hs, y):
    segh = npi(seg)
    n, E, d, F = int(segh[-1]), ex.E, ex.d, ex.F
    x = torch.from_numpy(R.values(R.unpack(npi(xc)[:n]), R.row_scales(npi(xs), segh, d))).to(DEV)
    h = torch.from_numpy(R.values(R.unpack(npi(hc)[:rows * F // 2].reshape(rows, F // 2)[:n]),
                                  R.row_scales(npi(hs), segh, F))).to(DEV)
    w1, w2 = ex.values(ex.w1, d, F), ex.values(ex.w2, F, d)
    w3 = ex.values(ex.w3, d, F) if ex.act == "swiglu" else None
    yd = y.double()
    assert torch.all(yd[n:] == 77.0)  # rows behind the last segment: as they were
    sq, ref2 = 0.0, 0.0
    for e in range(E):
        a, b = int(segh[e]), int(segh[e + 1])
        if a == b:
            continue
        xe = x[a:b]
        g, gm = xe @ w1[e], xe.abs() @ w1[e].abs()
        tol = d * 2.0 ** -23
        if ex.act == "swiglu":
            u, um = xe @ w3[e], xe.abs() @ w3[e].abs()
            s = g * torch.sigmoid(g)
            ref = s * u
            # |silu'| <= 1.1
            delta = 1.1 * tol * gm * u.abs() + tol * um * s.abs() + 1.1 * tol * tol * gm * um + 2.0 ** -18 * ref.abs()
        else:
            ref = 0.5 * g * torch.erfc(-g / 2 ** 0.5)
            delta = 1.2 * tol * gm + 2.0 ** -18 * ref.abs()  # |gelu'| <= 1.13
            # where the two terms of 1 + erf cancel: erf is good to 2^-22
            delta = delta + 2.0 ** -22 * g.abs()
        he = h[a:b]
        # The scale comes from a block maximum within delta of the exact one. Where that straddles a power
        # of two either scale is right, and each has its own error: with the smaller one, X, values from 6 X
        # to 8 X saturate and lose up to 2 X, which is more than half a step (0.5 * 2 X) of the larger one at
        # magnitudes below 4 * 2 X. So the bound is the larger of the two.
        rb, db = ref.reshape(b - a, -1, 32), delta.reshape(b - a, -1, 32)
        bound = torch.zeros_like(rb)
        for top in ((rb.abs() + db).amax(-1, keepdim=True), (rb.abs() - db).amax(-1, keepdim=True).clamp(min=1e-30)):
            X = torch.exp2(torch.floor(torch.log2(top)) - 2)
            m = (rb.abs() + db) / X
            half = torch.where(m < 2, 0.25, torch.where(m < 4, 0.5, torch.where(m <= 6, 1.0, torch.clamp(m - 6.0, min=1.0))))
            bound = torch.maximum(bound, half * X)
        assert torch.all((he.reshape(rb.shape) - rb).abs() <= bound * (1 + 1e-9) + db)
        yr, ym = he @ w2[e], he.abs() @ w2[e].abs()
        err = (yd[a:b] - yr).abs()
        assert torch.all(err <= 1.01 * (2.0 ** -8 * yr.abs() + F * 2.0 ** -23 * ym))
        sq, ref2 = sq + float(err.square().sum()), ref2 + float(yr.square().sum())
    # rounding to bf16 alone is at most 2^-8 of the norm
    assert ref2 == 0.0 or (sq / ref2) ** 0.5 <= 2.0 ** -8


FFN = [
    # E, d, F, counts, act
    (1, 128, 128, [1], "gelu"),
    (1, 128, 128, [1], "swiglu"),
    (2, 256, 128, [0, 5], "swiglu"),
    (3, 384, 384, [127, 0, 129], "gelu"),        # half stages, N = 128 tiles
    (3, 384, 384, [128, 1, 255], "swiglu"),
    (4, 512, 768, [3, 200, 1, 77], "swiglu"),
    (8, 256, 1024, [64, 0, 0, 300, 2, 1, 513, 31], "gelu"),
    (5, 1024, 512, [0, 0, 700, 0, 0], "swiglu"),  # one expert has every row
    (64, 256, 256, [(7 * e) % 13 for e in range(64)], "gelu"),
    (256, 128, 128, [(5 * e) % 3 for e in range(256)], "swiglu"),
    (2, 4096, 1152, [33, 140], "swiglu"),        # K of many stages
    (3, 640, 2304, [260, 1, 9], "gelu"),
]


# 256 rows an expert or more (of the buffer) and K >= 2048: CTA pairs
PAIRS = [
    # E, d, F, counts, act, rows past the last
    (2, 2048, 384, [33, 700], "swiglu", 0),        # up; single CTAs down
    (2, 2176, 2304, [511, 1], "swiglu", 0),        # both; half stages, N = 128 tiles down
    (1, 2048, 2304, [256], "gelu", 0),             # a whole tile
    (1, 2304, 2176, [257], "gelu", 3),             # one row more; N = 128 tiles up
    (3, 384, 4096, [0, 300, 500], "gelu", 0),      # down; single CTAs up
    (4, 4096, 2048, [1, 0, 1000, 130], "swiglu", 0),
    (8, 2048, 2048, [5, 0, 0, 0, 130, 0, 0, 1], "swiglu", 2048),  # few rows of a large buffer
    (3, 2048, 2048, [0, 0, 0], "gelu", 900),       # none
]


# a decode step: at most 32 rows in all (the weight stream, tiles cut between blocks)
FEW = [
    (1, 128, 128, [1], "swiglu"),
    (8, 4096, 1792, [0, 1, 0, 0, 0, 0, 1, 0], "swiglu"),
    (4, 384, 640, [3, 0, 8, 1], "gelu"),          # half stages
    (2, 2176, 3200, [31, 1], "swiglu"),
    (256, 256, 384, [1 if e % 9 == 4 else 0 for e in range(256)], "gelu"),
    (3, 128, 4096, [0, 32, 0], "swiglu"),          # one stage a tile up, sixteen down
    (6, 7168, 128, [5, 0, 0, 2, 0, 25], "swiglu"),  # a tile cut between many blocks
    (64, 512, 2048, [1 if e in (0, 17, 40, 63) else 0 for e in range(64)], "gelu"),
]


@pytest.mark.parametrize("E,d,F,counts,act", FFN + FEW)
@pytest.mark.parametrize("extra", [0, 19])
def test_ffn(E, d, F, counts, act, extra):
    ex = Experts(E, d, F, act, seed=d + F)
    rows, seg, xc, xs = rows_of(ex, counts, extra, seed=E)
    hc, hs, y, ws = run_ffn(ex, xc, xs, rows, seg)
    assert abi.moe_get_device_error(ws) == 0
    check_ffn(ex, rows, seg, xc, xs, hc, hs, y)


@pytest.mark.parametrize("E,d,F,counts,act,extra", PAIRS)
def test_ffn_pairs(E, d, F, counts, act, extra):
    test_ffn(E, d, F, counts, act, extra)


def test_ffn_no_rows_in_use():
    ex = Experts(4, 128, 256, "swiglu", 1)
    rows, seg, xc, xs = rows_of(ex, [0, 0, 0, 0], 8, 1)
    hc, _, y, ws = run_ffn(ex, xc, xs, rows, seg)
    assert abi.moe_get_device_error(ws) == 0
    assert torch.all(y == 77.0) and torch.all(hc == 255)


@pytest.mark.parametrize("d,counts", [(256, [40, 50]), (2048, [40, 500]), (256, [4, 60]), (256, [20, 12])])
def test_ffn_nan_rows_stay_alone(d, counts):
    ex = Experts(2, d, d, "swiglu", 2)
    rows, seg, xc, xs = rows_of(ex, counts, 0, 3)
    bad_row = rows - 5
    g, r = R.row_groups(npi(seg))
    xs[int(R.scale_at(g[bad_row], d // 128, r[bad_row], 1))] = 255   # one NaN block
    _, _, y, ws = run_ffn(ex, xc, xs, rows, seg)
    bad = torch.isnan(y).any(1)
    assert bad.sum().item() == 1 and bad[bad_row].item() and torch.isnan(y[bad_row]).all()


@pytest.mark.parametrize("d,F,counts", [(512, 1024, [130, 0, 4, 260, 1, 70]), (512, 1024, [3, 0, 4, 0, 1, 17]),
                                        (2048, 2048, [900, 0, 300, 1, 257, 100]),
                                        (512, 2048, [900, 0, 300, 1, 257, 100])])
def test_ffn_repeats_bit_for_bit_on_one_workspace_and_in_a_graph(d, F, counts):
    ex = Experts(6, d, F, "swiglu", 4)
    rows, seg, xc, xs = rows_of(ex, counts, 3, 5)
    hc, hs, y, ws = run_ffn(ex, xc, xs, rows, seg)
    for _ in range(3):
        a, b, c, _ = run_ffn(ex, xc, xs, rows, seg, ws=ws)
        assert torch.equal(a, hc) and torch.equal(b, hs) and torch.equal(c, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = run_ffn(ex, xc, xs, rows, seg, ws=ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], hc) and torch.equal(got[2], y)
    assert abi.moe_get_device_error(ws) == 0


@pytest.mark.parametrize("counts", [[40, 0, 24], [1, 0, 6]])
def test_ffn_of_one_row_does_not_depend_on_the_others(counts):
    """The same rows alone (few: the weight stream) and among others give the
    same h, and y within the two orders of summation."""
    ex = Experts(3, 1024, 768, "swiglu", 9)
    rows, seg, xc, xs = rows_of(ex, counts, 0, 10)
    hc, hs, y, _ = run_ffn(ex, xc, xs, rows, seg)
    solo = torch.tensor([0, 1, 1, 1], dtype=torch.int32, device=DEV)
    hc1, hs1, y1, ws = run_ffn(ex, xc[:1].contiguous(), xs, 1, solo)
    assert abi.moe_get_device_error(ws) == 0
    same = (hc1[:ex.F // 2] == hc[:ex.F // 2]).float().mean().item()
    assert same >= 0.99  # a sum next to a rounding step may fall on its other side
    assert float((y1[0].double() - y[0].double()).norm() / y[0].double().norm()) <= 2.0 ** -6


def test_ffn_bad_segments_set_the_error_bit():
    ex = Experts(2, 128, 128, "gelu", 6)
    rows, seg, xc, xs = rows_of(ex, [10, 20], 0, 7)
    bad = torch.tensor([0, 10, 31], dtype=torch.int32, device=DEV)  # one row past the buffer
    _, _, y, ws = run_ffn(ex, xc, xs, rows, bad)
    assert abi.moe_get_device_error(ws) & abi.DEVERR_ROW_RANGE
    assert torch.all(y[10:] == 77.0)  # the bad expert's rows are skipped


def test_decode_wait_for_h_runs_out_then_workspace_init_recovers():
    """The down projection's blocks of a decode step wait until the up
    projection's ranges are done, at most the workspace's wait limit. Here the
    counter that hands out the ranges starts behind those of the up projection,
    so nobody does them: every block gives up after 1 ms, sets
    MOE_DEVERR_TIMEOUT and returns, and the context stays usable."""
    stream_next = 188  # byte of that counter in the control block
    ex = Experts(8, 4096, 1792, "swiglu", 11)
    rows, seg, xc, xs = rows_of(ex, [0, 1, 0, 0, 0, 0, 1, 0], 0, 12)  # 448 stages up, 256 down
    hc, hs, y, ws = run_ffn(ex, xc, xs, rows, seg)
    abi.moe_workspace_set_wait_limit(ws, 1000)
    again = run_ffn(ex, xc, xs, rows, seg, ws=ws)  # the limit alone changes nothing
    assert torch.equal(again[2], y) and abi.moe_get_device_error(ws) == 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws[stream_next:stream_next + 4].view(torch.int32).fill_(sms)  # a range each of the up projection
    run_ffn(ex, xc, xs, rows, seg, ws=ws)
    torch.cuda.synchronize()
    assert abi.moe_get_device_error(ws) & abi.DEVERR_TIMEOUT
    abi.moe_workspace_init(ws)
    again = run_ffn(ex, xc, xs, rows, seg, ws=ws)
    assert abi.moe_get_device_error(ws) == 0
    assert torch.equal(again[0], hc) and torch.equal(again[2], y)


def test_quantise_gather_ffn_combine_together():
    """The operators one after another as a layer uses them: routing and permute
    of this library, 4-bit gather and experts, the bf16 combine."""
    T, d, E, k, F = 200, 512, 8, 2, 768
    ex = Experts(E, d, F, "swiglu", 8)
    _, w, p, rows = routing(T, E, k, 1.0, 12)
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    codes, scales = u8(rows * d // 2), u8(abi.moe_mxfp4_row_scales_size(rows, E, d))
    ws = new_ws(abi.moe_expert_ffn_mxfp4_workspace_size(rows, d, F, E))
    seg = p["seg_offsets"][:E + 1]
    abi.moe_gather_mxfp4(x, T, d, k, p["slot_to_row"], seg, E, rows, codes, scales, ws)
    hc, hs, y, _ = run_ffn(ex, codes, scales, rows, seg, ws=ws)
    out = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    abi.moe_combine(y, w, p["slot_to_row"], T, d, k, rows, out, ws)
    assert abi.moe_get_device_error(ws) == 0
    check_ffn(ex, rows, seg, codes[:rows * d // 2].reshape(rows, d // 2), scales, hc, hs, y)
    s2r = npi(p["slot_to_row"])[:T * k].reshape(T, k)
    yn, wn = np32(y).astype(np.float64), np32(w).astype(np.float64)
    ref = sum(np.where(s2r[:, j] >= 0, wn[:, j], 0.0)[:, None] * yn[np.maximum(s2r[:, j], 0)] for j in range(k))
    mag = sum(np.abs(np.where(s2r[:, j] >= 0, wn[:, j], 0.0)[:, None] * yn[np.maximum(s2r[:, j], 0)]) for j in range(k))
    assert np.all(np.abs(np32(out) - ref) <= 1.01 * (2.0 ** -8 * np.abs(ref) + 2 * k * 2.0 ** -24 * mag))


def test_offsets_past_32_bits():
    """Codes, values and h of more than 2^32 bytes: the last rows against the same rows on their own."""
    d, F, E, k = 8192, 8192, 2, 2
    T = (1 << 32) * 2 // d // k + 300            # T k rows of d / 2 bytes: past 4 GiB
    rows = T * k
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    x[-300:] = torch.randn(300, d, device=DEV, generator=g)
    s2r = torch.stack((torch.arange(T), torch.arange(T) + T), 1).to(torch.int32).to(DEV)
    seg = torch.tensor([0, T, rows], dtype=torch.int32, device=DEV)
    codes, scales = u8(rows * d // 2), u8(abi.moe_mxfp4_row_scales_size(rows, E, d))
    ws = new_ws(256)
    abi.moe_gather_mxfp4(x, T, d, k, s2r, seg, E, rows, codes, scales, ws)
    assert abi.moe_get_device_error(ws) == 0
    rc, _ = R.quantise(np32(x[-300:]))
    tail = codes[-300 * (d // 2):].reshape(300, d // 2)
    assert np.array_equal(R.unpack(npi(tail)), rc)
    ex = Experts(E, d, F, "gelu", 3)
    hc, hs, y, ws2 = run_ffn(ex, codes, scales, rows, seg)
    assert abi.moe_get_device_error(ws2) == 0
    # the last 300 rows on their own, as expert 1's only rows (the same place in their scale tiles)
    pad = T % 128 - 300 % 128
    n = 300 + (pad if pad >= 0 else pad + 128)
    seg1 = torch.tensor([0, 0, n], dtype=torch.int32, device=DEV)
    xs1 = u8(abi.moe_mxfp4_row_scales_size(n, E, d))
    xc1 = u8(n * d // 2).reshape(n, d // 2)
    s2r1 = torch.arange(n, dtype=torch.int32, device=DEV)
    abi.moe_gather_mxfp4(x[-n:].contiguous(), n, d, 1, s2r1, seg1, E, n, xc1, xs1, ws)
    _, _, y1, _ = run_ffn(ex, xc1, xs1, n, seg1)
    assert torch.equal(y[-300:], y1[-300:])
    assert y.shape[0] * d * 2 > 1 << 33
    out = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    abi.moe_mxfp4_dequantize_rows(codes, scales, seg, E, rows, d, out, ws)
    assert torch.equal(out[-300:], out[T - 300:T])
    assert np.array_equal(np32(out[-300:]).astype(np.float64), R.values(*R.quantise(np32(x[-300:]))))
    # and the gradients' way over rows of that many bytes
    w = torch.full((T, k), 0.5, device=DEV)
    dw = torch.empty(T, k, device=DEV)
    abi.moe_combine_backward(x, y, w, s2r, T, d, k, rows, out, dw, ws)
    assert torch.equal(out[-300:], 0.5 * x[-300:]) and torch.equal(out[T - 300:T], 0.5 * x[-300:])
    ref = (x[-300:].double() * y[-300:].double()).sum(1)
    mag = (x[-300:].double() * y[-300:].double()).abs().sum(1)
    assert torch.all((dw[-300:, 1].double() - ref).abs() <= 1.01 * (d + 1) * 2.0 ** -24 * mag)
    dx = torch.empty_like(x)
    abi.moe_gather_backward(out, s2r, None, T, d, k, rows, dx, ws)
    assert torch.equal(dx[-300:], x[-300:])
    assert abi.moe_get_device_error(ws) == 0
