"""The gather's and the combine's backward passes against the chain rule in
float64, at the sizes, layouts and drops where they can go wrong.

Tolerances: dy is one fp32 product rounded once more to its type; dw and dx are
fp32 sums in some order, |error| <= n 2^-24 * (sum of the terms' magnitudes)
for n additions and products (first order; 1.01 covers the rest), dx rounded
once more to its type."""
import numpy as np
import pytest
import torch

from mixture_experts_routing_route_b200 import _abi as abi
from tests import mx_reference as R
from tests.gpu_helpers import new_ws, np32, npi

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative


def routing(T, E, k, cf, seed, binned=False, capacity=None):
    """Picks and weights, and moe_permute's outputs for them."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32).to(DEV)
    w = torch.softmax(torch.randn(T, k, generator=g), 1).to(DEV)
    cap = abi.moe_capacity(cf, T, k, E) if capacity is None else capacity
    rows = abi.moe_rows_max_binned(T, k, E, cap) if binned else abi.moe_rows_max(T, k, E, cap)
    i32 = lambda n: torch.empty(max(n, 4), dtype=torch.int32, device=DEV)  # noqa: E731
    p = dict(counts=i32(E), bins=i32(E), sorted_slot=i32(T * k), slot_to_row=i32(T * k),
             row_slot=i32(rows), drop_mask=torch.empty(max(T * k, 16), dtype=torch.uint8, device=DEV),
             kept_counts=i32(E), seg_offsets=i32(E + 1))
    ws = new_ws(abi.moe_permute_workspace_size(T, k, E))
    f = abi.moe_permute_binned if binned else abi.moe_permute
    f(idx, T, k, E, cap, p["counts"], p["bins"], p["sorted_slot"], p["slot_to_row"], p["row_slot"],
      p["drop_mask"], p["kept_counts"], p["seg_offsets"], ws)
    assert abi.moe_get_device_error(ws) == 0
    return idx, w, p, rows


def randn(n, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, d, generator=g).to(DT[dt]).to(DEV)


CASES = [
    (1, 128, 1, 1, "bf16", 0.0),       # one token, one expert
    (1, 4096, 8, 2, "bf16", 0.0),
    (7, 4, 4, 2, "f32", 0.0),          # one 16-byte vector a row
    (256, 64, 4, 1, "f32", 1.25),      # the tiny layer
    (129, 640, 5, 3, "bf16", 1.0),     # k = 3, drops
    (61, 1028, 9, 5, "f32", 0.5),      # k = 5, half the slots dropped, a vector past 256
    (300, 1152, 16, 6, "bf16", 0.0),
    (33, 2052, 11, 7, "f32", 1.0),
    (77, 4096, 256, 8, "bf16", 0.0),   # fine-grained
    (1500, 1024, 64, 2, "bf16", 1.0),  # capacity
    (50, 8320, 6, 4, "bf16", 0.0),     # rows past one pass of a warp
    (3000, 256, 3, 2, "f32", 0.0),     # more slots than one grid of warps
]


@pytest.mark.parametrize("T,d,E,k,dt,cf", CASES)
def test_combine_backward(T, d, E, k, dt, cf):
    _, w, p, rows = routing(T, E, k, cf, T + d)
    dout, y = randn(T, d, dt, 1), randn(rows, d, dt, 2)
    dy = torch.full((rows, d), 77.0, dtype=DT[dt], device=DEV)
    dw = torch.full((T, k), 77.0, device=DEV)
    ws = new_ws(256)
    abi.moe_combine_backward(dout, y, w, p["slot_to_row"], T, d, k, rows, dy, dw, ws)
    assert abi.moe_get_device_error(ws) == 0
    s2r = npi(p["slot_to_row"])[:T * k]
    rdy, rdw, mag = R.combine_backward(np32(dout), np32(y), np32(w), s2r, rows)
    held = ~np.isnan(rdy)
    got = np32(dy).astype(np.float64)
    assert np.all(got[~held] == 77.0)  # rows that hold no slot stay as they were
    assert np.all(np.abs(got - rdy)[held] <= 1.01 * (U[dt] + 2.0 ** -24) * np.abs(rdy)[held])
    gdw = np32(dw).astype(np.float64)
    assert np.all(gdw[s2r.reshape(T, k) < 0] == 0.0)
    assert np.all(np.abs(gdw - rdw) <= 1.01 * (d + 1) * 2.0 ** -24 * mag)
    # one output alone: the same bits
    dy2, dw2 = torch.zeros_like(dy), torch.zeros_like(dw)
    abi.moe_combine_backward(dout, None, w, p["slot_to_row"], T, d, k, rows, dy2, None, ws)
    abi.moe_combine_backward(dout, y, None, p["slot_to_row"], T, d, k, rows, None, dw2, ws)
    assert np.array_equal(np32(dy2)[held], np32(dy)[held])
    assert torch.equal(dw2, dw)


@pytest.mark.parametrize("T,d,E,k,dt,cf", CASES)
@pytest.mark.parametrize("add", ["none", "other", "in place"])
def test_gather_backward(T, d, E, k, dt, cf, add):
    _, _, p, rows = routing(T, E, k, cf, T + d)
    g = randn(rows, d, dt, 3)
    dx_in = None if add == "none" else randn(T, d, dt, 4)
    dx = dx_in if add == "in place" else torch.full((T, d), 77.0, dtype=DT[dt], device=DEV)
    ref, mag = R.gather_backward(np32(g), npi(p["slot_to_row"])[:T * k], T, k,
                                 None if dx_in is None else np32(dx_in))
    ws = new_ws(256)
    abi.moe_gather_backward(g, p["slot_to_row"], dx_in, T, d, k, rows, dx, ws)
    assert abi.moe_get_device_error(ws) == 0
    assert np.all(np.abs(np32(dx) - ref) <= 1.01 * (U[dt] * np.abs(ref) + k * 2.0 ** -24 * mag))


@pytest.mark.parametrize("capacity", [0, 3])
def test_everything_or_nearly_everything_dropped(capacity):
    T, d, E, k = 40, 256, 4, 2
    _, w, p, rows = routing(T, E, k, 0.0, 5, capacity=capacity)
    assert rows == E * capacity
    dout, dx_in = randn(T, d, "bf16", 1), randn(T, d, "bf16", 2)
    y = randn(max(rows, 1), d, "bf16", 3)
    dy, dw = torch.zeros_like(y), torch.full((T, k), 9.0, device=DEV)
    dx = torch.empty_like(dx_in)
    ws = new_ws(256)
    abi.moe_combine_backward(dout, y, w, p["slot_to_row"], T, d, k, rows, dy, dw, ws)
    abi.moe_gather_backward(y, p["slot_to_row"], dx_in, T, d, k, rows, dx, ws)
    assert abi.moe_get_device_error(ws) == 0
    dropped = npi(p["slot_to_row"])[:T * k].reshape(T, k) < 0
    assert np.all(np32(dw)[dropped] == 0.0)
    gone = dropped.all(1)
    assert gone.any() and torch.equal(dx[torch.from_numpy(gone).to(DEV)], dx_in[torch.from_numpy(gone).to(DEV)])


def test_binned_layout():
    T, d, E, k = 200, 256, 8, 2
    _, w, p, rows = routing(T, E, k, 1.0, 6, binned=True)
    dout, y = randn(T, d, "bf16", 1), randn(rows, d, "bf16", 2)
    dy = torch.full((rows, d), 77.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(T, k, device=DEV)
    ws = new_ws(256)
    abi.moe_combine_backward(dout, y, w, p["slot_to_row"], T, d, k, rows, dy, dw, ws)
    rdy, rdw, mag = R.combine_backward(np32(dout), np32(y), np32(w), npi(p["slot_to_row"])[:T * k], rows)
    held = ~np.isnan(rdy)
    assert np.all(np32(dy)[~held] == 77.0)
    assert np.all(np.abs(np32(dy) - rdy)[held] <= 1.01 * (2.0 ** -8 + 2.0 ** -24) * np.abs(rdy)[held])
    assert np.all(np.abs(np32(dw) - rdw) <= 1.01 * (d + 1) * 2.0 ** -24 * mag)
    assert abi.moe_get_device_error(ws) == 0


def test_row_past_the_buffer_sets_the_error_bit_and_counts_as_dropped():
    T, d, k = 6, 128, 2
    s2r = torch.tensor([0, 1, 2, 50, 3, 4, 5, -1, 6, 7, 8, 9], dtype=torch.int32, device=DEV)
    rows = 10
    dout, y, w = randn(T, d, "bf16", 1), randn(rows, d, "bf16", 2), torch.rand(T, k, device=DEV)
    dy, dw, dx = torch.zeros_like(y), torch.empty(T, k, device=DEV), torch.empty_like(dout)
    ws = new_ws(256)
    abi.moe_combine_backward(dout, y, w, s2r, T, d, k, rows, dy, dw, ws)
    assert abi.moe_get_device_error(ws) == abi.DEVERR_ROW_RANGE
    assert dw[1, 1].item() == 0.0 and dw[3, 1].item() == 0.0
    abi.moe_gather_backward(y, s2r, None, T, d, k, rows, dx, ws)
    assert abi.moe_get_device_error(ws) == abi.DEVERR_ROW_RANGE
    assert torch.equal(dx[1], y[2]) and torch.equal(dx[3], y[5])


def test_no_tokens():
    ws = new_ws(256)
    n0 = abi.moe_kernel_launches()
    e = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    abi.moe_combine_backward(e, e, None, None, 0, 128, 2, 0, e, None, ws)
    abi.moe_gather_backward(e, None, None, 0, 128, 2, 0, e, ws)
    assert abi.moe_kernel_launches() == n0


def test_non_finite_values_stay_in_their_rows():
    T, d, E, k = 64, 256, 4, 2
    _, w, p, rows = routing(T, E, k, 0.0, 8)
    dout, y = randn(T, d, "f32", 1), randn(rows, d, "f32", 2)
    dout[3, 5], y[7, 9] = float("nan"), float("inf")
    dy, dw, dx = torch.empty_like(y), torch.empty(T, k, device=DEV), torch.empty_like(dout)
    ws = new_ws(256)
    abi.moe_combine_backward(dout, y, w, p["slot_to_row"], T, d, k, rows, dy, dw, ws)
    abi.moe_gather_backward(y, p["slot_to_row"], None, T, d, k, rows, dx, ws)
    s2r = npi(p["slot_to_row"])[:T * k].reshape(T, k)
    bad = np.isnan(np32(dw)) | np.isinf(np32(dw))
    assert np.array_equal(bad, (np.arange(T) == 3)[:, None] | (s2r == 7))
    assert np.isnan(np32(dy)).sum() == k and np.isinf(np32(dx)).sum() == 1


def test_other_stream_and_captured_graph_give_the_same_bits():
    T, d, E, k = 500, 512, 8, 2
    _, w, p, rows = routing(T, E, k, 0.0, 9)
    dout, y = randn(T, d, "bf16", 1), randn(rows, d, "bf16", 2)
    dy, dw, dx = torch.empty_like(y), torch.empty(T, k, device=DEV), torch.empty_like(dout)
    ws = new_ws(256)

    def run():
        abi.moe_combine_backward(dout, y, w, p["slot_to_row"], T, d, k, rows, dy, dw, ws)
        abi.moe_gather_backward(dy, p["slot_to_row"], dout, T, d, k, rows, dx, ws)

    run()
    torch.cuda.synchronize()
    first = [t.clone() for t in (dy, dw, dx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (dy, dw, dx):
            t.zero_()
        run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, (dy, dw, dx)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    dout.mul_(2.0)  # new inputs in the captured buffers
    for t in (dy, dw, dx):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(2 * a, b) for a, b in zip(first, (dy, dw, dx)))


def test_training_step_of_a_layer():
    """Route, permute, gather, experts (torch), combine, and the backward of all
    of it: the gradients of x and of the router weight against float64 autograd
    over the same picks, and against differences."""
    T, d, E, k, F = 96, 128, 4, 2, 64
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, d, generator=g).to(DEV)
    wg = (0.3 * torch.randn(d, E, generator=g)).to(DEV)
    w1 = (0.1 * torch.randn(E, d, F, generator=g)).to(DEV)
    w2 = (0.1 * torch.randn(E, F, d, generator=g)).to(DEV)
    dout = torch.randn(T, d, generator=g).to(DEV)
    f32 = lambda *n: torch.empty(*n, device=DEV)  # noqa: E731
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    tw, aux, logits, probs = f32(T, k), f32(1), f32(T, E), f32(T, E)
    wr = new_ws(abi.moe_route_workspace_size(T, d, E))
    abi.moe_route_train(x, wg, None, None, T, d, E, k, idx, tw, aux, None, logits, probs, wr)
    R_ = T * k
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    s2r, row_slot, kept, seg = i32(R_), i32(R_), i32(E), i32(E + 1)
    wp = new_ws(abi.moe_permute_workspace_size(T, k, E))
    abi.moe_permute(idx, T, k, E, -1, i32(E), i32(E), i32(R_), s2r, row_slot,
                    torch.empty(R_, dtype=torch.uint8, device=DEV), kept, seg, wp)
    ws = new_ws(256)
    x_perm, out = f32(R_, d), f32(T, d)
    abi.moe_gather(x, T, d, k, row_slot, seg, E, R_, x_perm, ws)
    bounds = seg.tolist()
    xp = x_perm.clone().requires_grad_(True)
    y = torch.cat([torch.tanh(xp[a:b] @ w1[e]) @ w2[e] for e, (a, b) in enumerate(zip(bounds, bounds[1:]))])
    y_perm = y.detach().contiguous()
    abi.moe_combine(y_perm, tw, s2r, T, d, k, R_, out, ws)
    # backward
    dy, dw = f32(R_, d), f32(T, k)
    abi.moe_combine_backward(dout, y_perm, tw, s2r, T, d, k, R_, dy, dw, ws)
    y.backward(dy)
    dlog, dxr, dwg, dx = f32(T, E), f32(T, d), f32(d, E), f32(T, d)
    wb = new_ws(abi.moe_route_backward_workspace_size(T, d, E))
    abi.moe_route_backward(x, wg, T, d, E, k, probs, None, idx, tw, dw, 0.7, 0.0, 1.0, dlog, dxr, dwg, wb)
    abi.moe_gather_backward(xp.grad, s2r, dxr, T, d, k, R_, dx, ws)
    for w_ in (wr, wp, ws, wb):
        assert abi.moe_get_device_error(w_) == 0

    picks = idx.long().cpu()
    counts = torch.bincount(picks.reshape(-1), minlength=E).double()
    A = [t.double().cpu() for t in (w1, w2, dout)]

    def loss(xx, ww):
        p = torch.softmax(xx @ ww, 1)
        sel = p.gather(1, picks)
        wt = sel / sel.sum(1, keepdim=True)
        o = sum(wt[:, j, None] * torch.einsum("tf,tfd->td", torch.tanh(torch.einsum("td,tdf->tf", xx, A[0][picks[:, j]])),
                                             A[1][picks[:, j]]) for j in range(k))
        return (o * A[2]).sum() + 0.7 * E * (counts / (T * k) * p.mean(0)).sum()

    x64, w64 = x.double().cpu().requires_grad_(True), wg.double().cpu().requires_grad_(True)
    loss(x64, w64).backward()
    for got, ref in ((dx, x64.grad), (dwg, w64.grad)):
        # fp32 sums of at most T d terms in some 20 steps: 1e-5 of the norm is far above their rounding
        assert float((got.double().cpu() - ref).norm() / ref.norm()) <= 1e-5
    # directional differences of the float64 loss along random directions
    with torch.no_grad():
        for seed in range(3):
            v = torch.randn(T, d, generator=torch.Generator().manual_seed(seed)).double()
            h = 1e-5
            num = (loss(x64 + h * v, w64) - loss(x64 - h * v, w64)) / (2 * h)
            ana = (dx.double().cpu() * v).sum()
            scale = float(x64.grad.norm() * v.norm())
            assert abs(float(num - ana)) <= 1e-5 * scale
