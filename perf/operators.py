"""Cases of the layer's training-side row movement and of its 4-bit expert path.

Operators, each reached through the library's entry points:

* ``combine_bwd``   the weighted combine's gradient: rows' gradients and the top-k weights' gradients;
* ``gather_bwd``    the gather's gradient: each token's rows summed, the router's dx added;
* ``quant_weights`` expert weights [E, K, N] to MXFP4 (E2M1 elements, one E8M0 scale per 32 along K) and read back;
* ``gather_mxfp4``  token rows gathered by expert and quantised to MXFP4 in one pass, and read back;
* ``ffn_mxfp4``     the experts' FFN on MXFP4 rows and weights.

Plain forms are elementary torch operations in 32 bits, rounded once at the end.
"""
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# The eight magnitudes of E2M1, by code.
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the tiny fp32 layer (top-1, capacity 1.25): a latency-bound training step
        dict(name="combine_bwd tiny", op="combine_bwd", T=256, d=64, E=4, k=1, cf=1.25, skew=0.0, dtype="f32"),
        # the Mixtral-shaped layer's training step
        dict(name="combine_bwd mixtral", op="combine_bwd", T=4096, d=4096, E=8, k=2, cf=0.0, skew=0.0, dtype="bf16"),
        # the fine-grained layer: eight rows a token
        dict(name="combine_bwd fine", op="combine_bwd", T=4096, d=4096, E=256, k=8, cf=0.0, skew=0.0, dtype="bf16"),
        # the capacity-binned layer: skewed load, dropped slots, short rows
        dict(name="gather_bwd capacity", op="gather_bwd", T=16384, d=1024, E=64, k=2, cf=1.0, skew=1.5, dtype="bf16"),
        # the Mixtral-shaped layer, fp32 rows
        dict(name="gather_bwd mixtral f32", op="gather_bwd", T=4096, d=4096, E=8, k=2, cf=0.0, skew=0.0, dtype="f32"),
        # one expert's down projection, as a checkpoint loader quantises expert by expert
        dict(name="quant_weights expert", op="quant_weights", E=1, K=14336, N=4096, dtype="bf16"),
        # a whole layer's expert weights at once
        dict(name="quant_weights layer", op="quant_weights", E=64, K=1024, N=4096, dtype="f32"),
        # a decode step's rows
        dict(name="gather_mxfp4 decode", op="gather_mxfp4", T=48, d=4096, E=8, k=2, cf=0.0, skew=0.0, dtype="bf16"),
        # a prefill's rows
        dict(name="gather_mxfp4 prefill", op="gather_mxfp4", T=16384, d=4096, E=8, k=2, cf=0.0, skew=0.0, dtype="bf16"),
        # a single token through the Mixtral-shaped experts
        dict(name="ffn_mxfp4 token", op="ffn_mxfp4", T=1, d=4096, E=8, k=2, F=14336, cf=0.0, skew=0.0, act="swiglu"),
        # the capacity-binned layer's GELU experts under skew
        dict(name="ffn_mxfp4 capacity", op="ffn_mxfp4", T=16384, d=1024, E=64, k=2, F=4096, cf=1.0, skew=1.5, act="gelu"),
        # the Mixtral-shaped layer's prefill
        dict(name="ffn_mxfp4 mixtral", op="ffn_mxfp4", T=4096, d=4096, E=8, k=2, F=14336, cf=0.0, skew=0.0, act="swiglu"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["combine_bwd", "gather_bwd", "quant_weights", "gather_mxfp4", "ffn_mxfp4"])
    while True:
        if op == "quant_weights":
            c = dict(op=op, E=_log(rng, 1, 64), K=128 * _log(rng, 1, 112), N=128 * _log(rng, 1, 112),
                     dtype=rng.choice(["bf16", "f32"]))
            if c["E"] * c["K"] * c["N"] <= 1 << 28:
                return c
            continue
        E = _log(rng, 1, 256)
        c = dict(op=op, T=_log(rng, 1, 16384), d=128 * _log(rng, 1, 40), E=E, k=rng.randint(1, min(8, E)))
        slots = c["T"] * c["k"]
        c["cf"], c["skew"] = rng.choice([0.0, 0.0, 1.0, 1.25]), rng.choice([0.0, 0.5, 1.5])
        if c["cf"] > 0 and slots < E:
            c["cf"] = 0.0  # a capacity below one row would drop everything
        if op == "ffn_mxfp4":
            c["F"], c["act"] = 128 * _log(rng, 1, 112), rng.choice(["swiglu", "gelu"])
            mats = 3 if c["act"] == "swiglu" else 2
            # within the largest listed case: its products, its expert weights, and the padded plain form
            if slots * c["d"] * c["F"] * mats > 8192 * 4096 * 14336 * 3 // (4 if c["skew"] else 1):
                continue
            if E * c["d"] * c["F"] * mats > 8 * 4096 * 14336 * 3 or E * c["T"] * max(c["d"], c["F"]) > 1 << 31:
                continue
            return c
        c["dtype"] = rng.choice(["bf16", "f32"])
        if c["dtype"] == "f32" and op != "gather_mxfp4":
            c["d"] = 4 * _log(rng, 1, 1100)  # fp32 rows: any multiple of 4
        if slots * c["d"] * (2 if c["dtype"] == "f32" else 1) <= 4096 * 8 * 4096:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _routing(case, g):
    """Top-k picks without repetition and the permutation they give: experts in order, slots in order within an
    expert, each expert cut at its capacity. R is the rows' bound known before the routing; the rows in use end at
    seg[E]."""
    T, E, k = case["T"], case["E"], case["k"]
    score = -torch.log(-torch.log(torch.rand(T, E, device=DEV, generator=g).clamp(1e-7, 1 - 1e-7)))
    score -= case["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    idx = score.topk(k, dim=1).indices.reshape(-1)
    logits = torch.randn(T, k, device=DEV, generator=g)
    w = torch.softmax(logits, 1)
    order = torch.sort(idx, stable=True).indices
    counts = torch.bincount(idx, minlength=E)
    start = counts.cumsum(0) - counts
    cap = int(case["cf"] * (k * T / E)) if case["cf"] > 0 else T * k
    kept = counts.clamp(max=cap)
    seg = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    seg[1:] = kept.cumsum(0)
    es = idx[order]
    rank = torch.arange(T * k, device=DEV) - start[es]
    keep = rank < cap
    s2r = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    s2r[order[keep]] = (seg[es] + rank)[keep].to(torch.int32)
    row_slot = torch.full((_kept_rows(case),), -1, dtype=torch.int32, device=DEV)
    row_slot[:int(seg[-1])] = order[keep].to(torch.int32)
    return dict(w=w, slot_to_row=s2r, row_slot=row_slot, seg=seg.to(torch.int32), R=len(row_slot), most=int(kept.max()))


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "quant_weights":
        w = torch.randn(case["E"], case["K"], case["N"], device=DEV, generator=g).mul_(0.02)
        s["w"] = w.to(DTYPES[case["dtype"]])
        return s
    s.update(_routing(case, g))
    T, d, R = case["T"], case["d"], s["R"]
    randn = lambda *n: torch.randn(*n, device=DEV, generator=g)  # noqa: E731
    if op == "ffn_mxfp4":
        E, F = case["E"], case["F"]
        x = randn(T, d)
        codes, scales = _quantise(x[s["row_slot"].long().clamp(min=0) // case["k"]])
        s["x"], s["xs"] = _pack(codes), _tile_rows(scales, s["seg"], E)
        for name, K, N in (("w1", d, F), ("w3", d, F), ("w2", F, d)):
            if name == "w3" and case["act"] != "swiglu":
                s["w3"] = s["w3s"] = None
                continue
            s[name] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
            s[name + "s"] = torch.empty(E, N * K // 32, dtype=torch.uint8, device=DEV)
            for e in range(E):
                codes, scales = _quantise(randn(N, K).mul_(0.02))
                s[name][e] = _pack(codes)
                s[name + "s"][e] = _tile(scales).reshape(-1)
        return s
    dt = DTYPES[case["dtype"]]
    s["x"] = randn(T, d).to(dt)
    if op != "gather_mxfp4":  # the expert rows' side
        s["rows"] = randn(R, d).to(dt)
    return s


# -------------------------------------------------- MXFP4, elementary torch
def _quantise(v):
    """Codes (0..15) and E8M0 bytes of blocks of 32 along the last axis."""
    b = v.float().unflatten(-1, (-1, 32))
    a = b.abs().amax(-1)
    e = (torch.frexp(a).exponent - 3).clamp(-127, 127)  # floor(log2 a) - 2
    e = torch.where(a == 0, -127, e)
    m = torch.ldexp(b.abs(), -e[..., None])
    code = (m > 0.25).to(torch.uint8)
    for lo, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (m >= lo) if tie_up else (m > lo)
    code += torch.signbit(b).to(torch.uint8) * 8
    finite = torch.isfinite(a)
    scale = torch.where(finite, e + 127, 255).to(torch.uint8)
    return torch.where(finite[..., None], code, 0).flatten(-2).to(torch.uint8), scale


def _values(codes, scales):
    """fp32 values of codes [..., K] and scales [..., K/32]."""
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    s = scales.to(torch.int32)
    f = torch.where(s == 0, 0x400000, s << 23).view(torch.float32)
    f = torch.where(s == 255, float("nan"), f)
    return (lut[codes.int()].unflatten(-1, (-1, 32)) * f[..., None]).flatten(-2)


def _pack(codes):
    """Two codes a byte, the first in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _tile(scales):
    """[..., N, K/32] row-major scales to tiles of 128 rows x 4 blocks, 512 bytes each (row r, block b of a tile at
    byte (r % 32) * 16 + (r / 32) * 4 + b), row tiles outer, block groups inner."""
    n, kb = scales.shape[-2:]
    t = scales.reshape(*scales.shape[:-2], n // 128, 4, 32, kb // 4, 4)
    return t.movedim(-2, -4).transpose(-2, -3).contiguous()


def _untile(t, n, kb):
    t = t.reshape(*t.shape[:-1], n // 128, kb // 4, 32, 4, 4)
    return t.transpose(-2, -3).movedim(-4, -2).reshape(*t.shape[:-5], n, kb)


def _row_place(seg, R):
    """Each row's expert, its rank there and the scale tile that holds it (rows past the last one used go with the
    last expert)."""
    r = torch.arange(R, device=seg.device)
    e = torch.searchsorted(seg[1:].long(), r, right=True).clamp(max=len(seg) - 2)
    first = seg.long()[e]
    rank = r - first
    return e, rank, first // 128 + e + rank // 128


def _tile_rows(scales, seg, E):
    """Row scales [R, K/32] in the library's tiles: expert e's rows start at tile seg[e] / 128 + e."""
    R, kb = scales.shape
    _, rank, tile = _row_place(seg, R)
    t = torch.zeros(R // 128 + E, kb // 4, 32, 4, 4, dtype=torch.uint8, device=scales.device)
    t[tile, :, rank % 32, rank % 128 // 32] = scales.reshape(R, kb // 4, 4)
    return t.reshape(-1)


def _untile_rows(t, seg, R, E, kb):
    _, rank, tile = _row_place(seg, R)
    return t.reshape(R // 128 + E, kb // 4, 32, 4, 4)[tile, :, rank % 32, rank % 128 // 32].reshape(R, kb)


# --------------------------------------------------------------------- run
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quant_weights":
        codes, scales = _quantise(s["w"].transpose(1, 2))
        return _values(codes, scales).to(s["w"].dtype).transpose(1, 2).contiguous()
    T, d, k, R = case["T"], case["d"], case["k"], s["R"]
    slot = s["row_slot"].long().clamp(min=0)
    token = slot // k
    live = (torch.arange(R, device=DEV) < s["seg"][-1])[:, None]  # rows behind the last one stay as they were: zero
    if op == "combine_bwd":
        rows = s["slot_to_row"].long().view(T, k)
        dout = s["x"].float()
        dy = torch.where(live, s["w"].reshape(-1)[slot][:, None] * dout[token], 0).to(s["x"].dtype)
        dots = (s["rows"].float() * dout[token]).sum(-1)
        dw = torch.cat((dots, dots.new_zeros(1)))[torch.where(rows < 0, R, rows)]
        return dy, dw
    if op == "gather_bwd":
        rows = s["slot_to_row"].long().view(T, k)
        padded = torch.cat((s["rows"].float(), s["x"].new_zeros(1, d).float()))
        return (s["x"].float() + padded[torch.where(rows < 0, R, rows)].sum(1)).to(s["x"].dtype)
    if op == "gather_mxfp4":
        return torch.where(live, _values(*_quantise(s["x"][token])), 0).to(s["x"].dtype)
    E, F, C = case["E"], case["F"], s["most"]
    e, rank, _ = _row_place(s["seg"], R)
    at = torch.where(live[:, 0], e * C + rank, E * C)
    up = lambda n, N, K: _values(_unpack(s[n]), _untile(s[n + "s"], N, K // 32))  # noqa: E731
    x = torch.zeros(E * C + 1, d, device=DEV)
    x[at] = _values(_unpack(s["x"]), _untile_rows(s["xs"], s["seg"], R, E, d // 32))
    x = x[:E * C].view(E, C, d)
    h = torch.bmm(x, up("w1", F, d).transpose(1, 2))
    if case["act"] == "swiglu":
        h = h * torch.sigmoid(h) * torch.bmm(x, up("w3", F, d).transpose(1, 2))
    else:
        h = 0.5 * h * (1 + torch.erf(h * 0.5 ** 0.5))
    h = _values(*_quantise(h))
    y = torch.bmm(h, up("w2", d, F).transpose(1, 2)).view(E * C, d)
    return torch.where(live, y[at.clamp(max=E * C - 1)], 0).to(torch.bfloat16)


def _kept(s, abi):
    """What a program keeps between calls: output buffers and the workspace."""
    if "kept" not in s:
        case, op = s["case"], s["case"]["op"]
        u8 = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731
        k = s["kept"] = {}
        nbytes = 256
        if op == "quant_weights":
            E, K, N = case["E"], case["K"], case["N"]
            k["codes"], k["scales"] = u8(E * N * K // 2), u8(abi.moe_mxfp4_weight_scales_size(E, K, N))
            k["out"] = torch.empty_like(s["w"])
        elif op == "combine_bwd":
            k["dy"] = torch.zeros_like(s["rows"])
            k["dw"] = torch.empty(case["T"], case["k"], device=DEV)
        elif op == "gather_bwd":
            k["dx"] = torch.empty_like(s["x"])
        elif op == "gather_mxfp4":
            k["codes"] = u8(s["R"] * case["d"] // 2)
            k["scales"] = u8(abi.moe_mxfp4_row_scales_size(s["R"], case["E"], case["d"]))
            k["out"] = torch.zeros(s["R"], case["d"], dtype=s["x"].dtype, device=DEV)
        else:
            R, d, F, E = s["R"], case["d"], case["F"], case["E"]
            k["h"], k["hs"] = u8(R * F // 2), u8(abi.moe_mxfp4_row_scales_size(R, E, F))
            k["y"] = torch.zeros(R, d, dtype=torch.bfloat16, device=DEV)
            nbytes = abi.moe_expert_ffn_mxfp4_workspace_size(R, d, F, E)
        k["ws"] = u8(max(256, nbytes))
        abi.moe_workspace_init(k["ws"])
    return s["kept"]


def _run_own(s):
    from mixture_experts_routing_route_b200 import _abi as abi
    case, op, b = s["case"], s["case"]["op"], _kept(s, abi)
    if op == "quant_weights":
        E, K, N = case["E"], case["K"], case["N"]
        abi.moe_mxfp4_quantize_weights(s["w"], E, K, N, b["codes"], b["scales"])
        abi.moe_mxfp4_dequantize_weights(b["codes"], b["scales"], E, K, N, b["out"])
        return b["out"]
    T, d, k, E, R = case["T"], case["d"], case["k"], case["E"], s["R"]
    if op == "combine_bwd":
        abi.moe_combine_backward(s["x"], s["rows"], s["w"], s["slot_to_row"], T, d, k, R, b["dy"], b["dw"], b["ws"])
        return b["dy"], b["dw"]
    if op == "gather_bwd":
        abi.moe_gather_backward(s["rows"], s["slot_to_row"], s["x"], T, d, k, R, b["dx"], b["ws"])
        return b["dx"]
    if op == "gather_mxfp4":
        abi.moe_gather_mxfp4(s["x"], T, d, k, s["slot_to_row"], s["seg"], E, R, b["codes"], b["scales"], b["ws"])
        abi.moe_mxfp4_dequantize_rows(b["codes"], b["scales"], s["seg"], E, R, d, b["out"], b["ws"])
        return b["out"]
    act = abi.MOE_ACT_SWIGLU if case["act"] == "swiglu" else abi.MOE_ACT_GELU
    abi.moe_expert_ffn_mxfp4(s["x"], s["xs"], s["w1"], s["w1s"], s["w3"], s["w3s"], s["w2"], s["w2s"], act, R, d,
                             case["F"], E, s["seg"], b["h"], b["hs"], b["y"], b["ws"])
    return b["y"]


# -------------------------------------------------------------------- work
def _kept_rows(case):
    """Rows that take part: all slots, or (with a capacity) at most E * C of them."""
    slots = case["T"] * case["k"]
    if case["cf"] <= 0:
        return slots
    return min(slots, case["E"] * int(case["cf"] * (slots / case["E"])))


def work(case):
    op = case["op"]
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    q = 17 / 32  # bytes of one MXFP4 element with its share of the scale
    if op == "quant_weights":  # read, written as MXFP4, read back, written as values
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": n * (2 * es + 2 * q), "flops": 2 * n}
    T, d, k, R = case["T"], case["d"], case["k"], _kept_rows(case)
    if op == "combine_bwd":
        return {"bytes": es * d * (T + 2 * R) + 12 * T * k, "flops": 3 * R * d}
    if op == "gather_bwd":
        return {"bytes": es * d * (2 * T + R) + 4 * T * k, "flops": R * d}
    if op == "gather_mxfp4":
        return {"bytes": es * d * (min(T, R) + R) + 2 * q * R * d + 4 * R, "flops": 2 * R * d}
    mats = 3 if case["act"] == "swiglu" else 2
    return {"bytes": q * min(case["E"], R) * mats * d * case["F"] + R * d * (q + 2), "flops": 2 * mats * R * d * case["F"]}


# ------------------------------------------------- from the definition, 64 bits
def _nearest64(v):
    """MXFP4 value of every element of v (float64, blocks of 32 along the last axis)."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    x = torch.pow(2.0, torch.floor(torch.log2(torch.where(top == 0, 1.0, top))) - 2)
    x = torch.where(top == 0, 2.0 ** -127, x).clamp(min=2.0 ** -127)
    m = (b / x).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    near = (torch.round(m / step) * step).clamp(max=6.0)
    return (torch.copysign(near, b) * x).reshape(v.shape)


def _read64(packed, scale):
    """float64 values of packed codes [n, K/2] with E8M0 bytes [n, K/32]."""
    nib = torch.empty(packed.shape[0], packed.shape[1] * 2, dtype=torch.float64, device=packed.device)
    for half, c in ((0, packed % 16), (1, packed // 16)):
        c = c.double()
        neg = (c >= 8).double()
        c = c - 8 * neg
        ex = torch.floor(c / 2)
        mant = c - 2 * ex
        mag = torch.where(ex == 0, mant * 0.5, (1 + mant / 2) * torch.pow(2.0, ex - 1))
        nib[:, half::2] = mag * (1 - 2 * neg)
    return nib * torch.pow(2.0, scale.double() - 127).repeat_interleave(32, 1)


def _scale64(tiles, row, K):
    """E8M0 bytes [len(row), K/32] of tiled scales; row: row number counted through the tiles."""
    b = torch.arange(K // 32, device=tiles.device)
    row = row[:, None]
    return tiles[((row // 128) * (K // 128) + b // 4) * 512 + (row % 32) * 16 + (row % 128 // 32) * 4 + b % 4]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quant_weights":
        out = torch.empty(s["w"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            out[e] = _nearest64(s["w"][e].double().t()).t()
        return out
    T, d, k, R = case["T"], case["d"], case["k"], s["R"]
    s2r = s["slot_to_row"].long().view(T, k)
    if op == "combine_bwd":
        dy = torch.zeros(R, d, dtype=torch.float64, device=DEV)
        dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        for j in range(k):
            t = torch.nonzero(s2r[:, j] >= 0)[:, 0]
            r = s2r[t, j]
            up = s["x"][t].double()
            dy[r] = s["w"][t, j].double()[:, None] * up
            dw[t, j] = (up * s["rows"][r].double()).sum(1)
        return dy, dw
    if op == "gather_bwd":
        dx = s["x"].double()
        n = int(s["seg"][-1])
        return dx.index_add_(0, s["row_slot"][:n].long() // k, s["rows"][:n].double())
    if op == "gather_mxfp4":
        n = int(s["seg"][-1])
        out = torch.zeros(R, d, dtype=torch.float64, device=DEV)
        out[:n] = _nearest64(s["x"].double())[s["row_slot"][:n].long() // k]
        return out
    E, F = case["E"], case["F"]
    y = torch.zeros(R, d, dtype=torch.float64, device=DEV)
    seg = s["seg"].tolist()
    for e in range(E):
        a, n = seg[e], seg[e + 1] - seg[e]
        if n == 0:
            continue
        row = (a // 128 + e) * 128 + torch.arange(n, device=DEV)
        x = _read64(s["x"][a:a + n], _scale64(s["xs"], row, d))
        col = torch.arange(max(d, F), device=DEV)
        g = x @ _read64(s["w1"][e], _scale64(s["w1s"][e], col[:F], d)).t()
        if case["act"] == "swiglu":
            h = g / (1 + torch.exp(-g)) * (x @ _read64(s["w3"][e], _scale64(s["w3s"][e], col[:F], d)).t())
        else:
            h = g * 0.5 * torch.erfc(-g / 2 ** 0.5)
        y[a:a + n] = _nearest64(h) @ _read64(s["w2"][e], _scale64(s["w2s"][e], col[:d], F)).t()
    return y
