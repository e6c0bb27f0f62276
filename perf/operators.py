"""Workloads of the operators around the sparse attention of a video-DiT layer: the
gated residual with its norms, the rotary positions of Q and K, and the
microscaled 4-bit projections.

`run` computes a case in plain torch operations (`own` false) or through the
library's entry points (`own` true), from the same state.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
DEV = "cuda"


# ------------------------------------------------------------------ cases

def _norm_case(name, back, N, D, G, even, x, y, pre, post, affine, with_y, res_scale):
    return {"name": name, "op": "norm", "back": back, "N": N, "D": D, "G": G, "even": even, "x": x, "y": y,
            "pre": pre, "post": post, "affine": affine, "with_y": with_y, "res_scale": res_scale}


def _rope_case(name, back, B, N, H, d, T, Hh, W, at, ah, aw, half, norm, dtype, explicit):
    return {"name": name, "op": "rope", "back": back, "B": B, "N": N, "H": H, "d": d, "T": T, "Hh": Hh, "W": W,
            "at": at, "ah": ah, "aw": aw, "half": half, "norm": norm, "dtype": dtype, "explicit": explicit}


def _quant_case(name, M, K, head_d, dtype):
    return {"name": name, "op": "quant", "M": M, "K": K, "head_d": head_d, "dtype": dtype}


def _linear_case(name, M, N, K, dtype, bias):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "bias": bias}


def listed():
    return [
        # the conditioning token of a 40-head layer: latency alone counts
        _norm_case("norm one token", False, 1, 5120, 1, True, "bf16", "bf16", "layer", "none", False, True, 1.0),
        # the residual between attention and MLP of a 40-head layer, modulated per latent frame
        _norm_case("norm 75600 tokens", False, 75600, 5120, 21, True, "bf16", "bf16", "layer", "none", False, True, 1.0),
        # a packed batch of seven clips of unequal length, norms on both sides of the block, float32
        _norm_case("norm ragged clips", False, 4999, 2048, 7, False, "f32", "f32", "rms", "rms", True, True, 0.5),
        # fine-tuning step of a 16-head layer on a 32x32x32 grid
        _norm_case("norm backward 32768 tokens", True, 32768, 2048, 32, True, "bf16", "bf16", "layer", "none", False, True, 1.0),
        # one latent frame of 32 x 32 tokens (a frame-by-frame generator)
        _rope_case("rope one frame", False, 1, 1024, 8, 128, 1, 32, 32, 44, 42, 42, False, "head", "bf16", False),
        # two packed samples with given positions, text behind the frames, float32, half-split pairs
        _rope_case("rope given positions", False, 2, 4097, 4, 64, 16, 16, 16, 16, 24, 24, True, "none", "f32", True),
        # Q, K, V of a 40-head layer at 21 x 45 x 80 tokens, norm over the whole token
        _rope_case("rope 75600 tokens", False, 1, 75600, 40, 128, 21, 45, 80, 44, 42, 42, False, "token", "bf16", False),
        # fine-tuning step of a 16-head layer on a 32x32x32 grid
        _rope_case("rope backward 32768 tokens", True, 1, 32768, 16, 128, 32, 32, 32, 44, 42, 42, False, "token", "bf16", False),
        # the attention's head-major output of a 16-head layer, on its way into the output projection
        _quant_case("quantise attention output", 32768, 2048, 128, "bf16"),
        # a short ragged prompt in float32
        _quant_case("quantise prompt", 333, 1056, 0, "f32"),
        # the modulation projection: one time embedding to six vectors of 5120
        _linear_case("linear one token", 1, 30720, 5120, "bf16", True),
        # the QKV projection of a 40-head layer
        _linear_case("linear 75600 tokens", 75600, 15360, 5120, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "quant", "linear"])
    if op == "norm":
        back = rng.random() < 0.4
        D = 8 * _log(rng, 8, 1024)
        N = _log(rng, 1, max(1, min(90000, (128 if back else 256) * 2 ** 20 // D)))
        x, y = rng.choice([("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
        c = _norm_case("", back, N, D, rng.randint(1, min(24, N)), False, x, y, rng.choice(["layer", "rms"]),
                       rng.choice(["none", "rms", "layer"]), rng.random() < 0.5, rng.random() < 0.8, rng.choice([1.0, 0.7]))
        if not c["with_y"]:
            c["post"], c["res_scale"] = "none", 1.0
    elif op == "rope":
        d = rng.choice([64, 128])
        H, B = _log(rng, 1, 48), rng.choice([1, 1, 2, 3])
        Hh, W = rng.randint(1, 45), rng.randint(1, 80)
        T = rng.randint(1, max(1, min(24, (128 * 2 ** 20 // (H * d * B)) // (Hh * W))))
        at = 2 * rng.randint(0, d // 6)
        ah = 2 * rng.randint(1, (d - at) // 4)
        aw = d - at - ah if rng.random() < 0.7 else 2 * rng.randint(1, (d - at - ah) // 2)
        c = _rope_case("", rng.random() < 0.4, B, T * Hh * W + rng.choice([0, 0, 1, 77, 256]), H, d, T, Hh, W, at, ah, aw,
                       rng.random() < 0.4, rng.choice(["none", "head", "token"]), rng.choice(["bf16", "bf16", "f32"]),
                       rng.random() < 0.4)
    elif op == "quant":
        head_d = rng.choice([0, 0, 64, 128])
        K = head_d * rng.randint(1, 48) if head_d else 32 * _log(rng, 1, 256)
        c = _quant_case("", _log(rng, 1, min(80000, 256 * 2 ** 20 // K)), K, head_d, rng.choice(["bf16", "f32"]))
    else:
        K, N = 32 * _log(rng, 2, 256), 8 * _log(rng, 4, 2560)
        c = _linear_case("", _log(rng, 1, max(1, min(75600, 2 ** 40 // (K * N)))), N, K,
                         rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32, mul=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(mul)


def _stream(g, N, D, dtype):
    """Rows as a residual stream has them: unequal channels, a few of them large."""
    ch = torch.exp(_randn(g, (D,), mul=0.5))
    ch[torch.rand(D, generator=g, device=DEV) < 0.01] *= 20
    off = _randn(g, (D,), mul=0.3)
    x = _randn(g, (N, D), dtype)
    x.mul_(ch.to(dtype)).add_(off.to(dtype))
    return x


def _offsets(case, seed):
    """Row offsets of the groups: even ones, or cut at random (some may be empty)."""
    N, G = case["N"], case["G"]
    if case["even"]:
        return None
    cuts = torch.randint(0, N + 1, (G - 1,), generator=torch.Generator().manual_seed(seed)).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), N)]).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "norm":
        N, D, G = case["N"], case["D"], case["G"]
        tx, ty = DT[case["x"]], DT[case["y"]]
        st["x"] = _stream(g, N, D, tx)
        st["y"] = _stream(g, N, D, ty) if case["with_y"] else None
        st["gate"] = _randn(g, (G, D), mul=0.3) if case["with_y"] else None
        st["scale"], st["shift"] = _randn(g, (G, D), mul=0.2), _randn(g, (G, D), mul=0.2)
        aff = case["affine"]
        st["weight"] = 1 + _randn(g, (D,), mul=0.1) if aff else None
        st["bias"] = _randn(g, (D,), mul=0.1) if aff and case["pre"] == "layer" else None
        st["post_weight"] = 1 + _randn(g, (D,), mul=0.1) if aff and case["post"] != "none" else None
        st["offsets"] = _offsets(case, seed)
        if case["back"]:
            st["dh"] = _randn(g, (N, D), ty)
            st["dr"] = _randn(g, (N, D), tx) if case["with_y"] else None
    elif case["op"] == "rope":
        B, N, H, d = case["B"], case["N"], case["H"], case["d"]
        tt = DT[case["dtype"]]
        # one fused projection row: [q | k | v] of all heads
        qkv = _randn(g, (B, N, 3, H, d), tt)
        st["q"], st["k"], st["v"] = qkv.unbind(2)
        P = {"none": 0, "head": d, "token": H * d}[case["norm"]]
        st["wq"], st["wk"] = ((1 + _randn(g, (P,), mul=0.1) for _ in range(2)) if P else (None, None))
        st["positions"] = None
        if case["explicit"]:
            vol = case["T"] * case["Hh"] * case["W"]
            n = torch.arange(N, device=DEV)
            hw = case["Hh"] * case["W"]
            pos = torch.stack([n // hw, n // case["W"] % case["Hh"], n % case["W"]], -1)
            pos[vol:] = 0  # text: no rotation
            first = torch.randint(0, 2000, (B, 1, 1), generator=g, device=DEV)
            pos = pos.expand(B, N, 3) + first * (n < vol)[:, None] * torch.tensor([1, 0, 0], device=DEV)
            st["positions"] = pos.to(torch.int32).contiguous()
        if case["back"]:
            st["dQ"], st["dK"], st["dV"] = (_randn(g, (B * H, N, d), tt) for _ in range(3))
    elif case["op"] == "quant":
        M, K, hd = case["M"], case["K"], case["head_d"]
        x = _stream(g, M, K, DT[case["dtype"]])
        x[torch.rand(M, generator=g, device=DEV) < 0.02] = 0  # rows that a mask emptied
        st["x"] = x.view(M, K // hd, hd).transpose(0, 1).contiguous() if hd else x
    else:
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = _stream(g, M, K, DT[case["dtype"]])
        # a checkpoint's 4-bit weights: packed codes and one exponent per 32
        st["w_codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        st["w_scales"] = torch.randint(116, 122, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        st["bias"] = _randn(g, (N,), mul=0.1) if case["bias"] else None
    return st


# -------------------------------------------------------------- plain form

EPS = 1e-6


def _row_groups(st):
    """The group of every row."""
    c = st["case"]
    if st["offsets"] is None:
        return torch.arange(c["N"], device=DEV) // (c["N"] // c["G"])
    return torch.searchsorted(st["offsets"][1:].long(), torch.arange(c["N"], device=DEV), right=True)


def _normed(v, kind):
    """(normed rows, 1 / deviation)."""
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    inv = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * inv, inv


def _normed_back(du, n, inv, kind):
    if kind == "none":
        return du
    du = du - n * (du * n).mean(-1, keepdim=True) - (du.mean(-1, keepdim=True) if kind == "layer" else 0)
    return du * inv


def _plain_norm(st):
    c = st["case"]
    grp = _row_groups(st)
    x = st["x"].float()
    scale1, w, w2 = 1 + st["scale"], st["weight"], st["post_weight"]
    if c["with_y"]:
        m, inv_m = _normed(st["y"].float(), c["post"])
        gate = st["gate"][grp]
        r = c["res_scale"] * x + gate * (m if w2 is None else m * w2)
    else:
        r = x
    n, inv_n = _normed(r, c["pre"])
    if not c["back"]:
        h = n if w is None else n * w
        h = h if st["bias"] is None else h + st["bias"]
        h = h * scale1[grp] + st["shift"][grp]
        out = {"h": h.to(DT[c["y"]])}
        if c["with_y"]:
            out["r"] = r.to(DT[c["x"]])
        return out
    one = (torch.arange(c["G"], device=DEV)[:, None] == grp).float()  # sums over a group: a product with its indicator
    dh = st["dh"].float()
    S1, S2 = one @ dh, one @ (dh * n)
    u = dh * scale1[grp]
    u = u if w is None else u * w
    R = _normed_back(u, n, inv_n, c["pre"])
    dscale = S2 if w is None else S2 * w
    out = {"dshift": S1, "dscale": dscale if st["bias"] is None else dscale + st["bias"] * S1}
    if w is not None:
        out["dweight"] = (scale1 * S2).sum(0)
    if st["bias"] is not None:
        out["dbias"] = (scale1 * S1).sum(0)
    if c["with_y"]:
        R = R + st["dr"].float()
        U = one @ (R * m)
        out["dgate"] = U if w2 is None else U * w2
        if w2 is not None:
            out["dpost_weight"] = (st["gate"] * U).sum(0)
        dm = R * gate
        out["dy"] = _normed_back(dm if w2 is None else dm * w2, m, inv_m, c["post"]).to(DT[c["y"]])
    out["dx"] = (c["res_scale"] * R).to(DT[c["x"]])
    return out


def _positions(st):
    """[B, N, 3] positions: the given ones, or raster order with zeros behind the grid."""
    c = st["case"]
    if st["positions"] is not None:
        return st["positions"]
    n = torch.arange(c["N"], device=DEV)
    hw = c["Hh"] * c["W"]
    pos = torch.stack([n // hw, n // c["W"] % c["Hh"], n % c["W"]], -1)
    return (pos * (n < c["T"] * hw)[:, None]).expand(c["B"], c["N"], 3)


def _cos_sin(st):
    """cos and sin [B, N, 1, pairs] of every rotated pair; angles in 64 bits."""
    c = st["case"]
    pos = _positions(st).double()
    ang = torch.cat([pos[..., i:i + 1] * 10000.0 ** (-torch.arange(0, a, 2, device=DEV, dtype=torch.float64) / max(a, 1))
                     for i, a in enumerate((c["at"], c["ah"], c["aw"]))], -1)[:, :, None]
    return ang.cos().float(), ang.sin().float()


def _rotate(z, cos, sin, half):
    """Rotates the first pairs of every head of z [..., d] (float32)."""
    d, n = z.shape[-1], cos.shape[-1]
    a, b = (z[..., :d // 2], z[..., d // 2:]) if half else (z[..., 0::2], z[..., 1::2])
    ra = torch.cat([a[..., :n] * cos - b[..., :n] * sin, a[..., n:]], -1)
    rb = torch.cat([a[..., :n] * sin + b[..., :n] * cos, b[..., n:]], -1)
    return torch.cat([ra, rb], -1) if half else torch.stack([ra, rb], -1).flatten(-2)


def _head_norm(x, kind):
    """x [B, N, H, d] over its head or its token: (normed, 1 / rms)."""
    if kind == "none":
        return x, None
    inv = torch.rsqrt(x.square().mean((-1,) if kind == "head" else (-1, -2), keepdim=True) + EPS)
    return x * inv, inv


def _plain_rope(st):
    c = st["case"]
    B, N, H, d = c["B"], c["N"], c["H"], c["d"]
    tt = DT[c["dtype"]]
    cos, sin = _cos_sin(st)
    heads = lambda t: t.transpose(1, 2).reshape(B * H, N, d)  # noqa: E731
    weight = lambda w: w.view(1, 1, -1, d)  # noqa: E731
    if not c["back"]:
        out = {"V": heads(st["v"].float()).to(tt)}
        z, _ = _head_norm(st["q"].float(), c["norm"])
        out["Q"] = heads(_rotate(z if st["wq"] is None else z * weight(st["wq"]), cos, sin, c["half"])).to(tt)
        z, _ = _head_norm(st["k"].float(), c["norm"])
        out["K"] = heads(_rotate(z if st["wk"] is None else z * weight(st["wk"]), cos, sin, c["half"])).to(tt)
        return out
    tokens = lambda t: t.view(B, H, N, d).transpose(1, 2).float()  # noqa: E731
    out = {"dv": tokens(st["dV"]).to(tt)}

    def back(name, x, w, dX):
        dz = _rotate(tokens(dX), cos, -sin, c["half"])
        if w is None:
            out["d" + name] = dz.to(tt)
            return
        n, inv = _head_norm(x.float(), c["norm"])
        dw = (dz * n).sum((0, 1))
        out["dw" + name] = dw.sum(0) if c["norm"] == "head" else dw.flatten()
        u = dz * weight(w)
        mean = (u * n).mean((-1,) if c["norm"] == "head" else (-1, -2), keepdim=True)
        out["d" + name] = ((u - n * mean) * inv).to(tt)

    back("q", st["q"], st["wq"], st["dQ"])
    back("k", st["k"], st["wk"], st["dK"])
    return out


def _plain_quantise(x):
    """(signed values / scale, exponent bytes) of x [M, K] float32 in blocks of 32."""
    M, K = x.shape
    b = x.view(M, K // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)  # floor(log2 amax) - 2
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = torch.ldexp(b, -e)
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5).int())
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.copysign(grid[code], v), (e + 127).squeeze(-1).to(torch.uint8)


def _plain_values(codes, scales):
    """Values [N, K] float32 of packed codes and exponent bytes."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).view(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).view(codes.shape[0], -1)


def _token_major(st):
    """The rows [M, K] of a head-major or plain input."""
    x = st["x"]
    return x.transpose(0, 1).reshape(x.shape[1], -1) if x.dim() == 3 else x


def _plain_quant(st):
    v, e = _plain_quantise(_token_major(st).float())
    values = torch.ldexp(v, e.int()[..., None] - 127)
    return {"values": values.view(st["case"]["M"], -1).to(torch.bfloat16), "scales": e}


def _plain_linear(st):
    v, e = _plain_quantise(st["x"].float())
    a = torch.ldexp(v, e.int()[..., None] - 127).view(st["case"]["M"], -1)
    y = a @ _plain_values(st["w_codes"], st["w_scales"]).T
    return (y if st["bias"] is None else y + st["bias"]).to(torch.bfloat16)


# ------------------------------------------------------- the library's calls

# names of the kinds, as the binding spells them
PRE = {"rms": "SVGEAR_NORM_RMS", "layer": "SVGEAR_NORM_LAYER", "none": "SVGEAR_NORM_NONE"}
QK = {"none": "SVGEAR_QKNORM_NONE", "head": "SVGEAR_QKNORM_HEAD", "token": "SVGEAR_QKNORM_TOKEN"}


def _own(st):
    from clustered_sparse_attention_flash_b200 import svgear as sv
    c = st["case"]
    if c["op"] == "norm":
        args = dict(gate=st["gate"], scale=st["scale"], shift=st["shift"], weight=st["weight"], bias=st["bias"],
                    post_weight=st["post_weight"], pre=getattr(sv, PRE[c["pre"]]), post=getattr(sv, PRE[c["post"]]),
                    eps=EPS, res_scale=c["res_scale"], offsets=st["offsets"])
        if c["back"]:
            got = sv.block_norm_backward(st["x"], st["y"], st["dr"], st["dh"], **args)
            return {k: v for k, v in got.items() if v is not None}
        r, h = sv.block_norm(st["x"], st["y"], dtype=DT[c["y"]], **args)
        return {"h": h, "r": r} if c["with_y"] else {"h": h}
    if c["op"] == "rope":
        args = dict(wq=st["wq"], wk=st["wk"], axes=(c["at"], c["ah"], c["aw"]), grid=(c["T"], c["Hh"], c["W"]),
                    positions=st["positions"], pairing=sv.SVGEAR_PAIR_HALF if c["half"] else sv.SVGEAR_PAIR_ADJACENT,
                    norm=getattr(sv, QK[c["norm"]]), eps=EPS)
        if c["back"]:
            got = sv.qkv_rope_backward(st["dQ"], st["dK"], st["dV"], st["q"], st["k"], **args)
            return {k: v for k, v in got.items() if v is not None}
        Q, K, V = sv.qkv_rope(st["q"], st["k"], st["v"], **args)
        return {"Q": Q, "K": K, "V": V}
    if c["op"] == "quant":
        codes, scales = sv.mx_quantize(st["x"])
        return {"values": sv.mx_dequantize(codes, scales), "scales": scales}
    return sv.mx_linear(st["x"], st["w_codes"], st["w_scales"], st["bias"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "quant": _plain_quant, "linear": _plain_linear}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "norm":
        nd = case["N"] * case["D"]
        ex, ey = ES[case["x"]], ES[case["y"]]
        par = 4 * case["D"] * case["G"] * (3 if case["with_y"] else 2)
        if case["back"]:  # x, dh (y, dr) in, dx (dy) out; the parameters and their gradients
            return {"bytes": nd * (3 * ex + 3 * ey if case["with_y"] else 2 * ex + ey) + 2 * par, "flops": 30 * nd}
        return {"bytes": nd * (2 * ex + 2 * ey if case["with_y"] else ex + ey) + par, "flops": 12 * nd}
    if case["op"] == "rope":
        n = case["B"] * case["N"] * case["H"] * case["d"] * ES[case["dtype"]]
        if case["back"]:
            return {"bytes": n * (6 if case["norm"] == "none" else 8), "flops": 20 * n}
        return {"bytes": n * 6, "flops": 8 * n}
    if case["op"] == "quant":
        mk = case["M"] * case["K"]
        return {"bytes": mk * (ES[case["dtype"]] + 2) + mk // 2 + mk // 32, "flops": 4 * mk}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": M * K * ES[case["dtype"]] + N * K * 17 // 32 + 2 * M * N + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}


# ------------------------------------------------ 64-bit values, written apart

def _exact_stat(v, kind):
    """Mean and deviation of the rows of v."""
    mu = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return mu, ((v - mu) ** 2).mean(1, keepdim=True).add(EPS).sqrt()


def _exact_norm_group(st, c, a, b, g, out):
    """Rows a..b, which are group g's."""
    f = lambda n: None if st[n] is None else st[n][a:b].double()  # noqa: E731
    one = torch.ones(c["D"], device=DEV, dtype=torch.float64)
    par = lambda n: one if st[n] is None else st[n].double()  # noqa: E731
    w, w2, bias = par("weight"), par("post_weight"), 0 if st["bias"] is None else st["bias"].double()
    s, t = 1 + st["scale"][g].double(), st["shift"][g].double()
    r = f("x")
    if c["with_y"]:
        gate, y = st["gate"][g].double(), f("y")
        if c["post"] != "none":
            mu, sd_y = _exact_stat(y, c["post"])
            y = (y - mu) / sd_y
        r = r * c["res_scale"] + y * w2 * gate
    mu, sd = _exact_stat(r, c["pre"])
    n = (r - mu) / sd
    if not c["back"]:
        out["h"][a:b] = (n * w + bias) * s + t
        if c["with_y"]:
            out["r"][a:b] = r
        return
    dh = st["dh"][a:b].double()
    out["dshift"][g] = dh.sum(0)
    out["dscale"][g] = (dh * (n * w + bias)).sum(0)
    if "dweight" in out:
        out["dweight"] += (dh * s * n).sum(0)
    if "dbias" in out:
        out["dbias"] += (dh * s).sum(0)

    def through(d, n, sd, kind):  # the Jacobian of a norm, transposed
        res = d - n * (d * n).mean(1, keepdim=True)
        if kind == "layer":
            res = res - d.mean(1, keepdim=True)
        return res / sd

    R = through(dh * s * w, n, sd, c["pre"])
    if c["with_y"]:
        R = R + st["dr"][a:b].double()
        out["dgate"][g] = (R * y * w2).sum(0)
        if "dpost_weight" in out:
            out["dpost_weight"] += (R * gate * y).sum(0)
        dy = R * gate * w2
        out["dy"][a:b] = dy if c["post"] == "none" else through(dy, y, sd_y, c["post"])
    out["dx"][a:b] = c["res_scale"] * R


def _exact_norm(st):
    c = st["case"]
    N, D, G = c["N"], c["D"], c["G"]
    z = lambda *s: torch.zeros(s, device=DEV, dtype=torch.float64)  # noqa: E731
    names = ["h"] + ["r"] * c["with_y"]
    if c["back"]:
        names = ["dx", "dshift", "dscale"] + ["dy", "dgate"] * c["with_y"]
        names += [n for n, p in (("dweight", "weight"), ("dbias", "bias"), ("dpost_weight", "post_weight")) if st[p] is not None]
    out = {n: z(N, D) if n in ("h", "r", "dx", "dy") else z(D) if n in ("dweight", "dbias", "dpost_weight") else z(G, D)
           for n in names}
    cuts = [g * (N // G) for g in range(G + 1)] if st["offsets"] is None else st["offsets"].tolist()
    for g in range(G):
        if cuts[g + 1] > cuts[g]:
            _exact_norm_group(st, c, cuts[g], cuts[g + 1], g, out)
    return out


def _exact_turn(st, sign):
    """Unit complex numbers [B, N, 1, d/2] by which pairs are multiplied (1 where nothing turns)."""
    c = st["case"]
    B, N = c["B"], c["N"]
    if st["positions"] is None:
        grid = torch.cartesian_prod(*(torch.arange(s, device=DEV) for s in (c["T"], c["Hh"], c["W"]))).view(-1, 3)
        pos = torch.zeros(B, N, 3, device=DEV, dtype=torch.float64)
        pos[:, :grid.shape[0]] = grid.double()
    else:
        pos = st["positions"].double()
    ang = torch.zeros(B, N, 1, c["d"] // 2, device=DEV, dtype=torch.float64)
    at = 0
    for ax, width in enumerate((c["at"], c["ah"], c["aw"])):
        for i in range(width // 2):
            ang[:, :, 0, at] = pos[:, :, ax] * math.exp(-math.log(10000.0) * 2 * i / width)
            at += 1
    return torch.polar(torch.ones_like(ang), sign * ang)


def _exact_rope_one(st, x, w, dX, turn):
    c = st["case"]
    B, N, H, d = c["B"], c["N"], c["H"], c["d"]
    if x is not None:
        x = x.double()
        rms = None
        if c["norm"] == "head":
            rms = ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
        elif c["norm"] == "token":
            rms = ((x ** 2).sum((2, 3), keepdim=True) / (H * d) + EPS).sqrt()
        n = x if rms is None else x / rms
    wt = None if w is None else w.double().view(-1, d)

    def turned(z):
        if c["half"]:
            p = torch.complex(z[..., :d // 2].contiguous(), z[..., d // 2:].contiguous()) * turn
            return torch.cat([p.real, p.imag], -1)
        return torch.view_as_real(torch.view_as_complex(z.reshape(B, N, H, d // 2, 2)) * turn).reshape(B, N, H, d)

    if dX is None:
        return turned(n if wt is None else n * wt).permute(0, 2, 1, 3).reshape(B * H, N, d), None
    dz = turned(dX.double().view(B, H, N, d).permute(0, 2, 1, 3).contiguous())
    if wt is None:
        return dz, None
    dw = torch.einsum("bnhd,bnhd->hd", dz, n)
    u = dz * wt
    dims = (-1,) if c["norm"] == "head" else (2, 3)
    count = d if c["norm"] == "head" else H * d
    return (u - n * ((u * n).sum(dims, keepdim=True) / count)) / rms, dw.sum(0) if c["norm"] == "head" else dw.reshape(-1)


def _exact_rope(st):
    c = st["case"]
    if not c["back"]:
        turn = _exact_turn(st, 1.0)
        V = st["v"].double().permute(0, 2, 1, 3).reshape(c["B"] * c["H"], c["N"], c["d"])
        return {"Q": _exact_rope_one(st, st["q"], st["wq"], None, turn)[0],
                "K": _exact_rope_one(st, st["k"], st["wk"], None, turn)[0], "V": V}
    turn = _exact_turn(st, -1.0)
    out = {"dv": st["dV"].double().view(c["B"], c["H"], c["N"], c["d"]).permute(0, 2, 1, 3)}
    for name, w, dX in (("q", st["wq"], st["dQ"]), ("k", st["wk"], st["dK"])):
        dx, dw = _exact_rope_one(st, st[name], w, dX, turn)
        out["d" + name] = dx
        if dw is not None:
            out["dw" + name] = dw
    return out


def _exact_quantise(x):
    """Values [M, K] in 64 bits: the nearest element of each block's grid, ties to the even code."""
    M, K = x.shape
    out = torch.empty(M, K, device=DEV, dtype=torch.float64)
    bits = torch.empty(M, K // 32, device=DEV, dtype=torch.int64)
    levels = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    rows = max(1, 2 ** 26 // K)
    for a in range(0, M, rows):
        b = x[a:a + rows].double().view(-1, K // 32, 32)
        top = b.abs().amax(-1)
        e = torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 2
        e = e + (2.0 ** (e + 3) <= top) - (2.0 ** (e + 2) > top).double()  # log2's last bit
        e = torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
        u = (b.abs() / 2.0 ** e[..., None]).clamp_max(6.0)
        best, far = torch.zeros_like(u), u.clone()
        for i, lev in enumerate(levels):
            gap = (u - lev).abs()
            take = (gap < far) | ((gap == far) & (i % 2 == 0))
            best, far = torch.where(take, torch.full_like(u, lev), best), torch.where(take, gap, far)
        out[a:a + rows] = (torch.sign(b) * best * 2.0 ** e[..., None]).view(-1, K)
        bits[a:a + rows] = (e + 127).long()
    return out, bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "quant":
        x = st["x"] if st["x"].dim() == 2 else torch.cat(list(st["x"]), 1)
        values, _ = _exact_quantise(x)
        return {"values": values, "scales": None}
    a, _ = _exact_quantise(st["x"])
    c = st["w_codes"]
    code = torch.empty(case["N"], case["K"], device=DEV, dtype=torch.uint8)
    code[:, 0::2], code[:, 1::2] = c % 16, c // 16
    mag, expo, neg = (code % 2).double(), code // 2 % 4, (code // 8).double()
    w = torch.where(expo == 0, mag * 0.5, (1 + mag * 0.5) * 2.0 ** (expo.double() - 1)) * (1 - 2 * neg)
    w *= (2.0 ** (st["w_scales"].double() - 127)).repeat_interleave(32, 1)
    y = a @ w.T
    return y if st["bias"] is None else y + st["bias"].double()
