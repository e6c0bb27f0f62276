"""Gated residual with the norms before and after a block: svgear_block_norm and
its backward against the formulas in 64 bits on the CPU.

Tolerances.  u = 2^-24.  An output is rounded once to its type (half a step:
eps/2 of the type, relative).  Before that every value passes fewer than K = 64
float32 roundings: a row sum adds at most 16 values in a thread, 5 + 5 levels
of a tree and up to 20 warps' totals, the rest are a dozen products and sums.
Each rounding is at most u times the largest magnitude in that step, which the
reference collects beside the values (`mag`).  Column sums add their rows one
by one in the worst case: (K + rows) u of the sum of magnitudes."""
import ctypes
import math

import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv
from clustered_sparse_attention_flash_b200.build import build

torch = pytest.importorskip("torch")

U, K = 2.0 ** -24, 64
KINDS = {"none": sv.SVGEAR_NORM_NONE, "rms": sv.SVGEAR_NORM_RMS, "layer": sv.SVGEAR_NORM_LAYER}
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------- the formulas

def norm_rows(v, kind, eps):
    """(normed rows, 1/deviation, largest magnitude in units of the normed row)."""
    if kind == "none":
        return v, torch.ones_like(v[:, :1]), v.abs().amax(1, keepdim=True)
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    inv = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    n = c * inv
    return n, inv, v.abs().amax(1, keepdim=True) * inv + n.abs().amax(1, keepdim=True)


class Problem:
    def __init__(self, N, D, types=(BF, BF), pre="layer", post="none", cuts=None, G=1, affine=True, mods=True,
                 with_y=True, a=0.75, eps=1e-6, seed=0):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.N, self.D, self.pre, self.post, self.eps = N, D, pre, post, eps
        self.a = a if with_y else 1.0
        self.cuts = cuts if cuts is not None else [i * (N // G) for i in range(G + 1)]
        self.G = len(self.cuts) - 1
        self.x = (rn(N, D) * 2 + rn(1, D)).to(types[0])
        self.y = (rn(N, D) + 0.5 * rn(1, D)).to(types[1]) if with_y else None
        self.gate = rn(self.G, D) if with_y and mods else None
        self.scale, self.shift = (rn(self.G, D) * 0.3, rn(self.G, D)) if mods else (None, None)
        self.weight, self.bias = (1 + 0.2 * rn(D), rn(D)) if affine else (None, None)
        self.post_weight = 1 + 0.2 * rn(D) if affine and with_y else None
        self.dr, self.dh = rn(N, D).to(types[0]), rn(N, D).to(types[1])
        self.offsets = torch.tensor(self.cuts, dtype=torch.int32) if cuts is not None else None
        self.types = types

    def kw(self, dev="cuda"):
        to = lambda t: None if t is None else t.to(dev)  # noqa: E731
        return dict(gate=to(self.gate), scale=to(self.scale), shift=to(self.shift), weight=to(self.weight),
                    bias=to(self.bias), post_weight=to(self.post_weight), pre=KINDS[self.pre], post=KINDS[self.post],
                    eps=self.eps, res_scale=self.a, offsets=to(self.offsets))

    def forward(self):
        kw = self.kw()
        r, h = sv.block_norm(self.x.cuda(), None if self.y is None else self.y.cuda(), dtype=self.types[1], **kw)
        torch.cuda.synchronize()
        return r, h

    def backward(self, dr=True, dh=True):
        kw = self.kw()
        out = sv.block_norm_backward(self.x.cuda(), None if self.y is None else self.y.cuda(),
                                     self.dr.cuda() if dr else None, self.dh.cuda() if dh else None, **kw)
        torch.cuda.synchronize()
        return out

    # -- 64-bit values and magnitudes; rows behind the last group are left out
    def groups(self):
        grp = torch.full((self.N,), -1)
        for i in range(self.G):
            grp[self.cuts[i]:self.cuts[i + 1]] = i
        return grp

    def reference(self, x=None, y=None, params=None):
        P = {n: getattr(self, n) for n in ("gate", "scale", "shift", "weight", "bias", "post_weight")}
        P.update(params or {})
        x = (self.x if x is None else x).double()
        one = torch.ones(self.D, dtype=torch.float64)
        row = lambda t, d: one.expand(self.N, -1) * d if t is None else t.double()[self.groups().clamp_min(0)]  # noqa: E731
        col = lambda t, d: one * d if t is None else t.double()  # noqa: E731
        s, t, g = row(P["scale"], 0.0), row(P["shift"], 0.0), row(P["gate"], 1.0)
        w, b, w2 = col(P["weight"], 1.0), col(P["bias"], 0.0), col(P["post_weight"], 1.0)
        v = dict(s=s, t=t, g=g, w=w, b=b, w2=w2)
        if self.y is not None:
            y = (self.y if y is None else y).double()
            m, inv_m, mag_m = norm_rows(y, self.post, self.eps)
            r = self.a * x + g * m * w2
            mag_r = (self.a * x).abs().amax(1, keepdim=True) + (g * w2).abs().amax(1, keepdim=True) * mag_m
            v.update(m=m, inv_m=inv_m, mag_m=mag_m)
        else:
            r, mag_r = x, x.abs().amax(1, keepdim=True)
        n, inv_n, mag_n = norm_rows(r, self.pre, self.eps)
        mag_n = mag_n + mag_r * inv_n
        A, B = w * (1 + s), b * (1 + s) + t
        v.update(r=r, mag_r=mag_r, n=n, inv_n=inv_n, mag_n=mag_n, A=A, h=n * A + B,
                 mag_h=mag_n * A.abs() + b.abs() * (1 + s.abs()) + t.abs())
        return v

    def reference_backward(self, dr=True, dh=True):
        v = self.reference()
        live = (self.groups() >= 0)[:, None].double()
        DH = self.dh.double() * live if dh else torch.zeros(self.N, self.D, dtype=torch.float64)
        DR = self.dr.double() if dr else 0 * DH

        def through(du, n, inv, mag_n, kind):
            """The norm's Jacobian and the magnitude of what it adds up."""
            if kind == "none":
                return du, du.abs().amax(1, keepdim=True)
            out = du - n * (du * n).mean(1, keepdim=True)
            if kind == "layer":
                out = out - du.mean(1, keepdim=True)
            top = du.abs().amax(1, keepdim=True)
            return out * inv, inv * top * (2 + 2 * mag_n * n.abs().amax(1, keepdim=True) + mag_n ** 2)

        R, mag_R = through(DH * v["A"], v["n"], v["inv_n"], v["mag_n"], self.pre)
        R, mag_R = R + DR, mag_R + (DR.abs().amax(1, keepdim=True) if dr else 0)
        out, mag = {"dx": self.a * R}, {"dx": abs(self.a) * mag_R}
        grp = self.groups()
        sums = lambda t: torch.stack([t[grp == i].sum(0) for i in range(self.G)])  # noqa: E731
        S1, S2 = sums(DH), sums(DH * v["n"])
        M1, M2 = sums(DH.abs()), sums(DH.abs() * v["mag_n"])
        out.update(dshift=S1, dscale=S2 * v["w"] + S1 * v["b"])
        mag.update(dshift=M1, dscale=M2 * v["w"].abs() + M1 * v["b"].abs())
        s1 = 1 + (self.scale.double() if self.scale is not None else torch.zeros(self.G, self.D, dtype=torch.float64))
        out.update(dweight=(s1 * S2).sum(0), dbias=(s1 * S1).sum(0))
        mag.update(dweight=(s1.abs() * M2).sum(0), dbias=(s1.abs() * M1).sum(0))
        if self.y is not None:
            W, MW = sums(R * live * v["m"]), sums(mag_R * live * (v["m"].abs() + v["mag_m"]))
            g = self.gate.double() if self.gate is not None else torch.ones(self.G, self.D, dtype=torch.float64)
            out.update(dgate=W * v["w2"], dpost_weight=(g * W).sum(0))
            mag.update(dgate=MW * v["w2"].abs(), dpost_weight=(g.abs() * MW).sum(0))
            gw = v["g"] * v["w2"]
            dy, mag_dy = through(R * gw, v["m"], v["inv_m"], v["mag_m"], self.post)
            out["dy"] = dy
            mag["dy"] = mag_dy + v["inv_m"] * gw.abs().amax(1, keepdim=True) * mag_R * (2 + v["mag_m"] ** 2)
        return out, mag


def check(name, got, ref, mag, rows=0, live=None):
    got = got.double().cpu()
    lim = (K + rows) * U * (mag + ref.abs())
    lim = lim + HALF[name[1]] * ref.abs() + 1e-37
    if live is not None:
        got, ref, lim = got[live], ref[live], lim[live]
    bad = ~((got - ref).abs() <= lim)
    assert not bad.any(), f"{name[0]}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / lim).max():.3g} of the bound"


HALF = {BF: torch.finfo(BF).eps / 2, F32: torch.finfo(F32).eps / 2}

CASES = [
    dict(N=1, D=8, types=(F32, F32)),
    dict(N=1, D=5120, post="rms"),
    dict(N=3, D=64, pre="rms", post="layer", types=(F32, BF)),
    dict(N=150, D=72, G=3),
    dict(N=701, D=264, cuts=[0, 0, 1, 333, 333, 700, 701], post="layer", types=(F32, F32)),
    dict(N=333, D=256, cuts=[0, 5, 300], pre="rms"),
    dict(N=97, D=128, post="rms", affine=False, types=(F32, BF)),
    dict(N=601, D=1024, G=1, mods=False, pre="rms", post="rms"),
    dict(N=1024, D=2048, G=32, affine=False),
    dict(N=160, D=5120, cuts=[0, 40, 41, 159, 160], post="layer", types=(F32, BF)),
    dict(N=31, D=5128, pre="rms", post="rms", types=(F32, F32)),
    dict(N=449, D=8192, with_y=False, G=1),
    dict(N=1200, D=40, with_y=False, G=1200, types=(F32, F32)),
    dict(N=500, D=2560, with_y=False, pre="rms", affine=False, cuts=[0, 499], types=(F32, BF)),
    dict(N=64, D=512, pre="none", post="none", G=2),
    dict(N=200, D=1536, eps=0.5, post="rms", G=4),
    dict(N=40, D=8192, types=(F32, F32), post="layer", cuts=[0, 13, 40]),
    dict(N=700, D=4096, types=(F32, F32), pre="rms", cuts=[0, 1, 699, 700]),
    dict(N=5003, D=24, cuts=[0, 2, 3, 3, 9, 2500, 2501, 5000], types=(F32, BF), post="rms"),
    dict(N=3001, D=120, pre="rms", cuts=[0, 1500, 3001]),
    dict(N=900, D=640, G=900, affine=False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i):
    p = Problem(**CASES[i], seed=i)
    r, h = p.forward()
    v = p.reference()
    live = p.groups() >= 0
    if p.y is not None:
        check(("r", p.types[0]), r, v["r"], v["mag_r"], live=live)
    check(("h", p.types[1]), h, v["h"], v["mag_h"], live=live)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward(i):
    p = Problem(**CASES[i], seed=100 + i)
    got = p.backward()
    ref, mag = p.reference_backward()
    live = p.groups() >= 0
    rows = int(live.sum())
    for n, t in got.items():
        if t is None:
            continue
        wide = n in ("dx", "dy")
        check((n, {"dx": p.types[0], "dy": p.types[1]}.get(n, F32)), t, ref[n], mag[n], 0 if wide else rows,
              live if wide else None)
    assert (got["dgate"] is None) == (p.gate is None) and (got["dweight"] is None) == (p.weight is None)


@pytest.mark.gpu
@pytest.mark.parametrize("dr,dh", [(True, False), (False, True)])
def test_backward_of_one_output(dr, dh):
    p = Problem(130, 1032, post="rms", G=2, types=(F32, BF), seed=5)
    got = p.backward(dr, dh)
    ref, mag = p.reference_backward(dr, dh)
    for n, t in got.items():
        check((n, {"dx": F32, "dy": BF}.get(n, F32)), t, ref[n], mag[n], 130)


@pytest.mark.gpu
@pytest.mark.parametrize("pre,post", [("layer", "none"), ("rms", "rms"), ("layer", "layer")])
def test_gradients_against_differences(pre, post):
    """<gradient, direction> against central differences of the 64-bit forward."""
    p = Problem(24, 136, types=(F32, F32), pre=pre, post=post, cuts=[0, 7, 24], seed=11)
    got = p.backward()
    g = torch.Generator().manual_seed(3)
    names = {"dx": "x", "dy": "y", "dgate": "gate", "dscale": "scale", "dshift": "shift", "dweight": "weight",
             "dbias": "bias", "dpost_weight": "post_weight"}
    ref, mag = p.reference_backward()
    for gn, pn in names.items():
        base = getattr(p, pn).double()
        v = torch.randn(base.shape, generator=g, dtype=torch.float64)
        step = 1e-5

        def loss(t):
            kw = dict(x=t) if pn == "x" else dict(y=t) if pn == "y" else dict(params={pn: t})
            o = p.reference(**kw)
            return (o["r"] * p.dr.double()).sum() + (o["h"] * p.dh.double()).sum()

        want = (loss(base + step * v) - loss(base - step * v)) / (2 * step)
        have = (got[gn].double().cpu() * v).sum()
        # float32 gradients (their bound, weighted) plus step^2 of the third derivative, far below 1e-6
        lim = ((K + 24) * U * (mag[gn] + ref[gn].abs()) * v.abs()).sum() + 1e-6 * (ref[gn] * v).abs().sum()
        assert abs(have - want) <= lim, (gn, float(have), float(want), float(lim))


@pytest.mark.gpu
def test_rows_behind_the_last_group_are_left_as_they_were():
    p = Problem(60, 1024, cuts=[0, 10, 10, 41], seed=2)
    kw = p.kw()
    x, y = p.x.cuda(), p.y.cuda()
    P, _ = sv._norm_call(x, y, BF, kw["gate"], kw["scale"], kw["shift"], kw["weight"], kw["bias"], kw["post_weight"],
                      kw["pre"], kw["post"], p.eps, p.a, kw["offsets"])
    r, h, dx, dy = (torch.full_like(x, 7.0) for _ in range(4))
    par = (kw["gate"], kw["scale"], kw["shift"], kw["weight"], kw["bias"], kw["post_weight"], kw["offsets"])
    sv.svgear_block_norm(x, y, *par, P, r, h)
    ws = sv.workspace(sv.svgear_block_norm_backward_workspace_size(P))
    dg = [torch.full_like(t, 9.0) for t in par[:6]]
    par_b = par[:2] + par[3:]
    sv.svgear_block_norm_backward(x, y, p.dr.cuda(), p.dh.cuda(), *par_b, P, dx, dy, *dg, ws, ws.numel())
    for t in (r, h, dx, dy):
        assert (t[41:] == 7).all() and not (t[:41] == 7).all(1).any()
    for t in dg[:3]:
        assert (t[1] == 0).all()  # the empty group


@pytest.mark.gpu
def test_zeros_constants_and_a_nan_row():
    x = torch.zeros(4, 640, device="cuda")
    x[1] = 3.0
    x[2] = torch.randn(640, device="cuda")
    x[3] = float("nan")
    shift = torch.randn(1, 640, device="cuda")
    _, h = sv.block_norm(x, shift=shift)
    assert torch.equal(h[0], shift[0]) and torch.equal(h[1], shift[0])
    assert torch.isfinite(h[2]).all() and torch.isnan(h[3]).all()
    _, h = sv.block_norm(x, shift=shift, pre=sv.SVGEAR_NORM_RMS)
    assert torch.equal(h[0], shift[0]) and torch.isfinite(h[2]).all() and torch.isnan(h[3]).all()


@pytest.mark.gpu
def test_residual_only_and_in_place():
    p = Problem(77, 2048, post="rms", seed=9)
    kw = p.kw()
    x, y = p.x.cuda(), p.y.cuda()
    r, h = sv.block_norm(x, y, **kw)
    r2, none = sv.block_norm(x, y, want_h=False, **kw)
    assert none is None and torch.equal(r, r2)
    P, _ = sv._norm_call(x, y, BF, *(kw[n] for n in ("gate", "scale", "shift", "weight", "bias", "post_weight", "pre",
                                                   "post", "eps", "res_scale", "offsets")))
    sv.svgear_block_norm(x, y, *(kw[n] for n in ("gate", "scale", "shift", "weight", "bias", "post_weight", "offsets")),
                         P, x, y)
    assert torch.equal(x, r) and torch.equal(y, h)


@pytest.mark.gpu
def test_same_bits_on_another_stream_and_in_a_graph():
    p = Problem(3000, 1024, cuts=[0, 100, 2999, 3000], post="layer", seed=4)
    kw = p.kw()
    x, y, dr, dh = (t.cuda() for t in (p.x, p.y, p.dr, p.dh))
    ref = sv.block_norm(x, y, **kw), sv.block_norm_backward(x, y, dr, dh, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.block_norm(x, y, stream=s, **kw), sv.block_norm_backward(x, y, dr, dh, stream=s, **kw)
    s.synchronize()
    xs, ys = x.clone().zero_(), y.clone().zero_()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cap = sv.block_norm(xs, ys, **kw), sv.block_norm_backward(xs, ys, dr, dh, **kw)
    xs.copy_(x)
    ys.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    for a in (got, cap):
        assert torch.equal(a[0][0], ref[0][0]) and torch.equal(a[0][1], ref[0][1])
        for n, t in ref[1].items():
            assert torch.equal(a[1][n], t), n
    del graph


@pytest.mark.gpu
def test_more_than_2_to_the_31_elements():
    N, D = 266000, 8192
    x = torch.empty(N, D, dtype=BF, device="cuda").normal_()
    _, h = sv.block_norm(x)
    for rows in (slice(0, 64), slice(N - 64, N)):
        assert torch.equal(h[rows], sv.block_norm(x[rows])[1])


# ------------------------------------------------------------------ refusals

@pytest.mark.gpu
@pytest.mark.parametrize("types", [(BF, BF), (F32, F32), (F32, BF)])
def test_every_width(types):
    """Every number of columns, three rows and more per worker, against 64 bits on the device.  A sum of squares and
    the products of an RMS norm lose no digits, so K u of each term's magnitude bounds what precedes the rounding."""
    N, g = 450, torch.Generator(device="cuda").manual_seed(5)
    half = {BF: 2.0 ** -8, F32: 2.0 ** -24}
    wide = [torch.randn(N, 8192, generator=g, device="cuda") for _ in range(4)]
    mods = [torch.randn(1, 8192, generator=g, device="cuda") * 0.5 for _ in range(3)]
    for D in range(8, 8193, 8):
        x, y, dr, dh = (t[:, :D].to(k).contiguous() for t, k in zip(wide, (types[0], types[1]) * 2))
        gate, scale, shift = (t[:, :D].contiguous() for t in mods)
        kw = dict(gate=gate, scale=scale, pre=sv.SVGEAR_NORM_RMS)
        r, h = sv.block_norm(x, y, shift=shift, **kw)
        back = sv.block_norm_backward(x, y, dr, dh, shift=shift, **kw)
        X, Y, DR, DH, A, S, T = (t.double() for t in (x, y, dr, dh, gate, scale, shift))
        R = X + A * Y
        inv = 1 / torch.sqrt((R * R).mean(1, keepdim=True) + 1e-6)
        n, u = R * inv, DH * (1 + S)
        size = (X.abs() + (A * Y).abs()) * inv  # of the normed row before a and g y may cancel
        dR = DR + inv * (u - n * (u * n).mean(1, keepdim=True))
        mag = DR.abs() + inv * (u.abs() + size * (u * size).abs().mean(1, keepdim=True))
        for name, got, ref, m, k in (("r", r, R, X.abs() + (A * Y).abs(), types[0]),
                                     ("h", h, n * (1 + S) + T, size * (1 + S.abs()) + T.abs(), types[1]),
                                     ("dx", back["dx"], dR, mag, types[0]),
                                     ("dy", back["dy"], dR * A, mag * A.abs(), types[1])):
            over = (got.double() - ref).abs() - (half[k] * ref.abs() + K * U * m)
            assert over.max() <= 0, (name, D, over.max().item())
        for name, ref in (("dscale", DH * n), ("dgate", dR * Y)):
            m = DH.abs() * size if name == "dscale" else mag * Y.abs()
            over = (back[name].double() - ref.sum(0)).abs() - (K + N) * U * m.sum(0)
            assert over.max() <= 0, (name, D, over.max().item())


@pytest.fixture(scope="module")
def L():
    build()
    return sv.lib()


A = 4096  # an aligned non-null address: validation only, nothing runs


def fwd(L, p, **over):
    a = dict(x=A, y=A, gate=A, scale=A, shift=A, weight=A, bias=A, post_weight=A, offsets=A, r=A, h=A)
    a.update(over)
    return L.svgear_block_norm(a["x"], a["y"], a["gate"], a["scale"], a["shift"], a["weight"], a["bias"], a["post_weight"],
                               a["offsets"], ctypes.byref(p) if p else None, a["r"], a["h"], None)


def bwd(L, p, **over):
    names = "x y dr dh gate scale weight bias post_weight offsets".split()
    outs = "dx dy dgate dscale dshift dweight dbias dpost_weight ws".split()
    a = {n: A for n in names + outs}
    a["bytes"] = 1 << 40
    a.update(over)
    return L.svgear_block_norm_backward(*(a[n] for n in names), ctypes.byref(p), *(a[n] for n in outs), a["bytes"], None)


def P(**kw):
    d = dict(N=100, D=64, G=4, pre=2, post=1, eps=1e-6, res_scale=1.0, dtype=sv.SVGEAR_BF16, res_dtype=sv.SVGEAR_BF16)
    d.update(kw)
    return sv.svgear_norm_params(*(d[n] for n, _ in sv.svgear_norm_params._fields_))


def test_refusals_of_parameters(L):
    INV, UNS = sv.SVGEAR_ERR_INVALID, sv.SVGEAR_ERR_UNSUPPORTED
    bad = [(dict(N=0), INV), (dict(D=0), INV), (dict(G=0), INV), (dict(N=-1), INV), (dict(pre=3), INV), (dict(post=-1), INV),
           (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV),
           (dict(res_scale=math.nan), INV), (dict(res_scale=math.inf), INV), (dict(dtype=2), UNS), (dict(res_dtype=-1), UNS),
           (dict(dtype=sv.SVGEAR_F32), UNS), (dict(D=68), UNS), (dict(D=8200), UNS),
           (dict(N=2 ** 30 + 4), UNS)]
    for kw, code in bad:
        assert fwd(L, P(**kw)) == code, kw
        assert bwd(L, P(**kw)) == code, kw
        assert sv.svgear_block_norm_backward_workspace_size(P(**kw)) == 0
    assert fwd(L, None) == INV
    assert L.svgear_block_norm_backward_workspace_size(None) == 0


def test_refusals_of_pointers(L):
    INV = sv.SVGEAR_ERR_INVALID
    for over in (dict(x=None), dict(r=None), dict(x=A + 2), dict(y=A + 8), dict(r=A + 4), dict(h=A + 2), dict(gate=A + 4),
                 dict(scale=A + 4), dict(shift=A + 4), dict(weight=A + 4), dict(bias=A + 4), dict(post_weight=A + 4),
                 dict(offsets=A + 2), dict(y=None), dict(y=None, gate=None, post_weight=None, r=None)):
        assert fwd(L, P(), **over) == INV, over
    assert fwd(L, P(N=101), offsets=None) == INV       # 4 groups do not divide 101 rows
    alone = dict(y=None, gate=None, post_weight=None, r=None)
    assert fwd(L, P(post=0), **{**alone, "r": A}) == INV
    assert fwd(L, P(post=0), **{**alone, "h": None}) == INV
    assert fwd(L, P(post=0, res_scale=0.5), **alone) == INV
    for over in (dict(x=None), dict(dx=None), dict(dy=None), dict(y=None), dict(dr=None, dh=None), dict(dx=A + 2),
                 dict(dgate=A + 4), dict(dh=A + 2)):
        assert bwd(L, P(), **over) == INV, over
    alone = dict(y=None, gate=None, post_weight=None, dy=None)
    assert bwd(L, P(post=0), **alone, dpost_weight=None) == INV   # dgate without y
    need = sv.svgear_block_norm_backward_workspace_size(P())
    assert need > 0
    for over in (dict(ws=None), dict(bytes=need - 1), dict(ws=A + 8)):
        assert bwd(L, P(), **over) == sv.SVGEAR_ERR_WORKSPACE, over


def test_refusals_of_the_binding():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device tensor"):
        sv.block_norm(x)
    with pytest.raises(ValueError, match="dr or dh"):
        sv.block_norm_backward(x, None, None, None)
    with pytest.raises(ValueError, match=r"\[N, D\]"):
        sv.block_norm(x[0])


@pytest.mark.gpu
def test_refusals_of_tensors():
    x = torch.zeros(4, 64, device="cuda")
    y16 = x.bfloat16()
    with pytest.raises(ValueError, match="contiguous"):
        sv.block_norm(x[:, ::2])
    with pytest.raises(ValueError, match="gate"):
        sv.block_norm(x, x, gate=torch.zeros(2, 32, device="cuda"))
    with pytest.raises(ValueError, match="weight"):
        sv.block_norm(x, weight=torch.zeros(64, device="cuda", dtype=BF))
    with pytest.raises(ValueError, match="shift"):
        sv.block_norm(x, scale=torch.zeros(2, 64, device="cuda"), shift=torch.zeros(1, 64, device="cuda"))
    with pytest.raises(ValueError, match="offsets"):
        sv.block_norm(x, offsets=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="y"):
        sv.block_norm(x, x.cpu())
    with pytest.raises(ValueError, match="dtype"):
        sv.block_norm(x, y16, dtype=F32)
    with pytest.raises(sv.SvgearError):
        sv.block_norm(y16, x)
    with pytest.raises(sv.SvgearError):
        sv.block_norm(x, gate=torch.zeros(1, 64, device="cuda"))  # a gate without y
    with pytest.raises(ValueError, match="unsupported"):
        sv.block_norm(x.half())


# ------------------------------------------- rows behind the last group

def test_clear_rest_is_a_known_flag(L):
    INV, flag = sv.SVGEAR_ERR_INVALID, sv.SVGEAR_NORM_CLEAR_REST
    assert sv.svgear_block_norm_backward_workspace_size(P(pre=2 | flag)) == sv.svgear_block_norm_backward_workspace_size(P())
    for kw in (dict(pre=3 | flag), dict(pre=flag << 1), dict(post=1 | flag)):
        assert fwd(L, P(**kw)) == INV and bwd(L, P(**kw)) == INV, kw


@pytest.fixture
def poisoned(monkeypatch):
    """New tensors hold NaN until something writes to them."""
    real = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: real(*a, **k).fill_(math.nan))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [24, 128, 256, 1024, 2560, 5120, 8192])
@pytest.mark.parametrize("types", [(BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("cuts", [[0, 10, 10, 41], [0, 0], [0, 599], [0, 600]])
def test_helpers_clear_the_rows_behind_the_last_group(poisoned, D, types, cuts):
    """The helpers' outputs are new memory, so the rows that no group owns have to be written too; the others are
    those of a call without them."""
    p = Problem(600, D, types=types, cuts=cuts, post="rms", seed=2)
    kw, end = p.kw(), cuts[-1]
    x, y, dr, dh = (t.cuda() for t in (p.x, p.y, p.dr, p.dh))
    for t in (x, y, dr, dh):
        t[end:] = math.nan  # padding: read into nothing
    r, h = sv.block_norm(x, y, **kw)
    got = sv.block_norm_backward(x, y, dr, dh, **kw)
    for t in (r, h, got["dx"], got["dy"]):
        assert (t[end:] == 0).all() and t[:end].isfinite().all()
    assert all(got[n].isfinite().all() for n in got)
    if end:
        short = lambda t: t[:end].contiguous()  # noqa: E731
        r2, h2 = sv.block_norm(short(x), short(y), **kw)
        want = sv.block_norm_backward(short(x), short(y), short(dr), short(dh), **kw)
        assert torch.equal(r[:end], r2) and torch.equal(h[:end], h2)
        assert torch.equal(got["dx"][:end], want["dx"]) and torch.equal(got["dy"][:end], want["dy"])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 2048])
def test_without_a_branch_the_rows_behind_pass_through(poisoned, D):
    """r is x itself, so the gradient of r is that of x where no group is."""
    p = Problem(50, D, types=(F32, BF), cuts=[0, 7, 30], with_y=False, seed=4)
    kw = p.kw()
    x, dr, dh = p.x.cuda(), p.dr.cuda(), p.dh.cuda()
    r, h = sv.block_norm(x, dtype=BF, **kw)
    assert r is x and (h[30:] == 0).all() and h[:30].isfinite().all()
    dx = sv.block_norm_backward(x, None, dr, dh, **kw)["dx"]
    assert torch.equal(dx[30:], dr[30:])
    dx = sv.block_norm_backward(x, None, None, dh, **kw)["dx"]
    assert (dx[30:] == 0).all() and dx.isfinite().all()


# ----------------------------------------------------------- in-place forms

@pytest.mark.gpu
@pytest.mark.parametrize("D", [48, 256, 640, 2048, 5120, 8192])
@pytest.mark.parametrize("types", [(BF, BF), (F32, BF), (F32, F32)])
def test_backward_in_place(D, types):
    """dx in the place of x or of dr, dy in that of y or of dh: the bits of a call with outputs of their own."""
    p = Problem(333, D, types=types, cuts=[0, 5, 5, 300], post="rms", seed=D)
    kw = p.kw()
    want = sv.block_norm_backward(*(t.cuda() for t in (p.x, p.y, p.dr, p.dh)), **kw)
    P_, _ = sv._norm_call(p.x.cuda(), p.y.cuda(), types[1], *(kw[n] for n in (
        "gate", "scale", "shift", "weight", "bias", "post_weight", "pre", "post", "eps", "res_scale", "offsets")))
    ws = sv.workspace(sv.svgear_block_norm_backward_workspace_size(P_))
    par = [kw[n] for n in ("gate", "scale", "weight", "bias", "post_weight", "offsets")]
    for over_x, over_y in ((True, True), (True, False), (False, True), (False, False)):
        x, y, dr, dh = (t.cuda() for t in (p.x, p.y, p.dr, p.dh))
        dx, dy = (x if over_x else dr), (y if over_y else dh)
        sums = [torch.full_like(kw[n], math.nan) for n in ("gate", "scale", "shift", "weight", "bias", "post_weight")]
        sv.svgear_block_norm_backward(x, y, dr, dh, *par, P_, dx, dy, *sums, ws, ws.numel())
        assert torch.equal(dx[:300], want["dx"][:300]) and torch.equal(dy[:300], want["dy"][:300])
        assert torch.equal(dx[300:], (p.x if over_x else p.dr).cuda()[300:])
        assert torch.equal(dy[300:], (p.y if over_y else p.dh).cuda()[300:])
        for t, n in zip(sums, ("dgate", "dscale", "dshift", "dweight", "dbias", "dpost_weight")):
            assert torch.equal(t, want[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("D", [48, 1032, 5120])
@pytest.mark.parametrize("types", [(BF, BF), (F32, F32)])
def test_forward_in_place_without_a_branch(D, types):
    p = Problem(333, D, types=types, with_y=False, G=1, seed=D)
    kw, x = p.kw(), p.x.cuda()
    _, want = sv.block_norm(x, **kw)
    P_, _ = sv._norm_call(x, None, types[1], *(kw[n] for n in (
        "gate", "scale", "shift", "weight", "bias", "post_weight", "pre", "post", "eps", "res_scale", "offsets")))
    sv.svgear_block_norm(x, None, None, kw["scale"], kw["shift"], kw["weight"], kw["bias"], None, None, P_, None, x)
    assert torch.equal(x, want)
