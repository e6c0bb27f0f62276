"""Norm, rotary positions and head order of Q, K, V: svgear_qkv_rope and its
backward against the formulas in 64 bits on the CPU.

Tolerances.  u = 2^-24.  An output is rounded once to its type (eps/2).  The
angle is reduced in float64 and enters float32 as a fraction of a half-turn:
its cos and sin are within 4 u (rounding of the argument: u pi; sincospi: 2
ulp).  A row sum adds 16 values in a thread and up to 5 + 5 levels, the rest
is fewer than 16 products and sums: K = 48 roundings, each at most u times the
largest magnitude of its step.  A weight's gradient adds its tokens (and
heads) one by one in the worst case: (K + count) u of the sum of magnitudes."""
import ctypes
import math

import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv
from clustered_sparse_attention_flash_b200.build import build

torch = pytest.importorskip("torch")

U, K = 2.0 ** -24, 48
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: torch.finfo(BF).eps / 2, F32: torch.finfo(F32).eps / 2}
NORM = {"none": sv.SVGEAR_QKNORM_NONE, "head": sv.SVGEAR_QKNORM_HEAD, "token": sv.SVGEAR_QKNORM_TOKEN}


class Problem:
    def __init__(self, B, N, H, d, axes, grid=None, pos=None, half=False, norm="none", dtype=BF, origin=(0, 0, 0),
                 theta=(10000.0,) * 3, pos_scale=(1.0,) * 3, eps=1e-6, weights=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.N, self.H, self.d, self.axes, self.grid = B, N, H, d, axes, grid
        self.half, self.norm, self.dtype, self.eps = half, norm, dtype, eps
        self.origin, self.theta, self.pos_scale = origin, theta, pos_scale
        rows = torch.randn(B, N, 3, H, d, generator=g)
        rows = (rows + 0.5 * torch.randn(1, 1, 3, H, d, generator=g)).to(dtype)
        self.q, self.k, self.v = rows.unbind(2)
        self.dQ, self.dK, self.dV = (torch.randn(B * H, N, d, generator=g).to(dtype) for _ in range(3))
        cols = {"none": 0, "head": d, "token": H * d}[norm]
        self.wq, self.wk = ((1 + 0.3 * torch.randn(cols, generator=g) for _ in range(2)) if cols and weights else (None, None))
        if pos == "shared":
            self.pos = torch.randint(-300, 3000, (N, 3), generator=g, dtype=torch.int32)
        elif pos == "batch":
            self.pos = torch.randint(0, 100000, (B, N, 3), generator=g, dtype=torch.int32)
        else:
            self.pos = None

    def kw(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(axes=self.axes, grid=self.grid, positions=c(self.pos), wq=c(self.wq), wk=c(self.wk), origin=self.origin,
                    theta=self.theta, pos_scale=self.pos_scale, norm=NORM[self.norm], eps=self.eps,
                    pairing=sv.SVGEAR_PAIR_HALF if self.half else sv.SVGEAR_PAIR_ADJACENT)

    def fused(self):
        """q, k, v on the GPU as views of one projection."""
        return torch.stack([self.q, self.k, self.v], 2).cuda().unbind(2)

    def angles(self):
        """[B, N, d/2] in 64 bits."""
        B, N = self.B, self.N
        ang = torch.zeros(B, N, self.d // 2, dtype=torch.float64)
        if self.pos is None:
            n = torch.arange(N)
            T, Hh, W = self.grid
            on = (n < T * Hh * W).double()
            Hh, W = max(Hh, 1), max(W, 1)
            xyz = torch.stack([n // (Hh * W), n // W % Hh, n % W], -1).double()
            p = xyz.expand(B, N, 3)
        else:
            p, on = self.pos.double().expand(B, N, 3), torch.ones(N, dtype=torch.float64)
        at = 0
        for a in range(3):
            for i in range(self.axes[a] // 2):
                f32 = lambda x: float(torch.tensor(x, dtype=F32))  # noqa: E731  (the call takes float32 bases)
                f = f32(self.pos_scale[a]) * f32(self.theta[a]) ** (-2.0 * i / self.axes[a])
                ang[:, :, at] = (p[:, :, a] + self.origin[a]) * f * on
                at += 1
        return ang

    def turn(self, z, sign=1):
        """z [B, N, H, d] by the angles."""
        c, s = (t[:, :, None] for t in (self.angles().cos(), sign * self.angles().sin()))
        out = torch.empty_like(z)
        if self.half:
            h = self.d // 2
            a, b = z[..., :h], z[..., h:]
            out[..., :h], out[..., h:] = a * c - b * s, a * s + b * c
        else:
            a, b = z[..., 0::2], z[..., 1::2]
            out[..., 0::2], out[..., 1::2] = a * c - b * s, a * s + b * c
        return out

    def normed(self, x):
        x = x.double()
        if self.norm == "none":
            return x, None
        dims = (-1,) if self.norm == "head" else (-1, -2)
        inv = 1 / torch.sqrt((x * x).mean(dims, keepdim=True) + self.eps)
        return x * inv, inv

    def weight(self, w):
        return 1.0 if w is None else w.double().view(-1, self.d)

    def heads(self, x):
        return x.permute(0, 2, 1, 3).reshape(self.B * self.H, self.N, self.d)

    def reference(self, x, w):
        return self.heads(self.turn(self.normed(x)[0] * self.weight(w)))

    def pair_mag(self, z):
        """|a| + |b| of every pair, at both places."""
        z = z.abs()
        if self.half:
            m = z[..., :self.d // 2] + z[..., self.d // 2:]
            return torch.cat([m, m], -1)
        return (z[..., 0::2] + z[..., 1::2]).repeat_interleave(2, -1)

    def reference_backward(self, x, w, dX):
        dz = self.turn(dX.double().view(self.B, self.H, self.N, self.d).permute(0, 2, 1, 3), -1)
        mag = self.pair_mag(dz)
        if self.norm == "none":
            return dz, mag, None, None
        n, inv = self.normed(x)
        dims = (-1,) if self.norm == "head" else (-1, -2)
        wt = self.weight(w)
        u = dz * wt
        dx = inv * (u - n * (u * n).mean(dims, keepdim=True))
        top = (mag * (wt if w is None else wt.abs())).amax(dims, keepdim=True)
        mag_dx = inv * top * (2 + 2 * n.abs().amax(dims, keepdim=True) * n.abs())
        dw, mag_dw = (dz * n).sum((0, 1)), (mag * n.abs()).sum((0, 1))
        if self.norm == "head":
            dw, mag_dw = dw.sum(0), mag_dw.sum(0)
        return dx, mag_dx, dw.flatten(), mag_dw.flatten()


def check(name, got, ref, mag, dtype, count=0):
    got = got.double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    lim = (K + count) * U * (mag + ref.abs()) + HALF[dtype] * ref.abs() + 1e-37
    bad = ~((got - ref).abs() <= lim)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / lim).max():.3g} of the bound"


CASES = [
    dict(B=1, N=1, H=1, d=64, axes=(16, 24, 24), grid=(1, 1, 1)),
    dict(B=1, N=1, H=40, d=128, axes=(44, 42, 42), pos="shared", norm="token"),
    dict(B=1, N=210, H=3, d=64, axes=(20, 22, 22), grid=(3, 7, 10), norm="head", dtype=F32),
    dict(B=1, N=290, H=8, d=128, axes=(44, 42, 42), grid=(3, 8, 11), norm="head", half=True),
    dict(B=3, N=57, H=5, d=128, axes=(32, 48, 48), pos="batch", norm="token", dtype=F32),
    dict(B=2, N=133, H=2, d=64, axes=(0, 32, 32), pos="shared", half=True, dtype=F32),
    dict(B=1, N=75, H=1, d=128, axes=(16, 56, 56), grid=(3, 5, 5), norm="token", half=True),
    dict(B=2, N=33, H=16, d=128, axes=(16, 16, 16), grid=(2, 4, 4), norm="token"),
    dict(B=1, N=40, H=128, d=128, axes=(44, 42, 42), grid=(1, 5, 8), norm="token"),
    dict(B=1, N=40, H=256, d=64, axes=(16, 24, 24), grid=(1, 5, 8), norm="head", dtype=F32),
    dict(B=1, N=64, H=7, d=64, axes=(64, 0, 0), grid=(64, 1, 1), norm="head", origin=(1000000, 0, 0)),
    dict(B=1, N=3000, H=4, d=128, axes=(44, 42, 42), grid=(30, 10, 10), norm="token", weights=False,
         theta=(256.0, 10000.0, 500.0), pos_scale=(0.5, 1.0, 2.25), origin=(5, -7, 0)),
    dict(B=1, N=12, H=2, d=64, axes=(0, 0, 0), grid=(0, 0, 0), norm="none"),
    dict(B=1, N=100, H=2, d=64, axes=(16, 24, 24), grid=(4, 5, 5), norm="head", eps=0.5, dtype=F32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i):
    p = Problem(**CASES[i], seed=i)
    q, k, v = p.fused()
    Q, K_, V = sv.qkv_rope(q, k, v, **p.kw())
    torch.cuda.synchronize()
    for name, got, x, w in (("Q", Q, p.q, p.wq), ("K", K_, p.k, p.wk)):
        n, _ = p.normed(x)
        check(name, got, p.reference(x, w), p.heads(p.pair_mag(n * p.weight(w))), p.dtype)
    assert torch.equal(V.cpu(), p.heads(p.v))


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)))
def test_backward(i):
    p = Problem(**CASES[i], seed=50 + i)
    q, k, _ = p.fused()
    got = sv.qkv_rope_backward(p.dQ.cuda(), p.dK.cuda(), p.dV.cuda(), q, k, **p.kw())
    torch.cuda.synchronize()
    count = p.B * p.N * (p.H if p.norm == "head" else 1)
    for name, x, w, dX in (("q", p.q, p.wq, p.dQ), ("k", p.k, p.wk, p.dK)):
        dx, mag, dw, mag_dw = p.reference_backward(x, w, dX)
        check("d" + name, got["d" + name], dx, mag, p.dtype)
        assert (got["dw" + name] is None) == (w is None)
        if w is not None:
            check("dw" + name, got["dw" + name], dw, mag_dw, F32, count)
    assert torch.equal(got["dv"].cpu(), p.dV.view(p.B, p.H, p.N, p.d).permute(0, 2, 1, 3))


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ["none", "head", "token"])
def test_gradients_against_differences(norm):
    p = Problem(2, 9, 3, 64, (16, 24, 24), pos="batch", norm=norm, dtype=F32, half=norm == "head", seed=8)
    q, k, _ = p.fused()
    got = sv.qkv_rope_backward(p.dQ.cuda(), None, None, q, None, **p.kw())
    g = torch.Generator().manual_seed(1)
    step = 1e-5
    dx, mag, dw, mag_dw = p.reference_backward(p.q, p.wq, p.dQ)
    for name, base, m, r in (("dq", p.q, mag, dx), ("dwq", p.wq, mag_dw, dw)):
        if base is None:
            continue
        v = torch.randn(base.shape, generator=g, dtype=torch.float64)
        f = (lambda t: p.reference(t, p.wq)) if name == "dq" else (lambda t: p.reference(p.q, t))
        want = ((f(base.double() + step * v) - f(base.double() - step * v)) * p.dQ.double()).sum() / (2 * step)
        have = (got[name].double().cpu() * v).sum()
        lim = ((K + 54) * U * (m + r.abs()) * v.abs()).sum() + 1e-6 * (r * v).abs().sum()
        assert abs(have - want) <= lim, (name, float(have), float(want), float(lim))


@pytest.mark.gpu
def test_parts_of_a_joint_sequence_leave_the_other_rows():
    p = Problem(1, 60, 6, 128, (44, 42, 42), grid=(3, 4, 5), norm="head", seed=3)
    t = Problem(1, 11, 6, 128, (44, 42, 42), grid=(0, 0, 0), norm="head", seed=4)
    out = tuple(torch.full((6, 80, 128), 7.0, dtype=BF, device="cuda") for _ in range(3))
    sv.qkv_rope(*p.fused(), out=out, out_at=2, **p.kw())
    sv.qkv_rope(*t.fused(), out=out, out_at=62, **t.kw())
    for o, a, b in zip(out, sv.qkv_rope(*p.fused(), **p.kw()), sv.qkv_rope(*t.fused(), **t.kw())):
        assert torch.equal(o[:, 2:62], a) and torch.equal(o[:, 62:73], b)
        assert (o[:, :2] == 7).all() and (o[:, 73:] == 7).all()


@pytest.mark.gpu
def test_one_of_the_three_and_other_layouts():
    p = Problem(2, 45, 4, 64, (16, 24, 24), grid=(1, 5, 9), norm="token", dtype=F32, seed=6)
    q, k, v = p.fused()
    ref = sv.qkv_rope(q, k, v, **p.kw())
    got = sv.qkv_rope(None, k, None, **p.kw())
    assert got[0] is None and got[2] is None and torch.equal(got[1], ref[1])
    dense = sv.qkv_rope(q.contiguous(), k.contiguous(), v.contiguous(), **p.kw())
    assert all(torch.equal(a, b) for a, b in zip(dense, ref))
    one = sv.qkv_rope(q[1], k[1], v[1], **p.kw())  # [N, H, d]
    assert all(torch.equal(a, b[4:]) for a, b in zip(one, ref))
    wide = torch.zeros(2, 45, 5, 4, 64, device="cuda")
    wide[:, :, 1] = q
    assert torch.equal(sv.qkv_rope(wide[:, :, 1], None, None, **p.kw())[0], ref[0])
    dQ, dK, dV = (t.cuda() for t in (p.dQ, p.dK, p.dV))
    full = sv.qkv_rope_backward(dQ, dK, dV, q, k, **p.kw())
    part = sv.qkv_rope_backward(None, dK, None, None, k.contiguous(), **p.kw())
    assert part["dq"] is None and torch.equal(part["dk"], full["dk"]) and torch.equal(part["dwk"], full["dwk"])
    kw = {**p.kw(), "norm": sv.SVGEAR_QKNORM_NONE, "wq": None, "wk": None}
    alone = sv.qkv_rope_backward(dQ, None, dV, H=4, **kw)
    assert torch.equal(alone["dv"], full["dv"]) and alone["dq"].shape == (2, 45, 4, 64)


@pytest.mark.gpu
def test_turning_back_is_the_inverse():
    """The backward pass of the forward's output gives the input back (a rotation's transpose is its inverse)."""
    p = Problem(1, 300, 2, 128, (44, 42, 42), pos="shared", dtype=F32, seed=1)
    q, k, v = p.fused()
    back = sv.qkv_rope_backward(*sv.qkv_rope(q, k, v, **p.kw()), H=2, **p.kw())
    for a, b in ((back["dq"], q), (back["dk"], k)):
        lim = 2 * K * U * p.pair_mag(b.double().cpu())  # both ways
        assert ((a.double() - b.double()).abs().cpu() <= lim + 1e-30).all()
    assert torch.equal(back["dv"], v)


@pytest.mark.gpu
def test_same_bits_on_another_stream_and_in_a_graph():
    p = Problem(1, 2000, 5, 64, (16, 24, 24), grid=(20, 10, 10), norm="token", seed=2)
    q, k, v = p.fused()
    kw = p.kw()
    grads = tuple(t.cuda() for t in (p.dQ, p.dK, p.dV))
    ref = sv.qkv_rope(q, k, v, **kw), sv.qkv_rope_backward(*grads, q, k, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.qkv_rope(q, k, v, stream=s, **kw), sv.qkv_rope_backward(*grads, q, k, stream=s, **kw)
    s.synchronize()
    qs = torch.zeros_like(q)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cap = sv.qkv_rope(qs, k, v, **kw), sv.qkv_rope_backward(*grads, qs, k, **kw)
    qs.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    for a in (got, cap):
        assert all(torch.equal(x, y) for x, y in zip(a[0], ref[0]))
        assert all(torch.equal(a[1][n], ref[1][n]) for n in ref[1])
    del graph


@pytest.mark.gpu
def test_nan_and_zero_tokens_stay_in_their_rows():
    p = Problem(1, 8, 4, 64, (16, 24, 24), grid=(2, 2, 2), norm="token", dtype=F32, seed=2)
    q, k, v = p.fused()
    ref = sv.qkv_rope(q, k, v, **p.kw())[0]
    q[0, 3] = float("nan")
    q[0, 5] = 0
    Q = sv.qkv_rope(q, k, v, **p.kw())[0]
    rest = [n for n in range(8) if n not in (3, 5)]
    assert torch.equal(Q[:, rest], ref[:, rest]) and torch.isnan(Q[:, 3]).all() and (Q[:, 5] == 0).all()


# ------------------------------------------------------------------ refusals

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["none", "head", "token"])
def test_every_head_count(d, dtype, norm):
    """Every number of heads, there and back.  Without a norm the way back restores the rows: each way is within
    eps/2 + K u of a pair's magnitude."""
    N, g = 450, torch.Generator(device="cuda").manual_seed(6)
    axes, grid = ((16, 24, 24) if d == 64 else (44, 42, 42)), (2, 15, 15)
    wide = torch.randn(N, 16384 // d, d, generator=g, device="cuda").to(dtype)
    w = 1 + 0.3 * torch.randn(16384, generator=g, device="cuda")
    for H in range(1, 16384 // d + 1):
        x = wide[:, :H].contiguous()
        cols = {"none": None, "head": d, "token": H * d}[norm]
        kw = dict(axes=axes, grid=grid, norm=NORM[norm], wq=None if cols is None else w[:cols].contiguous())
        Q, Km, V = sv.qkv_rope(x, x, x, **kw)
        assert torch.equal(V, x.transpose(0, 1)), H
        back = sv.qkv_rope_backward(Q, Km, V, x, x, **kw)
        assert torch.equal(back["dv"], x), H
        if norm == "none":
            lim = 2 * (HALF[dtype] + K * U) * 2 * x.double().abs().amax()
            assert (back["dq"].double() - x.double()).abs().max() <= lim and torch.equal(back["dq"], back["dk"]), H
        else:
            X = x.double()
            inv = 1 / torch.sqrt((X * X).mean((-1,) if norm == "head" else (-2, -1), keepdim=True) + 1e-6)
            W = (w[:cols].view(1, 1, d) if norm == "head" else w[:cols].view(1, H, d)).double()
            size = (Q.double() ** 2).sum(-1)  # a rotation keeps a head's length
            ref = ((X * inv * W) ** 2).sum(-1).T
            assert ((size - ref).abs() <= (2 * HALF[dtype] * 1.01 + 2 * K * U) * 2 * ref).all(), H
            assert back["dq"].isfinite().all() and back["dwq"].isfinite().all() and back["dwk"] is None, H


@pytest.fixture(scope="module")
def L():
    build()
    return sv.lib()


A = 4096  # an aligned non-null address: validation only, nothing runs


def P(**kw):
    d = dict(B=2, N=60, H=4, d=64, axes=(16, 24, 24), grid=(3, 4, 5), dtype=sv.SVGEAR_BF16, norm=sv.SVGEAR_QKNORM_HEAD)
    rest = {n: kw.pop(n) for n in ("ld", "batch", "grad_ld", "grad_batch") if n in kw}
    d.update(kw)
    p = sv.rope_params(**d)
    for n, v in rest.items():
        if n in ("ld", "batch"):
            getattr(p, n)[0] = v
        else:
            setattr(p, n, v)
    return p


def fwd(L, p, **over):
    a = {n: A for n in "q k v wq wk positions Q K V".split()}
    a["positions"] = None
    a.update(over)
    return L.svgear_qkv_rope(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["positions"], ctypes.byref(p), a["Q"], a["K"], a["V"], None)


def bwd(L, p, **over):
    first, last = "dQ dK dV q k wq wk positions".split(), "dq dk dv dwq dwk ws".split()
    a = {n: A for n in first + last}
    a.update(positions=None, bytes=1 << 40)
    a.update(over)
    return L.svgear_qkv_rope_backward(*(a[n] for n in first), ctypes.byref(p), *(a[n] for n in last), a["bytes"], None)


def test_refusals_of_parameters(L):
    INV, UNS = sv.SVGEAR_ERR_INVALID, sv.SVGEAR_ERR_UNSUPPORTED
    bad = [(dict(B=0), INV), (dict(N=0), INV), (dict(H=0), INV), (dict(axes=(15, 24, 24)), INV), (dict(axes=(-2, 24, 24)), INV),
           (dict(axes=(24, 24, 24)), INV), (dict(axes=(2 ** 31 - 2, 24, 24)), INV), (dict(grid=(-1, 4, 5)), INV),
           (dict(grid=(4, 4, 5)), INV), (dict(grid=(65536, 65536, 65536)), INV), (dict(theta=0.0), INV),
           (dict(theta=math.inf), INV), (dict(theta=math.nan), INV), (dict(pos_scale=math.inf), INV), (dict(pairing=2), INV),
           (dict(norm=3), INV), (dict(eps=0.0), INV), (dict(eps=math.nan), INV), (dict(out_tokens=59), INV),
           (dict(out_tokens=-1), INV), (dict(dtype=5), UNS), (dict(d=96), UNS), (dict(H=257), UNS),
           (dict(B=2 ** 20, N=2 ** 12), UNS), (dict(ld=260), INV), (dict(ld=128), INV), (dict(batch=4), INV),
           (dict(norm=0), INV)]  # the last: weights without a norm
    for kw, code in bad:
        assert fwd(L, P(**kw)) == code, kw
        if "ld" not in kw:
            assert bwd(L, P(**kw)) == code, kw
    for kw in (dict(grad_ld=128), dict(grad_ld=260), dict(grad_batch=12)):
        assert bwd(L, P(**kw)) == INV, kw
    assert sv.svgear_qkv_rope_backward_workspace_size(P(d=96)) == 0
    assert sv.svgear_qkv_rope_backward_workspace_size(P(norm=0)) == 0
    assert L.svgear_qkv_rope_backward_workspace_size(None) == 0


def test_refusals_of_pointers(L):
    INV = sv.SVGEAR_ERR_INVALID
    for over in (dict(q=None), dict(Q=None), dict(V=None), dict(q=None, k=None, v=None, Q=None, K=None, V=None), dict(q=A + 8),
                 dict(K=A + 2), dict(wq=A + 4), dict(positions=A + 2)):
        assert fwd(L, P(), **over) == INV, over
    for over in (dict(dq=None), dict(dQ=None), dict(q=None), dict(k=None), dict(dQ=A + 8), dict(dwq=A + 4),
                 dict(dQ=None, dK=None, dV=None, dq=None, dk=None, dv=None), dict(dQ=None, dq=None)):
        assert bwd(L, P(), **over) == INV, over
    need = sv.svgear_qkv_rope_backward_workspace_size(P())
    assert need > 0
    for over in (dict(ws=None), dict(ws=A + 8), dict(bytes=need - 1)):
        assert bwd(L, P(), **over) == sv.SVGEAR_ERR_WORKSPACE, over


def test_refusals_of_the_binding():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="one of q, k, v"):
        sv.qkv_rope(None, None, None, axes=(16, 24, 24))
    with pytest.raises(ValueError, match="device tensor"):
        sv.qkv_rope(x, None, None, axes=(16, 24, 24))
    with pytest.raises(ValueError, match="one of dQ"):
        sv.qkv_rope_backward(None, None, None, axes=(16, 24, 24))
    with pytest.raises(ValueError, match="three entries"):
        sv.rope_params(1, 1, 1, 64, (32, 32))


@pytest.mark.gpu
def test_refusals_of_tensors():
    x = torch.zeros(4, 2, 64, device="cuda")
    ax = dict(axes=(16, 24, 24), grid=(1, 2, 2))
    with pytest.raises(ValueError, match="k"):
        sv.qkv_rope(x, x.bfloat16(), x, **ax)
    with pytest.raises(ValueError, match="dense"):
        sv.qkv_rope(x.transpose(1, 2).contiguous().transpose(1, 2), None, None, **ax)
    with pytest.raises(ValueError, match="wq"):
        sv.qkv_rope(x, x, x, norm=sv.SVGEAR_QKNORM_HEAD, wq=torch.ones(128, device="cuda"), **ax)
    with pytest.raises(ValueError, match="positions"):
        sv.qkv_rope(x, x, x, positions=torch.zeros(4, 3, device="cuda"), **ax)
    with pytest.raises(ValueError, match="fit"):
        sv.qkv_rope(x, None, None, out=(torch.zeros(2, 5, 64, device="cuda"), None, None), out_at=2, **ax)
    with pytest.raises(ValueError, match="with a norm"):
        sv.qkv_rope_backward(torch.zeros(2, 4, 64, device="cuda"), None, None, norm=sv.SVGEAR_QKNORM_HEAD, H=2, **ax)
    with pytest.raises(ValueError, match="H:"):
        sv.qkv_rope_backward(torch.zeros(2, 4, 64, device="cuda"), None, None, **ax)
    with pytest.raises(sv.SvgearError):
        sv.qkv_rope(x[:, :, :32].contiguous(), None, None, axes=(8, 8, 8), grid=(1, 2, 2))
    with pytest.raises(ValueError, match="unsupported"):
        sv.qkv_rope(x.half(), None, None, **ax)


@pytest.mark.gpu
@pytest.mark.parametrize("d,heads", [(64, (1, 3, 9, 19, 33)), (128, (1, 3, 5, 9, 18, 51))])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_infinity_stays_in_its_column_of_the_weight_gradient(d, heads, dtype):
    """A head with one infinite element has an infinite norm: its other elements normalise to zero and add nothing
    to the weight's gradient, whatever the number of heads leaves idle in the last warp."""
    axes = (16, 24, 24) if d == 64 else (44, 42, 42)
    for H in heads:
        g = torch.Generator(device="cuda").manual_seed(H)
        q = torch.randn(40, H, d, generator=g, device="cuda").to(dtype)
        dQ = torch.randn(H, 40, d, generator=g, device="cuda").to(dtype)
        w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        kw = dict(axes=axes, grid=(1, 5, 8), norm=NORM["head"], wq=w)
        without = dQ.clone()
        without[0, 7] = 0  # that head's gradient
        want = sv.qkv_rope_backward(without, None, None, q, None, **kw)
        q[7, 0, 0] = math.inf
        got = sv.qkv_rope_backward(dQ, None, None, q, None, **kw)
        assert torch.equal(got["dwq"][1:], want["dwq"][1:]) and got["dwq"][0].isnan(), H
        rest = torch.ones(40, H, dtype=torch.bool, device="cuda")
        rest[7, 0] = False
        assert torch.equal(got["dq"][rest], want["dq"][rest]), H


def test_overlapping_gradient_rows_are_refused(L):
    """Two tokens' rows of an output that share memory would be written in no order.  All strides of a small grid
    against a list of the rows: a layout that is taken gets as far as the missing workspace."""
    W = 64
    taken = 0
    for B in (1, 2, 3, 4):
        for N in (1, 2, 3, 5):
            for ld in range(W, 7 * W, W // 2):
                for batch in range(W, 12 * W, W // 2):
                    starts = sorted(b * batch + n * ld for b in range(B) for n in range(N))
                    apart = all(y - x >= W for x, y in zip(starts, starts[1:]))
                    p = P(B=B, N=N, H=1, d=W, grid=(1, 1, 1), grad_ld=ld, grad_batch=batch)
                    assert bwd(L, p, ws=None) == (sv.SVGEAR_ERR_WORKSPACE if apart else sv.SVGEAR_ERR_INVALID), (B, N, ld, batch)
                    taken += apart
    assert taken > 1000
    for ld, batch in ((2 ** 62, 2 ** 62), (2 ** 62, W), (W, 2 ** 62)):  # no overflow on the way
        assert bwd(L, P(B=3, N=3, H=1, d=W, grid=(1, 1, 1), grad_ld=ld, grad_batch=batch), ws=None) == (
            sv.SVGEAR_ERR_INVALID if ld == batch else sv.SVGEAR_ERR_WORKSPACE)


@pytest.mark.gpu
def test_interleaved_gradient_rows():
    """Rows of two batch entries between one another, as strides that are neither nested way round allow."""
    W, N = 64, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    dQ = torch.randn(2, N, W, generator=g, device="cuda").to(BF)
    p = sv.rope_params(2, N, 1, W, (16, 24, 24), (1, 1, 3), grad_ld=2 * W, grad_batch=3 * W)
    out = torch.full((9, W), 7.0, dtype=BF, device="cuda")  # rows 0, 2, 4 and 3, 5, 7
    sv.svgear_qkv_rope_backward(dQ, None, None, None, None, None, None, None, p, out, None, None, None, None, None, 0)
    want = sv.qkv_rope_backward(dQ, None, None, H=1, axes=(16, 24, 24), grid=(1, 1, 3))["dq"]
    assert torch.equal(out[[0, 2, 4]], want[0, :, 0]) and torch.equal(out[[3, 5, 7]], want[1, :, 0])
    assert (out[[1, 6, 8]] == 7).all()


def test_outputs_have_to_match_the_inputs():
    x, o = torch.zeros(4, 2, 64), torch.zeros(2, 4, 64)
    for out in ((None, None, None), (o,), (o, o, o), (None, o, None), (o, None, None, None), (o[0], None, None)):
        with pytest.raises(ValueError, match="out:"):
            sv.qkv_rope(x, None, None, axes=(16, 24, 24), grid=(1, 2, 2), out=out)
    with pytest.raises(ValueError, match="device tensor"):
        sv.qkv_rope(x, None, None, axes=(16, 24, 24), grid=(1, 2, 2), out=(o, None, None))


@pytest.mark.gpu
def test_more_than_2_to_the_31_elements():
    N, H, d = 2 ** 17 + 70, 128, 128
    x = torch.empty(N, H, d, dtype=BF, device="cuda").normal_()
    w = 1 + 0.1 * torch.randn(H * d, device="cuda")
    kw = dict(axes=(44, 42, 42), norm=NORM["token"], wq=w)
    Q = sv.qkv_rope(x, None, None, grid=(1, 1, N), **kw)[0]
    back = sv.qkv_rope_backward(Q, None, None, x, None, grid=(1, 1, N), **kw)["dq"]
    for a in (0, N // 2, N - 64):
        pos = torch.zeros(64, 3, dtype=torch.int32, device="cuda")
        pos[:, 2] = torch.arange(a, a + 64, device="cuda")
        part = sv.qkv_rope(x[a:a + 64], None, None, positions=pos, **kw)[0]
        assert torch.equal(Q[:, a:a + 64], part)
        assert torch.equal(back[a:a + 64], sv.qkv_rope_backward(part, None, None, x[a:a + 64], None, positions=pos, **kw)["dq"])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["head", "token"])
def test_gradients_of_every_head_count(d, dtype, norm):
    """The gradients through the norms, with every number of heads, against 64 bits on the device; bounds as above."""
    N, g = 450, torch.Generator(device="cuda").manual_seed(7)
    axes, grid = ((16, 24, 24) if d == 64 else (44, 42, 42)), (2, 15, 15)
    wide = torch.randn(N, 16384 // d, d, generator=g, device="cuda").to(dtype)
    grads = torch.randn(16384 // d, N, d, generator=g, device="cuda").to(dtype)
    weights = 1 + 0.3 * torch.randn(16384, generator=g, device="cuda")
    t = torch.arange(N, device="cuda")
    pos = torch.stack([t // 225, t // 15 % 15, t % 15], -1).double()
    ang = torch.cat([pos[:, a:a + 1] * 10000.0 ** (-2.0 * torch.arange(s // 2, device="cuda").double() / s)
                     for a, s in enumerate(axes)], -1)
    back = torch.polar(torch.ones_like(ang), -ang)[:, None]
    dims = (-1,) if norm == "head" else (-1, -2)
    for H in range(1, 16384 // d + 1):
        x, dQ = wide[:, :H].contiguous(), grads[:H].contiguous()
        w = weights[:d if norm == "head" else H * d].contiguous()
        got = sv.qkv_rope_backward(dQ, None, None, x, None, axes=axes, grid=grid, norm=NORM[norm], wq=w)
        X, W, G = x.double(), w.double().view(-1, d), dQ.double().transpose(0, 1).contiguous()
        dz = torch.view_as_real(torch.view_as_complex(G.view(N, H, d // 2, 2)) * back).flatten(-2)
        mag = (dz[..., 0::2].abs() + dz[..., 1::2].abs()).repeat_interleave(2, -1)
        inv = 1 / torch.sqrt((X * X).mean(dims, keepdim=True) + 1e-6)
        n, u = X * inv, dz * W
        dx = inv * (u - n * (u * n).mean(dims, keepdim=True))
        mag_dx = inv * (mag * W.abs()).amax(dims, keepdim=True) * (2 + 2 * n.abs().amax(dims, keepdim=True) * n.abs())
        dw, mag_dw = (dz * n).sum(0), (mag * n.abs()).sum(0)
        if norm == "head":
            dw, mag_dw = dw.sum(0), mag_dw.sum(0)
        count = N * (H if norm == "head" else 1)
        for name, have, ref, m, k, c in (("dq", got["dq"], dx, mag_dx, dtype, 0),
                                         ("dwq", got["dwq"], dw.flatten(), mag_dw.flatten(), F32, count)):
            over = (have.double() - ref).abs() - ((K + c) * U * (m + ref.abs()) + HALF[k] * ref.abs() + 1e-37)
            assert over.max() <= 0, (name, H, float(over.max()))
