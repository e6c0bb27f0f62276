"""The operators around the attention run together, as one attention block of a
video DiT: every step is checked against its formula in 64 bits on the values
that the step before produced (quantisation, clustering and routing are
discontinuous, so the end of the chain says little by itself), the whole is
checked to be what the steps give, and to replay from a graph bit for bit."""
import math

import numpy as np
import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv
from clustered_sparse_attention_flash_b200.block import BlockWeights, attention_block
from helpers import check_forward_given_gpu_clusters

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16
H, d, GRID, AXES = 4, 128, (2, 16, 32), (44, 42, 42)
N, D, G = 1024, 384, 2
CL = dict(Cq=8, Ck=32, iters=3, rho=0.3)


def inputs(types=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, m=1.0: torch.randn(*s, generator=g, device="cuda") * m  # noqa: E731
    # smooth over the grid, so that the clusters mean something
    base = rn(16, D, m=2.0)[torch.arange(N, device="cuda") // 64]
    x = (base + rn(N, D)).to(types)
    w = BlockWeights(sv.mx_quantize(rn(3 * H * d, D, m=D ** -0.5)), sv.mx_quantize(rn(D, H * d, m=(H * d) ** -0.5)),
                     rn(3 * H * d, m=0.1), rn(D, m=0.1), 1 + rn(H * d, m=0.1), 1 + rn(H * d, m=0.1))
    mods = dict(shift=rn(G, D, m=0.2), scale=rn(G, D, m=0.2), gate=rn(G, D, m=0.3), next_shift=rn(G, D, m=0.2),
                next_scale=rn(G, D, m=0.2))
    return x, w, mods


def near(got, want, rel, what):
    err, size = (got.double() - want).norm(), want.norm()
    assert err <= rel * size, f"{what}: {float(err / size):.3g} off, {rel:.3g} allowed"


def groups(t):
    return t.double().repeat_interleave(N // G, 0)


def layer_norm(x, eps=1e-6):
    x = x.double()
    c = x - x.mean(1, keepdim=True)
    return c / torch.sqrt((c * c).mean(1, keepdim=True) + eps)


def test_every_step_and_the_whole():
    x, w, m = inputs()
    # Outputs in bf16 are rounded once: each within 2^-8 of its value, so the norm of the error is within 2^-8 of
    # the norm; float32 arithmetic before it is smaller by orders (2^-24 and a few dozen roundings).
    R = 1.01 * 2.0 ** -8
    _, n = sv.block_norm(x, scale=m["scale"], shift=m["shift"])
    near(n, layer_norm(x) * (1 + groups(m["scale"])) + groups(m["shift"]), R, "norm")
    qkv = sv.mx_linear(n, *w.qkv, w.qkv_bias)
    val = lambda c: sv.mx_dequantize(*c, torch.float32).double()  # noqa: E731
    near(qkv, val(sv.mx_quantize(n)) @ val(w.qkv).T + w.qkv_bias.double(), R, "qkv projection")
    q, k, v = qkv.view(N, 3, H, d).unbind(1)
    Q, K, V = sv.qkv_rope(q, k, v, axes=AXES, grid=GRID, wq=w.q_norm, wk=w.k_norm, norm=sv.SVGEAR_QKNORM_TOKEN)
    t = torch.arange(N, device="cuda")
    pos = torch.stack([t // 512, t // 32 % 16, t % 32], -1).double()
    ang = torch.cat([pos[:, a:a + 1] * 10000.0 ** (-2 * torch.arange(s // 2, device="cuda").double() / s)
                     for a, s in enumerate(AXES)], -1)
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]
    for got, x_, wt in ((Q, q, w.q_norm), (K, k, w.k_norm)):
        z = x_.double() / torch.sqrt((x_.double() ** 2).mean((1, 2), keepdim=True) + 1e-6) * wt.double().view(H, d)
        z = torch.view_as_real(torch.view_as_complex(z.view(N, H, d // 2, 2)) * turn).flatten(-2)
        near(got, z.transpose(0, 1), R, "rotary positions")
    assert torch.equal(V, v.transpose(0, 1))
    O, ws, p, _ = sv.forward(Q, K, V, **CL)
    torch.cuda.synchronize()
    views = sv.view_tensors(p, ws)
    f = lambda a: a.float().cpu().numpy()  # noqa: E731
    for h in range(H):
        check_forward_given_gpu_clusters(views, f(O[h]), h, f(Q[h]), f(K[h]), f(V[h]), CL["Cq"], CL["Ck"], CL["rho"],
                                         1 / math.sqrt(d), "bf16")
    c = sv.mx_quantize(O)
    joined = sv.mx_quantize(O.transpose(0, 1).reshape(N, H * d).contiguous())
    assert torch.equal(c[0], joined[0]) and torch.equal(c[1], joined[1])
    y = sv.mx_product(*c, *w.out, w.out_bias)
    near(y, val(c) @ val(w.out).T + w.out_bias.double(), R, "output projection")
    r, h = sv.block_norm(x, y, gate=m["gate"], scale=m["next_scale"], shift=m["next_shift"])
    want = x.double() + groups(m["gate"]) * y.double()
    near(r, want, R, "residual")
    near(h, layer_norm(want) * (1 + groups(m["next_scale"])) + groups(m["next_shift"]), R, "next norm")
    r2, h2 = attention_block(x, w, H, axes=AXES, grid=GRID, **CL, **m)
    assert torch.equal(r, r2) and torch.equal(h, h2)
    assert sv.svgear_get_status() == sv.SVGEAR_OK


def test_float32_residual_stream_and_ragged_groups():
    x, w, m = inputs(torch.float32, seed=1)
    off = torch.tensor([0, 100, N], dtype=torch.int32, device="cuda")
    r, h = attention_block(x, w, H, axes=AXES, grid=GRID, offsets=off, **CL, **m)
    assert r.dtype == torch.float32 and h.dtype == BF and torch.isfinite(r).all()
    # the residual is kept to float32: what the block adds is the gate times a bf16 y
    added = (r.double() - x.double())
    y = added / m["gate"].double()[(torch.arange(N, device="cuda") >= 100).long()]
    lim = 2.0 ** -22 * (r.abs().double() + x.abs().double()) / m["gate"].abs().double().amin() + 1e-30
    assert ((y - y.float().to(BF).double()).abs() <= lim + 2.0 ** -8 * y.abs()).all()


def test_two_blocks_replay_from_graphs_that_share_a_workspace():
    x, w, m = inputs(seed=2)
    x2, w2, m2 = inputs(seed=3)
    p = sv.params(H, N, N, d, CL["Cq"], CL["Ck"], CL["iters"], CL["rho"])
    ws = sv.workspace(sv.svgear_workspace_size(p))
    run = lambda a, ww, mm: attention_block(a, ww, H, axes=AXES, grid=GRID, ws=ws, **CL, **mm)  # noqa: E731
    ref, ref2 = run(x, w, m), run(x2, w2, m2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(x, w, m)
    s.synchronize()
    ins, outs, graphs = [torch.zeros_like(x) for _ in range(2)], [], []
    for a, ww, mm in ((ins[0], w, m), (ins[1], w2, m2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(run(a, ww, mm))
        graphs.append(g)
    for _ in range(2):
        ins[0].copy_(x)
        ins[1].copy_(x2)
        for g in graphs:  # one after the other on one stream, as graphs that share a workspace have to be
            g.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, (ref, ref2)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sv.svgear_get_status() == sv.SVGEAR_OK
    del graphs


def test_gradients_of_the_trained_parts_chain():
    """Norm -> rotary positions -> (any attention) backwards: the pieces' gradients compose, against differences
    of the composed 64-bit forward."""
    g = torch.Generator().manual_seed(5)
    n, heads, dd = 12, 2, 64
    x = torch.randn(n, heads * dd, generator=g)
    wq, scale = 1 + 0.2 * torch.randn(heads * dd, generator=g), 0.3 * torch.randn(1, heads * dd, generator=g)
    dQ = torch.randn(heads, n, dd, generator=g)
    pos = torch.randint(0, 500, (n, 3), generator=g, dtype=torch.int32)
    axes = (16, 24, 24)

    def forward(a):
        h = (layer_norm(a) * (1 + scale.double())).view(n, heads, dd)
        z = h / torch.sqrt((h * h).mean((1, 2), keepdim=True) + 1e-6) * wq.double().view(heads, dd)
        ang = torch.cat([pos[:, i:i + 1].double() * 10000.0 ** (-2 * torch.arange(s // 2).double() / s)
                         for i, s in enumerate(axes)], -1)
        t = torch.polar(torch.ones_like(ang), ang)[:, None]
        z = torch.view_as_real(torch.view_as_complex(z.reshape(n, heads, dd // 2, 2)) * t).flatten(-2)
        return (z.transpose(0, 1) * dQ.double()).sum()

    _, h = sv.block_norm(x.cuda(), scale=scale.cuda())
    back = sv.qkv_rope_backward(dQ.cuda(), None, None, h.view(n, heads, dd), None, axes=axes, positions=pos.cuda(),
                                wq=wq.cuda(), norm=sv.SVGEAR_QKNORM_TOKEN)
    got = sv.block_norm_backward(x.cuda(), None, None, back["dq"].reshape(n, -1), scale=scale.cuda())["dx"].double().cpu()
    v = torch.randn(x.shape, generator=g, dtype=torch.float64)
    e = 1e-5
    want = (forward(x.double() + e * v) - forward(x.double() - e * v)) / (2 * e)
    # two float32 passes of well-conditioned rows: relative 1e-5 of the sum of magnitudes is hundreds of roundings
    assert abs((got * v).sum() - want) <= 1e-5 * (got * v).abs().sum(), ((got * v).sum(), want)
    assert np.isfinite(float(want))


def test_rows_behind_the_last_group_are_zero_rows(monkeypatch):
    """Offsets that end before the last row, on memory that holds NaN: the block's rows of no group are zeros going
    into the projection and in its outputs, so every other row is what the steps give for such an input."""
    x, w, m = inputs(seed=4)
    end = N - 100
    off = torch.tensor([0, 300, end], dtype=torch.int32, device="cuda")
    _, n = sv.block_norm(x, scale=m["scale"], shift=m["shift"], offsets=off)
    n[end:] = 0
    q, k, v = sv.mx_linear(n, *w.qkv, w.qkv_bias).view(N, 3, H, d).unbind(1)
    Q, K, V = sv.qkv_rope(q, k, v, axes=AXES, grid=GRID, wq=w.q_norm, wk=w.k_norm, norm=sv.SVGEAR_QKNORM_TOKEN)
    y = sv.mx_product(*sv.mx_quantize(sv.forward(Q, K, V, **CL)[0]), *w.out, w.out_bias)
    r, h = sv.block_norm(x, y, gate=m["gate"], scale=m["next_scale"], shift=m["next_shift"], offsets=off)
    real = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda *a, **kw: real(*a, **kw).fill_(math.nan))
    r2, h2 = attention_block(x, w, H, axes=AXES, grid=GRID, offsets=off, **CL, **m)
    assert torch.equal(r[:end], r2[:end]) and torch.equal(h[:end], h2[:end]) and r2.isfinite().all()
    assert (r2[end:] == 0).all() and (h2[end:] == 0).all()


@pytest.mark.parametrize("cuts", [(0, 100, N), (0, 1, 1023, 1023, N)])
def test_float32_stream_and_ragged_groups_step_by_step(cuts):
    """Each step of a block with a float32 residual stream against its formula, and the block against the steps."""
    x, w, _ = inputs(torch.float32, seed=6)
    n_groups = len(cuts) - 1
    g = torch.Generator(device="cuda").manual_seed(7)
    m = {n: torch.randn(n_groups, D, generator=g, device="cuda") * 0.3
         for n in ("shift", "scale", "gate", "next_shift", "next_scale")}
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    count = torch.tensor([b - a for a, b in zip(cuts, cuts[1:])], device="cuda")
    rows = lambda t: t.double().repeat_interleave(count, 0)  # noqa: E731
    R = 1.01 * 2.0 ** -8  # one rounding to bfloat16, as above
    _, n = sv.block_norm(x, scale=m["scale"], shift=m["shift"], offsets=off, dtype=BF)
    near(n, layer_norm(x) * (1 + rows(m["scale"])) + rows(m["shift"]), R, "norm")
    q, k, v = sv.mx_linear(n, *w.qkv, w.qkv_bias).view(N, 3, H, d).unbind(1)
    Q, K, V = sv.qkv_rope(q, k, v, axes=AXES, grid=GRID, wq=w.q_norm, wk=w.k_norm, norm=sv.SVGEAR_QKNORM_TOKEN)
    y = sv.mx_product(*sv.mx_quantize(sv.forward(Q, K, V, **CL)[0]), *w.out, w.out_bias)
    r, h = sv.block_norm(x, y, gate=m["gate"], scale=m["next_scale"], shift=m["next_shift"], offsets=off)
    added = rows(m["gate"]) * y.double()
    want = x.double() + added
    # r = x + (g y): the product and the sum are rounded to float32, each within 2^-24 of its value
    assert r.dtype == torch.float32 and h.dtype == BF
    assert ((r.double() - want).abs() <= 2.0 ** -24 * 1.001 * (added.abs() + want.abs())).all()
    near(h, layer_norm(want) * (1 + rows(m["next_scale"])) + rows(m["next_shift"]), R, "next norm")
    r2, h2 = attention_block(x, w, H, axes=AXES, grid=GRID, offsets=off, **CL, **m)
    assert torch.equal(r, r2) and torch.equal(h, h2)
