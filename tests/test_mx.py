"""Microscaled 4-bit floats: quantisation, its values, and the product.

Quantisation and dequantisation are exact: codes and scales are compared bit
for bit with the definition in 64 bits.  The product multiplies exactly and
adds in float32: with every one of the K additions off by at most one unit in
the last place of the running magnitude, a sum is within K 2^-23 of the sum of
its terms' magnitudes; it is rounded once to bf16 (eps/2 = 2^-8)."""
import ctypes

import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv
from clustered_sparse_attention_flash_b200.build import build

torch = pytest.importorskip("torch")

BF, F32 = torch.bfloat16, torch.float32
LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def quantise(x):
    """(codes 0..15 [M, K], scale bytes [M, K/32]) of the definition."""
    M, K = x.shape
    b = x.double().view(M, K // 32, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(bad | (top == 0), torch.ones_like(top), top))[1] - 3
    e = torch.where(top == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    v = torch.where(bad[..., None], torch.zeros_like(b), b) / 2.0 ** e[..., None].double()
    gap = (v.abs()[..., None].clamp_max(6.0) - LEVELS).abs()
    near = gap.amin(-1, keepdim=True)
    even = torch.arange(8) % 2 == 0
    code = torch.where((gap == near) & even, 100, torch.where(gap == near, 50, 0)).argmax(-1)
    code = code + 8 * torch.signbit(v)
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    return code.view(M, K).to(torch.uint8), torch.where(bad, torch.full_like(e, 128), e).add(127).to(torch.uint8)


def unpacked(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def values(code, scales):
    """[M, K] in 64 bits."""
    v = LEVELS[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0).double()
    s = torch.where(scales == 255, float("nan"), 2.0 ** (scales.double() - 127))
    return v * s.repeat_interleave(32, 1)


def rows(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, K // 32, generator=g)).repeat_interleave(32, 1)
    x[torch.rand(M, generator=g) < 0.1] = 0
    x[:, ::5] *= 0.01
    return x.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,dtype", [(1, 32, F32), (1, 5120, BF), (3, 96, BF), (257, 160, F32), (333, 1056, F32),
                                       (1000, 2048, BF), (7, 8224, BF), (70000, 64, BF)])
def test_quantise_and_dequantise(M, K, dtype):
    x = rows(M, K, dtype, M + K)
    codes, scales = sv.mx_quantize(x.cuda())
    want_c, want_s = quantise(x)
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(unpacked(codes.cpu()), want_c)
    for t in (BF, F32):
        got = sv.mx_dequantize(codes, scales, t)
        assert got.dtype == t and torch.equal(got.double().cpu(), values(want_c, want_s))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantise_special_values(dtype):
    """Ties, saturation, signed zeros, the ends of the exponent range, NaN and infinities."""
    x = torch.zeros(14, 64, dtype=F32)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.96875, 0.2490234375, 0.2509765625])
    x[0, :12], x[0, 12:24], x[0, 31] = ties, -ties, 4.0
    x[1, :12], x[1, 31] = ties * 2.0 ** 100, 4.0 * 2.0 ** 100
    x[2, :12], x[2, 31] = ties * 2.0 ** -100, -4.0 * 2.0 ** -100
    x[3, :32] = -0.0
    x[4, 5], x[4, 40] = 3.0e38, -3.0e38
    x[5, 5], x[5, 40] = 2.0 ** -126, 2.0 ** -133       # the second is subnormal in both types
    x[6, 5], x[6, 40] = 2.0 ** -124, 1.75 * 2.0 ** -125
    x[7] = 1.0
    x[7, 3] = float("nan")
    x[8] = 1.0
    x[8, 35] = float("inf")
    x[9] = -2.0
    x[9, 0] = float("-inf")
    x[10] = torch.linspace(-6, 6, 64)
    x[11] = torch.linspace(-8, 8, 64)
    x[12] = 2.0 ** -127 * torch.arange(64)
    x[13] = torch.linspace(0, 1, 64) * 2.0 ** 127
    x = x.to(dtype)
    codes, scales = sv.mx_quantize(x.cuda())
    want_c, want_s = quantise(x)
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(unpacked(codes.cpu()), want_c)
    got = sv.mx_dequantize(codes, scales, F32).double().cpu()
    want = values(want_c, want_s)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got).any()
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))


@pytest.mark.gpu
def test_dequantise_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).view(-1, 16)[torch.arange(256) % 16]  # [256, 16]: 32 elements a row
    scales = torch.arange(256, dtype=torch.uint8)[:, None]
    got = sv.mx_dequantize(codes.cuda(), scales.cuda(), F32).cpu()
    want = values(unpacked(codes), scales).float()  # 6 * 2^127 is an infinity in float32
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0, 1e38, -1e38), want.nan_to_num(0, 1e38, -1e38))


@pytest.mark.gpu
@pytest.mark.parametrize("H,M,d,dtype", [(40, 77, 128, BF), (3, 129, 64, F32), (1, 5, 64, BF), (4, 1, 8, F32)])
def test_quantise_head_major(H, M, d, dtype):
    x = rows(M, H * d, dtype, 9)
    heads = x.view(M, H, d).transpose(0, 1).contiguous()
    a, b = sv.mx_quantize(x.cuda()), sv.mx_quantize(heads.cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def weights(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8),
            torch.randint(110, 135, (N, K // 32), generator=g, dtype=torch.uint8))


def product_check(a, sa, w, sw, bias, got):
    A, W = (values(unpacked(c), s).cuda() for c, s in ((a, sa), (w, sw)))
    ref, mag = A @ W.T, A.abs() @ W.abs().T
    if bias is not None:
        ref = ref + bias.double().cuda()
    K = A.shape[1]
    lim = 2.0 ** -8 * ref.abs() + (K + 2) * 2.0 ** -23 * (mag + ref.abs()) + 1e-38
    err = (got.double() - ref).abs()
    assert (err <= lim).all(), f"{int((~(err <= lim)).sum())} of {err.numel()} off, worst {(err / lim).max():.3g} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,bias", [
    (1, 8, 32, False), (16, 128, 64, False), (16, 128, 256, False), (16, 128, 512, True), (5, 136, 160, True),
    (17, 120, 288, False), (64, 256, 1024, True), (65, 128, 96, True), (192, 128, 256, False), (193, 1000, 2080, True),
    (500, 264, 352, True), (1, 30720, 512, True), (33, 2048, 5120, False), (1000, 5120, 2048, True), (3000, 1032, 4128, True),
    (14337, 2304, 544, True), (224, 256, 1312, False), (200, 264, 8224, True), (900, 2056, 416, False), (512, 512, 8192, True),
    (2, 40, 16384, False)])
def test_product(M, N, K, bias):
    a, sa = weights(M, K, 1)
    w, sw = weights(N, K, 2)
    b = torch.randn(N) * 100 if bias else None
    got = sv.mx_product(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), None if b is None else b.cuda())
    assert sv.svgear_get_status() == sv.SVGEAR_OK
    assert got.shape == (M, N) and got.dtype == BF
    product_check(a, sa, w, sw, b, got)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 40, 200])
def test_product_places_every_scale_and_element(M):
    """One-hot operands: each output is a single product, so a wrong row, block or nibble shows exactly."""
    N, K = 136, 544
    g = torch.Generator().manual_seed(M)
    ka, kw = torch.randint(0, K, (M,), generator=g), torch.randint(0, K, (N,), generator=g)
    kw[:min(M, N)] = ka[:min(M, N)]
    a, w = torch.zeros(M, K, dtype=torch.uint8), torch.zeros(N, K, dtype=torch.uint8)
    a[torch.arange(M), ka] = torch.randint(1, 8, (M,), generator=g, dtype=torch.uint8)
    w[torch.arange(N), kw] = torch.randint(9, 16, (N,), generator=g, dtype=torch.uint8)
    pack = lambda c: c[:, 0::2] | c[:, 1::2] << 4  # noqa: E731
    sa = torch.randint(100, 150, (M, K // 32), generator=g, dtype=torch.uint8)
    sw = torch.randint(100, 150, (N, K // 32), generator=g, dtype=torch.uint8)
    got = sv.mx_product(pack(a).cuda(), sa.cuda(), pack(w).cuda(), sw.cuda()).double().cpu()
    assert torch.equal(got, (values(a, sa) @ values(w, sw).T).to(BF).double())


@pytest.mark.gpu
def test_product_of_nan_scales_and_untouched_memory():
    M, N, K = 70, 264, 320
    a, sa = weights(M, K, 5)
    w, sw = weights(N, K, 6)
    sa[3, 2], sw[130, 9] = 255, 255
    args = [t.cuda() for t in (a, sa, w, sw)]
    y = torch.full((M + 2, N), 7.0, dtype=BF, device="cuda")
    sv.svgear_mx_product(*args, None, M, N, K, y)
    assert torch.isnan(y[3]).all() and torch.isnan(y[:M, 130]).all() and (y[M:] == 7).all()
    rest = y[:M].clone()
    rest[3], rest[:, 130] = 0, 0
    assert torch.isfinite(rest).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 300])
def test_same_bits_on_another_stream_and_in_two_graphs(M):
    N, K = 1280, 2048
    x = [rows(M, K, BF, s).cuda() for s in (1, 2)]
    w, sw = (t.cuda() for t in weights(N, K, 3))
    ref = [sv.mx_linear(t, w, sw) for t in x]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.mx_linear(x[0], w, sw, stream=s)
    s.synchronize()
    assert torch.equal(got, ref[0])
    ins, outs, graphs = [torch.zeros_like(t) for t in x], [], []
    for t in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(sv.mx_linear(t, w, sw))
        graphs.append(g)
    for t, v in zip(ins, x):
        t.copy_(v)
    s2 = torch.cuda.Stream()
    for st in (s, s2):
        st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphs[0].replay()
    with torch.cuda.stream(s2):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])
    assert sv.svgear_get_status() == sv.SVGEAR_OK
    del graphs


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_linears_in_a_row(M):
    """Each call reads what the one before has just written, and its memory is taken again: the same bits as with
    a pause after every call, eagerly and in a replayed graph."""
    K = 1024
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).cuda().bfloat16()
    ws = [tuple(t.cuda() for t in weights(K, K, i)) for i in range(3)]

    def chain(pause):
        y = x
        for i in range(12):
            y = sv.mx_linear(y, *ws[i % 3])
            y = y / y.float().abs().amax().clamp(min=1e-3).bfloat16() if i % 4 == 3 else y
            if pause:
                torch.cuda.synchronize()
        return y

    want = chain(True)
    assert want.isfinite().all() and want.count_nonzero() > 0
    assert all(torch.equal(chain(False), want) for _ in range(5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = chain(False)
    for _ in range(3):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_linears_on_two_streams_at_once():
    """Narrow, split and wide products beside each other: the bits of each alone."""
    shapes = [(1, 4096, 1024), (40, 512, 4096), (300, 1024, 2048), (2000, 2048, 512)]
    calls = []
    for i, (M, N, K) in enumerate(shapes):
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(i)).cuda().bfloat16()
        w = tuple(t.cuda() for t in weights(N, K, i))
        calls.append((x, w, sv.mx_linear(x, *w)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(40):
        x, w, want = calls[(i // 2 + (i & 1) * (1 + i // 8)) % 4]
        got.append((sv.mx_linear(x, *w, stream=streams[i & 1]), want))
    torch.cuda.synchronize()
    assert sv.svgear_get_status() == sv.SVGEAR_OK
    assert all(torch.equal(y, want) for y, want in got)


# ------------------------------------------------------------------ refusals

def test_chained_kernels_load_coherently():
    """A kernel that may run beside the one ahead of it must not promise that what it reads is constant."""
    import pathlib
    import re
    src = pathlib.Path(sv.HERE) / "csrc"
    chained = 0
    for f in sorted(src.glob("*.cu")):
        code = re.sub(r"//[^\n]*", "", f.read_text())
        # a kernel and what it calls in its file: the product's file whole, the dequantisation's own text
        parts = [code] if f.name == "mx_product.cu" else re.split(r"(?=\n(?:template|__global__))", code)
        for part in parts:
            if "wait_previous(" in part:
                chained += 1
                assert not re.search(r"__ldg|__restrict__|\.nc\b", part), (f.name, part[:200])
    assert chained == 2


@pytest.fixture(scope="module")
def L():
    build()
    return sv.lib()


A = 4096  # an aligned non-null address: validation only, nothing runs


def test_refusals(L):
    INV, UNS = sv.SVGEAR_ERR_INVALID, sv.SVGEAR_ERR_UNSUPPORTED
    q = lambda X=A, dt=1, M=4, K=64, hd=0, c=A, s=A: L.svgear_mx_quantize(X, dt, M, K, hd, c, s, None)  # noqa: E731
    for kw, code in ((dict(M=0), INV), (dict(K=0), INV), (dict(K=-32), INV), (dict(K=48), UNS), (dict(K=2 ** 20 + 32), UNS),
                     (dict(M=2 ** 30, K=1024), UNS), (dict(dt=2), UNS), (dict(hd=-8), INV), (dict(hd=12), INV),
                     (dict(hd=24), INV), (dict(X=None), INV), (dict(c=None), INV), (dict(s=None), INV), (dict(X=A + 8), INV),
                     (dict(c=A + 4), INV), (dict(s=A + 1), INV)):
        assert q(**kw) == code, kw
    d = lambda c=A, s=A, M=4, K=64, Y=A, dt=1: L.svgear_mx_dequantize(c, s, M, K, Y, dt, None)  # noqa: E731
    for kw, code in ((dict(M=0), INV), (dict(K=16), UNS), (dict(dt=-1), UNS), (dict(c=None), INV), (dict(s=None), INV),
                     (dict(Y=None), INV), (dict(Y=A + 2), INV)):
        assert d(**kw) == code, kw

    def p(M=4, N=64, K=64, b=A, Y=A, ac=A, as_=A, wc=A, ws_=A):
        return L.svgear_mx_product(ac, as_, wc, ws_, b, M, N, K, Y, None)

    for kw, code in ((dict(M=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=40), UNS), (dict(N=12), UNS),
                     (dict(M=2 ** 27, N=2 ** 24, K=32), UNS), (dict(ac=None), INV), (dict(as_=None), INV), (dict(wc=None), INV),
                     (dict(ws_=None), INV), (dict(Y=None), INV), (dict(b=A + 4), INV), (dict(Y=A + 8), INV), (dict(wc=A + 2), INV)):
        assert p(**kw) == code, kw
    with pytest.raises(ValueError, match="device tensor"):
        sv.mx_quantize(torch.zeros(2, 64))


def test_refusals_of_row_counts(L):
    """Row counters run up to a tile beyond the last row and stay below 2^31."""
    UNS = sv.SVGEAR_ERR_UNSUPPORTED
    for M in (2 ** 30 + 1, 2 ** 31 - 1):
        assert L.svgear_mx_quantize(A, 1, M, 32, 0, A, A, None) == UNS
        assert L.svgear_mx_dequantize(A, A, M, 32, A, 1, None) == UNS
        assert L.svgear_mx_product(A, A, A, A, None, M, 8, 32, A, None) == UNS
    for N in (2 ** 30 + 8, 2 ** 31 - 8):
        assert L.svgear_mx_product(A, A, A, A, None, 4, N, 32, A, None) == UNS


@pytest.mark.gpu
def test_refusals_of_tensors():
    x = torch.zeros(4, 64, device="cuda")
    c, s = sv.mx_quantize(x)
    with pytest.raises(ValueError, match="contiguous"):
        sv.mx_quantize(torch.zeros(64, 4, device="cuda").T)
    with pytest.raises(ValueError, match="unsupported"):
        sv.mx_quantize(x.half())
    with pytest.raises(sv.SvgearError):
        sv.mx_quantize(torch.zeros(4, 40, device="cuda"))
    with pytest.raises(ValueError, match="scales"):
        sv.mx_dequantize(c, s[:2])
    with pytest.raises(ValueError, match="w_codes"):
        sv.mx_product(c, s, c.int(), s)
    with pytest.raises(ValueError, match="a_scales"):
        sv.mx_product(c, s.cpu(), c, s)
    with pytest.raises(ValueError, match="bias"):
        sv.mx_product(c, s, c, s, torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="columns"):
        sv.mx_linear(torch.zeros(4, 128, device="cuda"), c, s)
    with pytest.raises(sv.SvgearError):
        sv.mx_product(c, s, c, s)  # four features: not a multiple of 8


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 300])
def test_chained_launches_captured_behind_copies_and_joined_streams(M):
    """The product and the dequantisation recorded behind a copy, behind a fill, behind two joined streams and first
    in a graph of their own: whatever stands ahead of them has ended before they read."""
    N, K = 264, 1024
    x = torch.randn(M, K, device="cuda").bfloat16()
    w, sw = (t.cuda() for t in weights(N, K, 3))
    codes, scales = sv.mx_quantize(x)
    want, vals = sv.mx_product(codes, scales, w, sw), sv.mx_dequantize(codes, scales)
    a, s = torch.zeros_like(codes), torch.zeros_like(scales)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def behind_a_copy():
        a.zero_()
        a.copy_(codes)
        s.copy_(scales)

    def behind_a_join():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            a.copy_(codes)
        s.copy_(scales)
        main.wait_stream(side)

    for ahead in (behind_a_copy, behind_a_join, lambda: None):
        for call, ref in ((lambda: sv.mx_product(a, s, w, sw), want), (lambda: sv.mx_dequantize(a, s), vals)):
            a.copy_(codes)
            s.copy_(scales)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                ahead()
                out = call()
            for _ in range(3):
                out.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, ref)
            del graph
    assert sv.svgear_get_status() == sv.SVGEAR_OK


def small_numbers(M, K, seed, device="cpu"):
    """Random codes under scales 1/2, 1 and 2: every product of two such matrices is a multiple of 2^-4."""
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randint(0, 256, (M, K // 2), generator=g, dtype=torch.uint8, device=device),
            torch.randint(126, 129, (M, K // 32), generator=g, dtype=torch.uint8, device=device))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 2048, 16384), (2, 40, 16384), (16, 512, 8192), (40, 136, 16384), (64, 1024, 5120),
                                   (128, 256, 8192), (300, 264, 8224), (500, 512, 16384), (2000, 1032, 4128), (3000, 2304, 1056)])
def test_sums_are_kept_to_float32_and_rounded_once(M, N, K):
    """The magnitudes add up to less than 2^24 units of 2^-4, so that float32 holds every partial sum exactly in any
    order, and the one rounding left is that of the result."""
    a, sa = small_numbers(M, K, 1)
    w, sw = small_numbers(N, K, 2)
    bias = torch.randint(-4000, 4000, (N,), generator=torch.Generator().manual_seed(3)).float() / 16
    A, W = (values(unpacked(c), s).cuda() for c, s in ((a, sa), (w, sw)))
    ref = A @ W.T
    assert ((A.abs() @ W.abs().T).amax() + 250) * 16 < 2 ** 24
    dev = [t.cuda() for t in (a, sa, w, sw)]
    assert torch.equal(sv.mx_product(*dev).double(), ref.to(BF).double())
    assert torch.equal(sv.mx_product(*dev, bias.cuda()).double(), (ref + bias.double().cuda()).to(BF).double())


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [False, True])
def test_quantise_more_than_2_to_the_31_elements(heads):
    M, K = 2 ** 21 + 64, 1024
    x = torch.empty((8, M, 128) if heads else (M, K), dtype=BF, device="cuda").normal_()
    codes, scales = sv.mx_quantize(x)
    y = sv.mx_dequantize(codes, scales)
    for at in (slice(0, 64), slice(M - 64, M)):
        part = x[:, at].contiguous() if heads else x[at]
        c, s = sv.mx_quantize(part)
        assert torch.equal(codes[at], c) and torch.equal(scales[at], s)
        assert torch.equal(y[at], sv.mx_dequantize(c, s))


@pytest.mark.gpu
def test_product_of_more_than_2_to_the_31_elements():
    M, N, K = 2 ** 21 + 64, 1032, 512
    a, sa = small_numbers(M, K, 1, "cuda")
    w, sw = small_numbers(N, K, 2, "cuda")
    y = sv.mx_product(a, sa, w, sw)
    assert sv.svgear_get_status() == sv.SVGEAR_OK
    for at in (slice(0, 64), slice(M // 2, M // 2 + 64), slice(M - 64, M)):
        assert torch.equal(y[at], sv.mx_product(a[at], sa[at], w, sw))
