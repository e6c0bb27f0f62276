"""Calls that share a kernel and nothing else: host threads on streams of their
own that launch it with different sizes, and sizes recorded into one graph.
Every call has to be taken, and to give the bits that it gives alone."""
import ctypes
import threading

import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Norm:
    """svgear_block_norm of N rows, or its backward pass."""
    def __init__(self, N, D, back, dtype=BF):
        g = torch.Generator(device="cuda").manual_seed(N + D)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x, self.y, self.dr, self.dh = (rn(N, D).to(dtype) for _ in range(4))
        self.scale = rn(1, D)
        code = sv.dtype_code(self.x)
        self.p = sv.svgear_norm_params(N, D, 1, sv.SVGEAR_NORM_LAYER, sv.SVGEAR_NORM_NONE, 1e-6, 1.0, code, code)
        self.out = [torch.zeros_like(self.x), torch.zeros_like(self.x)]
        self.ws = sv.workspace(sv.svgear_block_norm_backward_workspace_size(self.p))
        self.back = back

    def call(self, stream):
        a = lambda t: t.data_ptr()  # noqa: E731
        p, (o0, o1), s = ctypes.byref(self.p), self.out, self.scale
        if self.back:
            return sv.lib().svgear_block_norm_backward(a(self.x), a(self.y), a(self.dr), a(self.dh), None, a(s), None, None, None,
                                                       None, p, a(o0), a(o1), None, None, None, None, None, None, a(self.ws),
                                                       self.ws.numel(), stream)
        return sv.lib().svgear_block_norm(a(self.x), a(self.y), None, a(s), None, None, None, None, None, p, a(o0), a(o1), stream)


class Rope:
    """svgear_qkv_rope of N tokens of H heads of 128, or its backward pass."""
    def __init__(self, N, H, back, dtype=BF):
        g = torch.Generator(device="cuda").manual_seed(N + H)
        self.rows = [torch.randn(N, H, 128, generator=g, device="cuda").to(dtype) for _ in range(3)]
        self.heads = [t.transpose(0, 1).contiguous() for t in self.rows]
        self.p = sv.rope_params(1, N, H, 128, (44, 42, 42), (1, 1, N), norm=sv.SVGEAR_QKNORM_TOKEN,
                                dtype=sv.dtype_code(self.rows[0]))
        self.out = [torch.zeros_like(t) for t in (self.rows if back else self.heads)]
        self.back = back

    def call(self, stream):
        a = [t.data_ptr() for t in self.rows]
        o, p = [t.data_ptr() for t in self.out], ctypes.byref(self.p)
        if self.back:
            return sv.lib().svgear_qkv_rope_backward(*(t.data_ptr() for t in self.heads), a[0], a[1], None, None, None, p, *o, None,
                                                     None, None, 0, stream)
        return sv.lib().svgear_qkv_rope(*a, None, None, None, p, *o, stream)


class Means:
    """svgear_kmeans with C centroids."""
    def __init__(self, N, C):
        g = torch.Generator(device="cuda").manual_seed(C)
        self.x = torch.randn(1, N, 128, generator=g, device="cuda").bfloat16()
        self.out = [torch.zeros(1, C, 128, device="cuda"), torch.zeros(1, N, dtype=torch.int32, device="cuda"),
                    torch.zeros(1, C, dtype=torch.int32, device="cuda")]
        self.N, self.C, self.ws = N, C, sv.workspace(sv.svgear_kmeans_workspace_size(1, N, 128, C))

    def call(self, stream):
        return sv.lib().svgear_kmeans(self.x.data_ptr(), sv.SVGEAR_BF16, 1, self.N, 128, self.C, 1, None,
                                      *(t.data_ptr() for t in self.out), self.ws.data_ptr(), self.ws.numel(), stream)


class Product:
    """svgear_mx_quantize and svgear_mx_product."""
    def __init__(self, M, N, K):
        g = torch.Generator(device="cuda").manual_seed(M)
        self.x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        self.w = sv.mx_quantize(torch.randn(N, K, generator=g, device="cuda"))
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.out = [torch.zeros(M, K // 2, **u8), torch.zeros(M, K // 32, **u8), torch.zeros(M, N, dtype=BF, device="cuda")]
        self.shape = (M, N, K)

    def call(self, stream):
        (M, N, K), (c, s, y) = self.shape, (t.data_ptr() for t in self.out)
        code = sv.lib().svgear_mx_quantize(self.x.data_ptr(), sv.SVGEAR_BF16, M, K, 0, c, s, stream)
        return code or sv.lib().svgear_mx_product(c, s, self.w[0].data_ptr(), self.w[1].data_ptr(), None, M, N, K, y, stream)


class Attention:
    """svgear_forward of two heads."""
    def __init__(self, N, Ck, d):
        g = torch.Generator(device="cuda").manual_seed(N)
        self.qkv = [torch.randn(2, N, d, generator=g, device="cuda").bfloat16() for _ in range(3)]
        self.p = sv.params(2, N, N, d, 8, Ck, 2, 0.3)
        self.ws = sv.workspace(sv.svgear_workspace_size(self.p))
        self.out = [torch.zeros(2, N, d, dtype=BF, device="cuda")]

    def call(self, stream):
        return sv.lib().svgear_forward(*(t.data_ptr() for t in self.qkv), ctypes.byref(self.p), None, None,
                                       self.out[0].data_ptr(), self.ws.data_ptr(), self.ws.numel(), stream, None)


# two sizes of one kernel that ask for different amounts of shared memory
PAIRS = {
    "norm": (lambda: Norm(1200, 5120, False), lambda: Norm(1, 5120, False)),
    "norm, other width": (lambda: Norm(1200, 2048, False, F32), lambda: Norm(1200, 1032, False, F32)),
    "norm backward": (lambda: Norm(600, 5120, True), lambda: Norm(600, 2560, True)),
    "rope": (lambda: Rope(600, 40, False), lambda: Rope(300, 20, False)),
    "rope backward": (lambda: Rope(600, 16, True), lambda: Rope(1, 9, True)),
    "product, few tokens": (lambda: Product(5, 512, 2048), lambda: Product(40, 128, 8192)),
    "product": (lambda: Product(300, 512, 512), lambda: Product(1000, 2048, 256)),
    "attention": (lambda: Attention(1024, 64, 128), lambda: Attention(512, 16, 128)),
    "k-means": (lambda: Means(512, 500), lambda: Means(512, 16)),
}


@pytest.fixture(params=sorted(PAIRS))
def pair(request):
    """The two calls and what each gives alone."""
    calls = [make() for make in PAIRS[request.param]]
    alone = []
    for c in calls:
        assert c.call(None) == sv.SVGEAR_OK
        torch.cuda.synchronize()
        alone.append([t.clone() for t in c.out])
        for t in c.out:
            t.zero_()
    torch.cuda.synchronize()
    return calls, alone


def check(calls, alone):
    for c, want in zip(calls, alone):
        assert all(torch.equal(a, b) for a, b in zip(c.out, want))
    assert sv.svgear_get_status() == sv.SVGEAR_OK


def test_two_threads_launch_one_kernel(pair):
    calls, alone = pair
    streams = [torch.cuda.Stream() for _ in calls]
    refused, start = [0, 0], threading.Barrier(2)
    rounds = 400 if isinstance(calls[0], Attention) else 4000

    def work(i):
        start.wait()
        for _ in range(rounds):
            refused[i] += calls[i].call(streams[i].cuda_stream) != sv.SVGEAR_OK

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    check(calls, alone)


def test_two_sizes_in_one_graph(pair):
    calls, alone = pair
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            assert c.call(side.cuda_stream) == sv.SVGEAR_OK
    assert calls[1].call(None) == sv.SVGEAR_OK  # the smaller one again, after the larger was recorded
    torch.cuda.synchronize()
    for _ in range(2):
        for c in calls:
            for t in c.out:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(calls, alone)
    del graph
