"""Counts beyond a C int are refused, not cut to 32 bits: 2^32 + 16 rows must not
run as 16.  Tensors of such shapes exist on a GPU; here stand-ins have them, and
nothing is allocated or launched."""
import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv

torch = pytest.importorskip("torch")

ROWS = 2 ** 32 + 16


class Huge:
    """What the helpers ask of a tensor, without its memory."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Here:
    """In the place of the device guard."""
    def __init__(self, device, stream):
        pass

    def __enter__(self):
        return 0

    def __exit__(self, *e):
        pass


@pytest.fixture(autouse=True)
def nothing_runs(monkeypatch):
    monkeypatch.setattr(sv, "_On", Here)

    def no(*a, **k):
        raise AssertionError("a call got through")

    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, no)
    monkeypatch.setattr(sv, "lib", no)


U8 = dict(dtype=torch.uint8)
CALLS = {
    "norm": lambda: sv.block_norm(Huge(ROWS, 8)),
    "norm, groups": lambda: sv.block_norm(Huge(16, 8), scale=Huge(ROWS, 8, dtype=torch.float32)),
    "norm backward": lambda: sv.block_norm_backward(Huge(ROWS, 8), None, None, Huge(ROWS, 8)),
    "quantise": lambda: sv.mx_quantize(Huge(ROWS, 32)),
    "quantise heads": lambda: sv.mx_quantize(Huge(1, ROWS, 64)),
    "dequantise": lambda: sv.mx_dequantize(Huge(ROWS, 16, **U8), Huge(ROWS, 1, **U8)),
    "product": lambda: sv.mx_product(Huge(ROWS, 16, **U8), Huge(ROWS, 1, **U8), Huge(8, 16, **U8), Huge(8, 1, **U8)),
    "product, features": lambda: sv.mx_product(Huge(1, 16, **U8), Huge(1, 1, **U8), Huge(ROWS, 16, **U8), Huge(ROWS, 1, **U8)),
    "linear": lambda: sv.mx_linear(Huge(ROWS, 32), Huge(8, 16, **U8), Huge(8, 1, **U8)),
    "entry quantise": lambda: sv.svgear_mx_quantize(4096, sv.SVGEAR_BF16, ROWS, 32, 0, 4096, 4096, 0),
    "entry dequantise": lambda: sv.svgear_mx_dequantize(4096, 4096, ROWS, 32, 4096, sv.SVGEAR_BF16, 0),
    "entry product": lambda: sv.svgear_mx_product(4096, 4096, 4096, 4096, None, ROWS, 8, 32, 4096, 0),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_counts_beyond_an_int_are_refused(name, monkeypatch):
    monkeypatch.setattr(sv, "status_string", lambda code: "")
    with pytest.raises(sv.SvgearError) as e:
        CALLS[name]()
    assert e.value.code == sv.SVGEAR_ERR_UNSUPPORTED


def test_rotary_counts_beyond_an_int_are_refused():
    with pytest.raises(Exception, match="format|argument|range"):
        sv.rope_params(1, ROWS, 1, 64, (16, 24, 24))
