"""The helpers around the attention run where their tensors are; a stream of
another device is refused before anything is allocated or launched (a default
stream's handle is the same number on every device, so a launch would go to the
wrong one)."""
import pytest

from clustered_sparse_attention_flash_b200 import svgear as sv

torch = pytest.importorskip("torch")


class Elsewhere:
    device = torch.device("cuda", 1)
    cuda_stream = 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for current, wanted in ((0, 0), (1, 0), (0, 2)):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
        with pytest.raises(ValueError, match="stream: one of cuda"):
            sv._On(torch.device("cuda", wanted), Elsewhere())
    sv._On(torch.device("cuda", 0), None)


@pytest.mark.gpu
def test_streams_by_object_and_by_handle():
    x = torch.randn(5, 64, device="cuda")
    want = sv.block_norm(x)[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, torch.cuda.default_stream(), 0, None):
        got = sv.block_norm(x, stream=stream)[1]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
