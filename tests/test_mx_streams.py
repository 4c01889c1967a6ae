"""The stream that a call is given: on the tensors' device, or refused (CPU)."""
import pytest
import torch


class FakeStream:
    def __init__(self, device):
        self.device = torch.device(device)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    from lossless_float_weight_b200 import build
    build.build()
    from lossless_float_weight_b200 import mx, zipnn as Z
    used = []
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", used.append)
    here = torch.device("cuda", 0)
    with pytest.raises(Z.ZipnnError):
        mx._use(FakeStream("cuda:1"), here)
    assert not used
    s = FakeStream("cuda:0")
    mx._use(s, here)
    assert used == [s]


def test_arguments_are_looked_at_before_the_stream(monkeypatch):
    """A call that is refused is refused alike with a stream and without."""
    from lossless_float_weight_b200 import mx, pages, zipnn as Z
    x, kv = torch.zeros(4, 64), torch.zeros(2, 4, 16, 8)
    for call in (lambda s: mx.quantize(x, stream=s), lambda s: mx.matmul(x, x, stream=s), lambda s: mx.dequantize(x, stream=s),
                 lambda s: pages.copy(kv, [0], kv, [1], stream=s)):
        for s in (None, 0):
            with pytest.raises(Z.ZipnnError):
                call(s)
