"""Products whose waits give up: what is stored is right, what is not is left as it was, the
status says so, and the next call is whole."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_float_weight_b200 import mx
    return mx


# clusters of 8, 4 and 2 blocks, single blocks with more stages than places, with fewer, two to
# an SM, and pairs of blocks with one tile each and with several
SIZES = [(1, 512, 8192), (16, 4096, 4096), (64, 8192, 4096), (128, 11008, 4096), (100, 32000, 1024), (5, 130, 300),
         (2048, 1280, 4096), (4096, 4096, 2048), (1700, 2600, 700)]


# (polls, mask, value): every block at once, some blocks of a cluster or of a pair, or pairs among
# others that go on; and a single poll, which may find what it waits for or not
LIMITS = [(0, 0, 0), (0, 1, 0), (0, 1, 1), (0, 3, 2), (0, 7, 0), (0, 7, 5), (1, 0, 0), (1, 1, 1), (2, 3, 0)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_product_that_gives_up(mx, fmt, size):
    from lossless_float_weight_b200 import zipnn as Z
    m, n, k = size
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (mx.quantize(torch.randn(r, k, generator=g, device="cuda"), fmt) for r in (m, n))
    want = mx.matmul(a, b, torch.float32)
    assert mx.status() == Z.OK and want.isfinite().all()
    out = torch.empty_like(want)
    mark = 3e38  # no result of these
    try:
        for limit in LIMITS:
            assert Z.zipnn_test_mx_wait_limit(*limit) == Z.OK
            for _ in range(2):
                out.fill_(mark)
                mx.matmul(a, b, torch.float32, out=out)
                status = mx.status()
                left = out == mark
                assert status in (Z.OK, Z.ERR_TIMEOUT)
                assert torch.equal(torch.where(left, want, out), want), limit
                assert status == Z.ERR_TIMEOUT or not left.any()
                if limit == (0, 0, 0):
                    assert status == Z.ERR_TIMEOUT and left.all()
                if limit == (0, 1, 0):  # block 0 is one of these
                    assert status == Z.ERR_TIMEOUT and left.any()
    finally:
        Z.zipnn_test_mx_wait_limit(1 << 22, 0, 0)
    assert torch.equal(mx.matmul(a, b, torch.float32, out=out), want) and mx.status() == Z.OK
