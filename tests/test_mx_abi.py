"""Microscaled 4-bit tensors: sizes and refusals of the C calls and of the Python ones that
need no device (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def Z():
    from lossless_float_weight_b200 import build
    build.build()
    from lossless_float_weight_b200 import zipnn
    return zipnn


def test_sizes(Z):
    for cols, rb in ((1, 16), (32, 16), (33, 32), (4096, 2048), (4097, 2064)):
        assert Z.zipnn_mx_row_bytes(cols) == rb
    for fmt, blk in ((Z.MXFP4, 32), (Z.NVFP4, 16)):
        for rows, cols in ((1, 1), (128, 128), (129, 129), (77, 4080), (32000, 4096)):
            blocks = -(-cols // blk)
            assert Z.zipnn_mx_scale_bytes(fmt, rows, cols) == -(-rows // 128) * -(-blocks // 4) * 512
        assert Z.zipnn_mx_scale_bytes(fmt, 0, 5) == 0 and Z.zipnn_mx_scale_bytes(fmt, 5, 0) == 0
        assert Z.zipnn_mx_scale_bytes(fmt, (1 << 31) + 1, 5) == 0 and Z.zipnn_mx_scale_bytes(fmt, 5, (1 << 30) + 1) == 0
    assert Z.zipnn_mx_scale_bytes(2, 5, 5) == 0 and Z.zipnn_mx_row_bytes(0) == 0


def test_argument_errors_without_a_device(Z):
    fake, ws = 1 << 20, Z.MX_WORKSPACE_BYTES  # never dereferenced: every case fails before a launch

    def quant(fmt=Z.NVFP4, t=Z.VALUE_BF16, x=fake, rows=513, cols=64, stride=64, g=fake, find=1, codes=fake, scales=fake,
              w=fake, wb=ws):
        return Z.zipnn_mx_quantize(fmt, t, x, rows, cols, stride, g, find, codes, scales, w, wb, None)

    for bad in (dict(fmt=2), dict(t=3), dict(x=None), dict(x=fake + 1), dict(t=Z.VALUE_FP32, x=fake + 2), dict(rows=0),
                dict(cols=0, stride=0), dict(stride=63), dict(g=None), dict(g=fake + 2), dict(codes=None),
                dict(codes=fake + 8), dict(scales=fake + 4), dict(w=None), dict(w=fake + 4), dict(rows=(1 << 31) + 1),
                dict(cols=(1 << 30) + 1, stride=(1 << 30) + 1), dict(stride=(1 << 40) + 1)):
        assert quant(**bad) == Z.ERR_INVALID_ARG, bad
    assert quant(wb=ws - 1) == Z.ERR_OUT_TOO_SMALL

    def deq(fmt=Z.NVFP4, t=Z.VALUE_BF16, codes=fake, scales=fake, g=fake, rows=4, cols=64, out=fake, stride=64):
        return Z.zipnn_mx_dequantize(fmt, t, codes, scales, g, rows, cols, out, stride, None)

    for bad in (dict(fmt=-1), dict(t=9), dict(codes=None), dict(codes=fake + 1), dict(scales=None), dict(g=None),
                dict(rows=0), dict(cols=0), dict(out=None), dict(out=fake + 1), dict(stride=10)):
        assert deq(**bad) == Z.ERR_INVALID_ARG, bad
    def matmul(fmt=Z.NVFP4, ac=fake, asc=fake, ag=fake, bc=fake, bsc=fake, bg=fake, m=4, n=8, k=64, t=Z.VALUE_BF16, out=fake,
               stride=8):
        return Z.zipnn_mx_matmul(fmt, ac, asc, ag, bc, bsc, bg, m, n, k, t, out, stride, None)

    for bad in (dict(fmt=2), dict(ac=None), dict(asc=fake + 8), dict(ag=None), dict(bc=fake + 4), dict(bsc=None), dict(bg=fake + 1),
                dict(m=0), dict(n=0), dict(k=0), dict(t=5), dict(out=None), dict(out=fake + 1), dict(stride=7),
                dict(m=1 << 31, n=1 << 31, stride=1 << 31), dict(stride=(1 << 40) + 1)):
        assert matmul(**bad) == Z.ERR_INVALID_ARG, bad
    if not torch.cuda.is_available():
        assert matmul() == Z.ERR_UNSUPPORTED and matmul(fmt=Z.MXFP4, ag=None, bg=None) == Z.ERR_UNSUPPORTED
        assert Z.zipnn_mx_status(None) == Z.ERR_UNSUPPORTED
        assert quant() == Z.ERR_UNSUPPORTED and deq() == Z.ERR_UNSUPPORTED
        assert quant(fmt=Z.MXFP4, g=None, w=None, wb=0) == Z.ERR_UNSUPPORTED  # not needed for MXFP4
        assert quant(rows=512, w=None, wb=0) == Z.ERR_UNSUPPORTED  # nor for 1024 chunks
        assert quant(find=0, w=None, wb=0) == Z.ERR_UNSUPPORTED


def test_python_refusals(Z):
    from lossless_float_weight_b200 import mx
    x = torch.zeros(4, 64)
    for call in (lambda: mx.quantize(x), lambda: mx.quantize(x, "fp4"), lambda: mx.quantize(x.double()),
                 lambda: mx.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), (4, 64), "mxfp4"),
                 lambda: mx.MxTensor(None, None, (), "mxfp4")):
        with pytest.raises(Z.ZipnnError):
            call()


def test_tile_scales_is_the_documented_layout(Z):
    from lossless_float_weight_b200 import mx
    s = torch.randint(1, 255, (130, 9), dtype=torch.uint8)
    t = mx.tile_scales(s)
    assert t.numel() == 2 * 3 * 512
    want = torch.zeros(2 * 3 * 512, dtype=torch.uint8)
    for r in range(130):
        for b in range(9):
            want[512 * (r // 128 * 3 + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4] = s[r, b]
    assert torch.equal(t, want)


def test_wait_limit_is_a_host_setting(Z):
    assert Z.zipnn_test_mx_wait_limit(0, 7, 3) == Z.OK
    assert Z.zipnn_test_mx_wait_limit(0, 8, 0) == Z.ERR_INVALID_ARG and Z.zipnn_test_mx_wait_limit(0, 0, 8) == Z.ERR_INVALID_ARG
    assert Z.zipnn_test_mx_wait_limit(1 << 22, 0, 0) == Z.OK  # back to the default
