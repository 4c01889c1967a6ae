"""Microscaled 4-bit tensors at the ends of what a call takes: the longest rows, inputs that
carry gradients or a pending sign, and what a stored tensor shares with the one it came from."""
import numpy as np
import pytest
import torch

import mx_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_float_weight_b200 import mx
    return mx


@pytest.fixture(scope="module")
def Z():
    from lossless_float_weight_b200 import zipnn
    return zipnn


@pytest.mark.parametrize("fmt,cols", [("nvfp4", (1 << 29) + 65), ("nvfp4", 1 << 30), ("nvfp4", (1 << 30) - 7), ("mxfp4", (1 << 30) - 7)])
def test_the_longest_rows(mx, fmt, cols):
    """One row whose scale tiles pass 2^32 bytes (NVFP4, from column 2^29 on): both its ends,
    the middle, and the zeros between them. A power of two as the global scale, so that values
    read back as they are."""
    g = 0.25 if fmt == "nvfp4" else None
    gt = None if g is None else torch.tensor([g], device="cuda")
    x = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    rng = torch.Generator().manual_seed(cols % 1000)
    spans = [(0, 192), ((cols // 2) // 128 * 128, 192), (cols // 64 * 64 - 256, cols - (cols // 64 * 64 - 256))]
    parts = []
    for k, (at, n) in enumerate(spans):  # of different sizes, so that one end's scales are not the other's
        p = (torch.randn(1, n, generator=rng) * 5.0 ** k).to(torch.bfloat16)
        x[:, at:at + n] = p.cuda()
        parts.append(U.quantize(p.double().numpy(), fmt, g))
    q = mx.quantize(x, fmt, gt)
    y = mx.dequantize(q, torch.bfloat16, out=x)  # in place of the values: the memory is large
    for (at, n), (code, byte, _) in zip(spans, parts):
        got, _ = U.unpack(q.codes.view(torch.uint8)[:, at // 2:(at + n + 1) // 2].cpu().numpy(), 1, n)
        assert np.array_equal(got, code)
        blk = U.BLOCK[fmt]
        b = np.arange(at // blk, at // blk + byte.shape[1])
        sc = q.scales.view(torch.uint8)[torch.from_numpy(512 * (b // 4) + b % 4).cuda()].cpu().numpy()
        assert np.array_equal(sc, byte[0])
        want = torch.from_numpy(U.values(code, byte, fmt, g)).to(torch.bfloat16)
        assert torch.equal(y[:, at:at + n].cpu(), want)
    for (at, n), (then, _) in zip(spans, spans[1:]):
        assert not y[:, at + n:then].any()


def test_a_stored_tensor_keeps_its_own_scale(mx):
    """What happens to the scale of the tensor that was stored, or of one that was loaded, does
    not reach the container."""
    x = torch.randn(64, 96, generator=torch.Generator().manual_seed(3)).cuda()
    q = mx.quantize(x, "nvfp4")
    want = mx.dequantize(q, torch.float32)
    c = mx.compress(q)
    q.global_scale.mul_(3)
    a = mx.decompress(c)
    assert torch.equal(mx.dequantize(a, torch.float32), want)
    a.global_scale.mul_(5)
    assert torch.equal(mx.dequantize(mx.decompress(c), torch.float32), want)


def test_a_pending_negation_is_taken(mx, Z):
    """The imaginary part of a conjugate is a view whose sign is not in its memory."""
    z = torch.view_as_complex(torch.randn(40, 1, 2, generator=torch.Generator().manual_seed(1)).cuda())
    x = z.conj().imag
    assert x.is_neg()
    for view in (x, x[:1], x.t()):
        for fmt in ("mxfp4", "nvfp4"):
            a, b = mx.quantize(view, fmt), mx.quantize(view.clone(), fmt)
            assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
    q = mx.quantize(x)
    with pytest.raises(Z.ZipnnError):
        mx.dequantize(q, torch.float32, out=z.conj().imag)


def test_a_forward_gradient_is_refused(mx, Z):
    import torch.autograd.forward_ad as fw
    x = torch.ones(4, 64, device="cuda")
    b = mx.quantize(torch.ones(8, 64, device="cuda"))
    g = torch.ones(1, device="cuda")
    with fw.dual_level():
        d = fw.make_dual(x, torch.ones_like(x))
        for call in (lambda: mx.quantize(d), lambda: mx.matmul(d, b), lambda: mx.dequantize(mx.quantize(x), torch.float32, out=d),
                     lambda: mx.quantize(x, "nvfp4", fw.make_dual(g, torch.ones_like(g)))):
            with pytest.raises(Z.ZipnnError):
                call()
        mx.matmul(x, b)  # a plain tensor beside it
        mx.quantize(fw.unpack_dual(d).primal)


def test_gradients_of_scales_and_outputs_are_refused(mx, Z):
    x = torch.ones(4, 64, device="cuda")
    q, g = mx.quantize(x), torch.ones(1, device="cuda", requires_grad=True)
    out, prod = torch.zeros(4, 64, device="cuda", requires_grad=True), torch.zeros(4, 4, device="cuda", requires_grad=True)
    calls = (lambda: mx.quantize(x, "nvfp4", g), lambda: mx.dequantize(q, torch.float32, out=out),
             lambda: mx.matmul(q, q, torch.float32, out=prod))
    for call in calls:
        with pytest.raises(Z.ZipnnError):
            call()
    with torch.no_grad():
        for call in calls:
            call()
    assert torch.equal(out.detach(), torch.ones(4, 64, device="cuda")) and (prod.detach() == 64).all()


def test_an_output_saved_for_backward_is_seen_to_change(mx):
    q = mx.quantize(torch.ones(4, 64, device="cuda"))
    for write in (lambda o: mx.dequantize(q, torch.float32, out=o), lambda o: mx.matmul(q, mx.quantize(torch.ones(64, 64, device="cuda")), torch.float32, out=o)):
        out = torch.zeros(4, 64, device="cuda")
        w = torch.ones(4, 64, device="cuda", requires_grad=True)
        y = (w * out).sum()  # out is saved
        write(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_product_over_the_longest_rows(mx, Z, fmt):
    """2^30 - 7 products to a sum, in 2^22 stages over a cluster: values in the first columns, in
    those where the scale tiles pass 2^31 and 2^32 bytes, and in the last."""
    cols = (1 << 30) - 7
    f = {"mxfp4": Z.MXFP4, "nvfp4": Z.NVFP4}[fmt]
    rng = np.random.RandomState(2)
    at = np.unique(np.concatenate([np.arange(40), (1 << 28) + np.arange(-40, 40), (1 << 29) + np.arange(-40, 40), cols - 1 - np.arange(40)]))
    ones = {"mxfp4": 127, "nvfp4": 0x38}[fmt]
    parts = []
    for rows in (2, 3):
        v = rng.randint(1, 8, (rows, at.size))  # codes of positive values
        codes = torch.zeros(rows, Z.zipnn_mx_row_bytes(cols), dtype=torch.uint8, device="cuda")
        for odd in (0, 1):
            i = torch.from_numpy(at[at % 2 == odd] // 2).cuda()
            codes[:, i] |= torch.from_numpy(v[:, at % 2 == odd].astype(np.uint8) << (4 * odd)).cuda()
        scales = torch.full((Z.zipnn_mx_scale_bytes(f, rows, cols),), ones, dtype=torch.uint8, device="cuda")
        g = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
        parts.append((mx.MxTensor(codes, scales, (rows, cols), fmt, g), U.GRID[v]))
    (a, va), (b, vb) = parts
    y = mx.matmul(a, b, torch.float32)
    assert mx.status() == Z.OK
    assert np.array_equal(y.double().cpu().numpy(), va @ vb.T)
