"""Microscaled 4-bit tensors on the GPU: codes and scales equal, bit for bit, to the 64-bit
definition, and values read back rounded once or twice at most."""
import numpy as np
import pytest
import torch

import mx_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_float_weight_b200 import mx
    return mx


def make(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 2)
    x.view(-1)[torch.randperm(x.numel(), generator=g)[: x.numel() // 50]] *= 30
    x.view(-1)[torch.randperm(x.numel(), generator=g)[: x.numel() // 20]] = 0
    return x.clamp(-60000, 60000).to(DT[dtype])


def check_quantize(mx, x, fmt, g=None, xd=None):
    xd = x.cuda() if xd is None else xd
    g = None if g is None else float(np.float32(g))
    q = mx.quantize(xd, fmt, None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda"))
    cols = x.shape[-1]
    rows = x.numel() // cols
    code, byte, gw = U.quantize(x.reshape(rows, cols).double().numpy(), fmt, g)
    got, pad = U.unpack(q.codes.view(torch.uint8).cpu().numpy(), rows, cols)
    sc, rest = U.untile(q.scales.view(torch.uint8).cpu().numpy(), rows, cols, fmt)
    if fmt == "nvfp4":
        assert q.global_scale.item() == gw
    assert np.array_equal(sc, byte)
    assert np.array_equal(got, code)
    assert not pad.any() and not rest.any()
    return q, U.values(code, byte, fmt, gw)


SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 16), (7, 17), (128, 128), (129, 130), (33, 500), (300, 65), (1, 4096),
          (64, 257), (2, 11008), (1000, 15), (700, 200), (2049, 31)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_equals_the_definition(mx, fmt, dtype):
    for i, (r, c) in enumerate(SHAPES):
        check_quantize(mx, make(r, c, dtype, i), fmt)


@pytest.mark.parametrize("fmt,g", [("mxfp4", None), ("nvfp4", 1.0), ("nvfp4", 0.3), ("nvfp4", 2.0 ** -20),
                                   ("nvfp4", 1e-38), ("nvfp4", 1e-41), ("nvfp4", 1e30), ("nvfp4", 3e38)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_borders_and_extremes(mx, fmt, g, dtype):
    """Values on, just below and just above every border between two codes and two scales."""
    rng = np.random.RandomState(3)
    base = []
    unit = 1.0 if g is None else float(np.float32(g))
    top = 3e38 / max(1.0, unit)
    for s in (0.5, 1.0, 1.75, 3.25, 448.0, 2.0 ** -9, 2.0 ** -6, 0.0146484375):
        for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 1.0, 3.0):
            v = np.float32(min(m * s, top) * np.float64(unit))
            base += [v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))]
    base = np.array([b for b in base if np.isfinite(b)], np.float32)
    rows = []
    for lead in (6.0, 5.0, 4.0, 10.5, 6 * 448.0, 6 * 2.0 ** -9, 3 * 2.0 ** -9):  # the block's largest value
        b = np.float32(min(lead, top) * np.float64(unit))
        small = base[np.abs(base) <= max(abs(b), np.float32(1e-45))]
        if not small.size or not np.isfinite(b):
            continue
        r = rng.choice(small, (24, 64)) * rng.choice([-1, 1], (24, 64))
        r[:, ::16] = b
        rows.append(r.astype(np.float32))
    x = torch.from_numpy(np.concatenate(rows)).to(DT[dtype])
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    check_quantize(mx, x, fmt, g)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_zero_subnormal_and_largest(mx, fmt):
    x = torch.zeros(5, 96)
    x[1] = 1e-45
    x[2, 3:40] = -1e-40
    x[3] = 3.4028234e38
    x[4, ::2] = -0.0
    check_quantize(mx, x, fmt)
    check_quantize(mx, torch.zeros(3, 40), fmt)
    check_quantize(mx, torch.full((2, 40), 1e-45), fmt)
    check_quantize(mx, x[:3].contiguous(), fmt)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_not_finite_blocks(mx, fmt, dtype):
    x = make(6, 96, dtype, 9)
    x[0, 5], x[1, 40], x[2, 95], x[3, 0] = float("inf"), float("-inf"), float("nan"), -float("nan")
    for rows in (6, 2100):  # few enough for one launch, and more
        q, want = check_quantize(mx, x.repeat(rows // 6, 1), fmt)
        got = mx.dequantize(q, torch.float32).cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_dequantize(mx, fmt, out):
    """code x scale is exact in FP32 (6 bits; the test's scales do not overflow it); mxfp4 is
    then rounded once, and nvfp4 once by the global scale in FP32 (half a step, 2^-24) and once
    to the output's type (2^-8, 2^-11, 2^-24 of the value, or half of FP16's smallest step)."""
    half = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}[out]
    tiny = 2.0 ** -25 if out == "fp16" else 2.0 ** -134 if out == "bf16" else 2.0 ** -150
    for i, (r, c) in enumerate(SHAPES):
        x = make(r, c, "bf16", 50 + i)
        q, want = check_quantize(mx, x, fmt)
        got = mx.dequantize(q, DT[out])
        assert got.dtype == DT[out] and tuple(got.shape) == (r, c)
        got = got.double().cpu().numpy()
        bound = np.abs(want) * (half + 2.0 ** -24) + tiny
        over = np.abs(want) > 65504 if out == "fp16" else np.zeros_like(want, bool)
        assert (np.abs(got - want) <= bound)[~over].all()
        if fmt == "mxfp4" and out == "fp32":
            assert np.array_equal(got, want)


def test_views_strides_and_leading_dimensions(mx):
    big = make(40, 200, "bf16", 1).cuda()
    for view in (big[:, 3:180], big[::2, :130], big.t(), big[5:6, 1:2], big[:, :1], big.view(4, 10, 200),
                 big.view(4, 10, 200)[:, 2:7, 5:77], big[0], big[:1].expand(7, 200)):
        for fmt in ("mxfp4", "nvfp4"):
            q, _ = check_quantize(mx, view.cpu(), fmt, xd=view)
            assert q.shape == tuple(view.shape) and mx.dequantize(q).shape == view.shape
    # out: rows inside a wider tensor, neighbours untouched, wherever they start
    x = make(9, 45, "bf16", 2)
    q, want = check_quantize(mx, x, "mxfp4")
    for off in range(9):
        wide = torch.full((9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        r = mx.dequantize(q, torch.bfloat16, out=wide[:, off:off + 45])
        assert r.data_ptr() == wide[:, off:].data_ptr()
        assert np.array_equal(wide[:, off:off + 45].float().cpu().numpy(), torch.from_numpy(want).bfloat16().float().numpy())
        wide[:, off:off + 45] = 7.0
        assert (wide == 7.0).all()


def test_empty_rows(mx):
    for fmt in ("mxfp4", "nvfp4"):
        q = mx.quantize(torch.zeros(0, 64, device="cuda"), fmt)
        assert q.rows == 0 and mx.dequantize(q).shape == (0, 64)


def test_other_stream_and_graph(mx):
    x = make(257, 300, "bf16", 4).cuda()
    want = [mx.dequantize(mx.quantize(x, f), torch.float32) for f in ("mxfp4", "nvfp4")]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream, 0, torch.cuda.default_stream()):
        got = [mx.dequantize(mx.quantize(x, f, stream=handle), torch.float32, stream=handle) for f in ("mxfp4", "nvfp4")]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    xs, ys = x.clone(), x.clone()
    with torch.cuda.graph(g):
        a = [mx.dequantize(mx.quantize(xs, f), torch.float32) for f in ("mxfp4", "nvfp4")]
    with torch.cuda.graph(g2):
        b = [mx.dequantize(mx.quantize(ys, f), torch.float32) for f in ("mxfp4", "nvfp4")]
    ys.mul_(3)
    xs.copy_(x * 2)
    for _ in range(3):
        g.replay()
        g2.replay()
    torch.cuda.synchronize()
    for r, src in ((a, x * 2), (b, x * 3)):
        for f, t in zip(("mxfp4", "nvfp4"), r):
            assert torch.equal(t, mx.dequantize(mx.quantize(src, f), torch.float32))


def test_a_matrix_past_32_bits(mx):
    """Byte offsets past 2^32: the last rows of a 4.4 GB matrix as those of a small one."""
    rows, cols = 1_100_003, 2048
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = make(200, cols, "bf16", 8)
    x[-200:] = tail.cuda()
    q = mx.quantize(x)
    code, byte, _ = U.quantize(tail.double().numpy(), "mxfp4")
    got, _ = U.unpack(q.codes.view(torch.uint8)[-200:].cpu().numpy(), 200, cols)
    assert np.array_equal(got, code)
    y = mx.dequantize(q)
    assert torch.equal(y[-200:].float().cpu(), torch.from_numpy(U.values(code, byte, "mxfp4")).float())
    assert not y[:-200].any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_rows_longer_than_the_grid(mx, fmt):
    """More columns than the blocks beside each other cover in the pass for the largest value
    (1024 blocks of 8192): the largest is the last."""
    x = make(1, 9_000_011, "fp32", 3)
    x[0, -1] = 50000.0
    check_quantize(mx, x, fmt)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (129, 47), (5, 4097), (128, 64)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_nothing_written_past_codes_scales_and_scale(mx, fmt, rows, cols):
    from lossless_float_weight_b200 import zipnn as Z
    f = {"mxfp4": Z.MXFP4, "nvfp4": Z.NVFP4}[fmt]
    x = make(rows, cols, "bf16", 1).cuda()
    nc, ns = rows * Z.zipnn_mx_row_bytes(cols), Z.zipnn_mx_scale_bytes(f, rows, cols)
    codes, scales = (torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda") for n in (nc, ns))
    g = torch.full((9,), 7.0, device="cuda")
    ws = torch.full((Z.MX_WORKSPACE_BYTES + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert Z.zipnn_mx_quantize(f, Z.VALUE_BF16, x.data_ptr(), rows, cols, cols, g[4:].data_ptr(), 1, codes[256:].data_ptr(),
                               scales[256:].data_ptr(), ws.data_ptr(), Z.MX_WORKSPACE_BYTES, s) == Z.OK
    q = mx.quantize(x, fmt)
    for buf, n, want in ((codes, nc, q.codes), (scales, ns, q.scales)):
        assert torch.equal(buf[256:256 + n], want.view(torch.uint8).reshape(-1))
        assert (buf[:256] == 0xA5).all() and (buf[256 + n:] == 0xA5).all()
    assert (ws[Z.MX_WORKSPACE_BYTES:] == 0x5A).all()
    assert (g[:4] == 7).all() and (g[5:] == 7).all() and (fmt == "mxfp4" or g[4] == q.global_scale[0])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_through_the_codec(mx, fmt):
    x = make(300, 500, "bf16", 12).cuda()
    q = mx.quantize(x, fmt)
    c = mx.compress(q, chunk_bytes=16384)
    assert c.nbytes < q.codes.numel() + q.scales.numel()
    r = mx.decompress(c)
    assert torch.equal(r.codes.view(torch.uint8), q.codes.view(torch.uint8))
    assert torch.equal(r.scales.view(torch.uint8), q.scales.view(torch.uint8)) and r.scales.dtype == q.scales.dtype
    assert torch.equal(mx.dequantize(r), mx.dequantize(q))


def test_through_the_codec_with_a_plan(mx):
    """An FP4 plan made on one weight's codes codes another's."""
    from lossless_float_weight_b200 import zipnn as Z
    a, b = (mx.quantize(make(256, 1024, "bf16", s).cuda()) for s in (20, 21))
    plan = Z.Plan.create(a.codes, groups=2, chunk_bytes=16384)
    c = mx.compress(b, chunk_bytes=16384, plan=plan)
    r = mx.decompress(c)
    assert torch.equal(r.codes.view(torch.uint8), b.codes.view(torch.uint8))
    assert torch.equal(mx.dequantize(r), mx.dequantize(b))


def test_kernel_timing_counts_the_launches(mx):
    from lossless_float_weight_b200 import pages, zipnn as Z
    x = make(300, 512, "bf16", 1).cuda()
    kv = torch.zeros(2, 8, 16, 8, device="cuda")
    pool = pages.PagePool(kv, 16, 4, 4)
    torch.cuda.synchronize()
    Z.kernel_times()
    assert Z.zipnn_timing_enable(1) == Z.OK
    try:
        q = mx.quantize(x, "nvfp4")
        mx.dequantize(q)
        mx.matmul(q, q)
        pool.fork([0], [-1], [20])
        pool.free([0], compact=True)
        t = Z.kernel_times()
    finally:
        Z.zipnn_timing_enable(0)
    got = {k: n for k, (ms, n) in t.items() if n}
    assert got == {"mx_amax": 1, "mx_quantize": 1, "mx_dequantize": 1, "mx_matmul": 1, "pages_plan": 3, "pages_move": 2}
    assert all(ms > 0 for ms, n in t.values() if n)


def test_block_scales_and_from_parts(mx):
    x = make(150, 333, "fp32", 5).cuda()
    for fmt in ("mxfp4", "nvfp4"):
        q = mx.quantize(x, fmt)
        s = q.block_scales()
        assert tuple(s.shape) == (150, -(-333 // U.BLOCK[fmt]))
        assert torch.equal(mx.tile_scales(s).view(torch.uint8), q.scales.view(torch.uint8))


def test_refusals_on_the_device(mx):
    from lossless_float_weight_b200 import zipnn as Z
    x = torch.zeros(4, 64, device="cuda")
    q, n = mx.quantize(x), mx.quantize(x, "nvfp4")
    one = torch.ones(1, device="cuda")
    for call in (lambda: mx.quantize(x, "mxfp4", one), lambda: mx.quantize(x, "nvfp4", one.double()),
                 lambda: mx.quantize(x, "nvfp4", torch.ones(2, device="cuda")), lambda: mx.quantize(x, "nvfp4", torch.ones(1)),
                 lambda: mx.quantize(x[:, :0]), lambda: mx.quantize(x.clone().requires_grad_()), lambda: mx.quantize(x[0, 0]), lambda: mx.dequantize(q, torch.float64),
                 lambda: mx.dequantize(q, torch.bfloat16, out=torch.empty(4, 64, device="cuda")),
                 lambda: mx.dequantize(q, torch.float32, out=torch.empty(64, 4, device="cuda").t()),
                 lambda: mx.MxTensor(q.codes, q.scales, (4, 64), "nvfp4"),
                 lambda: mx.MxTensor(n.codes, n.scales, (4, 64), "mxfp4", n.global_scale),
                 lambda: mx.MxTensor(q.codes[:2], q.scales, (4, 64), "mxfp4"),
                 lambda: mx.MxTensor(q.codes, q.scales[:-1], (4, 64), "mxfp4"),
                 lambda: mx.MxTensor(q.codes, q.scales.cpu(), (4, 64), "mxfp4")):
        with pytest.raises(Z.ZipnnError):
            call()
