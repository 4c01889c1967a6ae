"""The product of microscaled matrices against the 64-bit product of the values they stand for."""
import numpy as np
import pytest
import torch

import mx_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_float_weight_b200 import mx
    return mx


def random_mx(mx, rows, cols, fmt, seed, exact=False):
    """A random MxTensor and its values in 64 bits. exact: few scales near 1, so that FP32 sums
    of a product of two have no rounding."""
    rng = np.random.RandomState(seed)
    code = rng.randint(0, 16, (rows, cols))
    nb = -(-cols // U.BLOCK[fmt])
    if fmt == "mxfp4":
        byte = rng.randint(127, 129, (rows, nb)) if exact else rng.randint(115, 135, (rows, nb))
        g = None
    else:
        byte = rng.choice([0x30, 0x38, 0x34], (rows, nb)) if exact else rng.randint(0x20, 0x58, (rows, nb))
        g = 1.0 if exact else float(np.float32(rng.uniform(0.01, 3)))
    byte = byte.astype(np.uint8)
    pad = -cols % 32
    c = np.concatenate([code, np.zeros((rows, pad), code.dtype)], 1)
    packed = torch.from_numpy((c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8)).cuda()
    scales = mx.tile_scales(torch.from_numpy(byte)).cuda()
    t = mx.MxTensor(packed, scales, (rows, cols), fmt, None if g is None else torch.tensor([g], device="cuda"))
    return t, U.values(code, byte, fmt, g)


def check(mx, m, n, k, fmt, out, seed=0, exact=False):
    a, va = random_mx(mx, m, k, fmt, seed, exact)
    b, vb = random_mx(mx, n, k, fmt, seed + 1, exact)
    got = mx.matmul(a, b, DT[out])
    assert tuple(got.shape) == (m, n) and got.dtype == DT[out]
    want = va @ vb.T
    got = got.double().cpu().numpy()
    if exact:
        assert np.array_equal(got, torch.from_numpy(want).to(DT[out]).double().numpy()), (m, n, k)
        return
    # FP32 sums of k products in any order, with a step lost at each addition (2^-23 of the sum
    # of magnitudes), two roundings by the global scales, and the output's own
    bound = (np.abs(va) @ np.abs(vb).T) * ((k + 2) * 2.0 ** -23) + np.abs(want) * HALF[out] * (1 + k * 2.0 ** -23) + 2.0 ** -25
    over = np.abs(want) + bound > 65504 if out == "fp16" else np.zeros(want.shape, bool)
    err = np.abs(got - want)
    assert (err <= bound)[~over].all(), (m, n, k, float((err / bound)[~over].max()))


SIZES = [(1, 1, 1), (1, 128, 256), (1, 4096, 512), (3, 130, 64), (16, 256, 4096), (17, 300, 96), (32, 128, 1000), (33, 1, 40),
         (64, 640, 2048), (77, 512, 4080), (128, 128, 128), (129, 127, 31), (300, 5, 700), (200, 333, 1300), (257, 500, 33),
         (130, 1000, 260), (512, 384, 640), (5, 2000, 11008), (1800, 1500, 700), (1537, 2049, 33), (2500, 1281, 1111), (10300, 100, 64),
         (300, 5200, 2048)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_exact_sums(mx, fmt, size):
    """Scales of 1 and 2 (or 0.5, 0.75, 1): every partial sum is a whole number of quarters (or
    of 64ths) below 2^24 of them, so FP32 holds it and the order does not matter."""
    m, n, k = size
    k = min(k, 4096)
    check(mx, m, n, k, fmt, "fp32", 3, exact=True)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmt,out", [("mxfp4", "bf16"), ("mxfp4", "fp16"), ("nvfp4", "bf16"), ("nvfp4", "fp32")])
def test_products(mx, fmt, out, size):
    check(mx, *size, fmt, out, 5)


def test_out_with_strides_and_guards(mx):
    for m, n in ((7, 300), (300, 7), (140, 200)):
        a, va = random_mx(mx, m, 320, "mxfp4", 1, True)
        b, vb = random_mx(mx, n, 320, "mxfp4", 2, True)
        wide = torch.full((m + 2, n + 5), 9.0, device="cuda")
        r = mx.matmul(a, b, torch.float32, out=wide[1:-1, 3:-2])
        assert r.data_ptr() == wide[1:, 3:].data_ptr()
        assert np.array_equal(r.double().cpu().numpy(), va @ vb.T)
        wide[1:-1, 3:-2] = 9.0
        assert (wide == 9.0).all()


def test_leading_dimensions_plain_activations_and_empty(mx):
    g = torch.Generator().manual_seed(0)
    w = torch.randn(200, 96, generator=g).to(torch.bfloat16).cuda()
    x = torch.randn(2, 5, 96, generator=g).to(torch.bfloat16).cuda()
    for fmt in ("mxfp4", "nvfp4"):
        b = mx.quantize(w, fmt)
        y = mx.matmul(x, b)
        assert y.shape == (2, 5, 200)
        assert torch.equal(y, mx.matmul(mx.quantize(x, fmt), b))
        assert torch.equal(y.view(10, 200), mx.matmul(x.view(10, 96), b))
        assert mx.matmul(x[:0], b).shape == (0, 5, 200)
        assert torch.equal(mx.matmul(x[1, 2], b), mx.matmul(x[1, 2:3], b)[0])
        assert mx.matmul(x, mx.quantize(w[:0], fmt)).shape == (2, 5, 0)


@pytest.mark.parametrize("m,n", [(66_000, 33_000), (40, 70_000_000)])
def test_an_output_past_32_bits(mx, m, n):
    """2.2 and 2.8 billion results: some rows and columns of each end against the 64-bit product."""
    k = 64
    a, va = random_mx(mx, m, k, "mxfp4", 1, exact=True)
    if n < 100_000:
        b, vb = random_mx(mx, n, k, "mxfp4", 2, exact=True)
    else:  # the same rows again and again
        b, vb = random_mx(mx, 1 << 12, k, "mxfp4", 2, exact=True)
        reps = -(-n // (1 << 12))
        rows = reps << 12
        b = mx.MxTensor(b.codes.repeat(reps, 1)[:n].contiguous(),
                        b.scales.view(torch.uint8).repeat(reps)[: -(-n // 128) * 512].contiguous(), (n, k), "mxfp4")
        assert rows >= n
    y = mx.matmul(a, b, torch.bfloat16)
    i, j = np.r_[0:3, m // 2, m - 3:m], np.r_[0:3, n // 2, n - 3:n]
    got = y[torch.from_numpy(i).cuda()][:, torch.from_numpy(j).cuda()].double().cpu().numpy()
    want = va[i] @ vb[j % vb.shape[0]].T
    assert np.array_equal(got, torch.from_numpy(want).to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("m,n", [(3, 200), (100, 300), (1700, 1600)])
@pytest.mark.parametrize("ga,gb", [(-100, 100), (-140, 120), (-30, -90), (-126, -10), (60, 60)])
def test_scales_of_far_apart_tensors(mx, m, n, ga, gb):
    """Powers of two, so that the sums stay exact: no scale alone takes a result out of range."""
    a, va = random_mx(mx, m, 96, "nvfp4", 1, exact=True)
    b, vb = random_mx(mx, n, 96, "nvfp4", 2, exact=True)
    a.global_scale.fill_(2.0 ** ga)
    b.global_scale.fill_(2.0 ** gb)
    y = mx.matmul(a, b, torch.float32).double().cpu().numpy()
    with np.errstate(over="ignore"):
        assert np.array_equal(y, (va @ vb.T * 2.0 ** (ga + gb)).astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_nan_blocks_stay_in_their_rows(mx, fmt):
    g = torch.Generator().manual_seed(1)
    w, x = torch.randn(140, 200, generator=g), torch.randn(20, 200, generator=g)
    w[3, 7] = float("nan")
    x[5, 199] = float("inf")
    y = mx.matmul(mx.quantize(x.cuda(), fmt), mx.quantize(w.cuda(), fmt), torch.float32).cpu()
    bad = torch.zeros(20, 140, dtype=torch.bool)
    bad[:, 3], bad[5] = True, True
    assert torch.equal(torch.isnan(y), bad)


def test_same_bits_each_time_two_streams_and_graphs(mx):
    a, _ = random_mx(mx, 5, 4096, "nvfp4", 1)
    b, _ = random_mx(mx, 1000, 4096, "nvfp4", 2)
    c, _ = random_mx(mx, 300, 4096, "nvfp4", 3)
    want = [mx.matmul(x, b, torch.float32) for x in (a, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [mx.matmul(x, b, torch.float32, stream=s) for x, s in zip((a, c), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    x = torch.randn(5, 4096, device="cuda")
    with torch.cuda.graph(graph):
        y = mx.matmul(x, b, torch.float32)
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, mx.matmul(x, b, torch.float32))
    from lossless_float_weight_b200 import zipnn as Z
    assert mx.status() == Z.OK


def test_every_kind_of_block_at_once(mx):
    """Products of all the kernels' shapes side by side on six streams, again and again: equal
    bits each time, whatever shares an SM with whatever."""
    sizes = [(1, 4096, 2048, "nvfp4"), (17, 3000, 1024, "nvfp4"), (64, 2000, 4096, "mxfp4"), (128, 4096, 2048, "nvfp4"),
             (1700, 1600, 512, "mxfp4"), (1537, 2049, 640, "nvfp4"), (100, 20000, 512, "mxfp4"), (9, 128, 11008, "mxfp4")]
    ab = [(random_mx(mx, m, k, f, 1)[0], random_mx(mx, n, k, f, 2)[0]) for m, n, k, f in sizes]
    want = [mx.matmul(a, b) for a, b in ab]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    for turn in range(10):
        got = [mx.matmul(a, b, stream=streams[(i + turn) % 6]) for i, (a, b) in enumerate(ab) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(got[3 * i + j], want[i]) for i in range(len(ab)) for j in range(3))
    from lossless_float_weight_b200 import zipnn as Z
    assert mx.status() == Z.OK


def test_weights_through_the_codec(mx):
    """A weight quantised, compressed, decompressed and multiplied, as a stored model is used."""
    g = torch.Generator().manual_seed(4)
    w = torch.randn(384, 512, generator=g).to(torch.bfloat16).cuda()
    x = torch.randn(9, 512, generator=g).to(torch.bfloat16).cuda()
    for fmt in ("mxfp4", "nvfp4"):
        q = mx.quantize(w, fmt)
        r = mx.decompress(mx.compress(q))
        y = mx.matmul(x, r, torch.float32)
        assert torch.equal(y, mx.matmul(x, q, torch.float32))
        want = mx.dequantize(mx.quantize(x, fmt), torch.float32).double() @ mx.dequantize(q, torch.float32).double().t()
        # FP32 sums of 512 products, and values read back in FP32 (one rounding each for nvfp4)
        mag = mx.dequantize(mx.quantize(x, fmt), torch.float32).double().abs() @ mx.dequantize(q, torch.float32).double().abs().t()
        assert ((y.double() - want).abs() <= mag * 516 * 2.0 ** -23).all()


def test_refusals(mx):
    from lossless_float_weight_b200 import zipnn as Z
    a, b = mx.quantize(torch.zeros(4, 64, device="cuda")), mx.quantize(torch.zeros(8, 64, device="cuda"))
    n, s = mx.quantize(torch.zeros(8, 64, device="cuda"), "nvfp4"), mx.quantize(torch.zeros(8, 65, device="cuda"))
    for call in (lambda: mx.matmul(a, n), lambda: mx.matmul(a, s), lambda: mx.matmul(a, b, torch.float64),
                 lambda: mx.matmul(a, torch.zeros(8, 64, device="cuda")), lambda: mx.matmul(torch.zeros(4, 64), b),
                 lambda: mx.matmul(a, mx.quantize(torch.zeros(2, 4, 64, device="cuda"))),
                 lambda: mx.matmul(a, b, out=torch.zeros(4, 8, device="cuda")),
                 lambda: mx.matmul(a, b, torch.float32, out=torch.zeros(8, 4, device="cuda").t())):
        with pytest.raises(Z.ZipnnError):
            call()
