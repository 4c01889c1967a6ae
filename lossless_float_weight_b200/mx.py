"""Microscaled 4-bit tensors: made, read back, multiplied, and stored compressed.

A matrix of E2M1 values whose blocks share a scale ("mxfp4": 32 values, E8M0 scales;
"nvfp4": 16 values, E4M3 scales and one FP32 scale of the tensor), in the layout of
include/zipnn.h. The codes are what the codec stores as FP4 and the scales as FP8, so a
quantised weight or K/V cache goes through :func:`compress` and comes back bit for bit::

    q = mx.quantize(w)                  # w: (..., K) BF16, FP16 or FP32
    w4 = mx.dequantize(q)               # BF16 values
    y = mx.matmul(x, q)                 # x (..., K), quantised alike, against the weight
    c = mx.compress(q)                  # two containers of the codec
    q2 = mx.decompress(c)               # the same codes and scales

The functions check their arguments, allocate with PyTorch and call the CUDA library on
the current stream of the tensors' device (or `stream`); they do not synchronise, except
:func:`compress` and :func:`decompress`, as the codec's own. They are for stored and served
tensors: no gradient passes through them, and an input or output that asks for one, in
reverse or forward mode, is refused.
"""
import torch
from torch.autograd import forward_ad

from . import zipnn as Z

BLOCK = {"mxfp4": 32, "nvfp4": 16}
_FORMATS = {"mxfp4": Z.MXFP4, "nvfp4": Z.NVFP4}
_SCALE_DTYPES = {"mxfp4": torch.float8_e8m0fnu, "nvfp4": torch.float8_e4m3fn}
_VALUES = {torch.bfloat16: Z.VALUE_BF16, torch.float32: Z.VALUE_FP32, torch.float16: Z.VALUE_FP16}


def _fail(what):
    raise Z.ZipnnError(Z.ERR_INVALID_ARG, what)


def _format(format):
    f = _FORMATS.get(format)
    return f if f is not None else _fail(f"mx: format {format!r} is not one of {sorted(_FORMATS)}")


def _no_gradient(t, what):
    """Refuses a tensor that a gradient is to pass through, in either mode."""
    if t.requires_grad and torch.is_grad_enabled():
        _fail(f"{what}: no gradient passes through this call; detach it or use torch.no_grad()")
    if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
        _fail(f"{what}: no gradient passes through this call; unpack the dual tensor")


# the handle of a device's current stream; the public way to it builds a Stream object, which
# takes longer (3.2 us) than the whole call of a small operator
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


# says that tensors were written through their addresses, so that a backward pass that saved one
# of them notices (the public name does the same in 0.3 us more)
_written = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def _call(fn, what, device, *args):
    """fn(*args, stream) on the current stream of the tensors' device, made current."""
    i = device.index
    if i == torch.cuda.current_device():
        status = fn(*args, _current_stream(i))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(i))
    if status:
        Z.check(status, what)


def _use(stream, device):
    """`stream` (a torch stream or a raw handle on `device`) as the current one: what a call
    allocates then belongs to the stream that writes it."""
    if device.type != "cuda":
        _fail(f"a call on a stream: tensors on {device}")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device)
    elif stream.device != device:  # else the work would go to the current stream of the tensors' device
        _fail(f"a stream of {stream.device} for tensors on {device}")
    return torch.cuda.stream(stream)


def _row_bytes(cols):
    return (cols + 31) // 32 * 16  # zipnn_mx_row_bytes


def _scale_bytes(format, rows, cols):
    per = 4 * BLOCK[format]
    return (rows + 127) // 128 * ((cols + per - 1) // per) * 512  # zipnn_mx_scale_bytes


def _rows(shape):
    n = 1
    for d in shape[:-1]:
        n *= d
    return n


class MxTensor:
    """A microscaled 4-bit tensor of `shape` (its last dimension in blocks).

    codes: one row of zipnn_mx_row_bytes(shape[-1]) bytes for each row of the flattened
    leading dimensions (torch.float4_e2m1fn_x2 or uint8, contiguous); scales: the 1-D tiles
    of the blocks' scales (one byte each); global_scale: a one-element FP32 CUDA tensor for
    "nvfp4", None for "mxfp4". A tensor without rows has empty codes and scales."""

    __slots__ = ("codes", "scales", "shape", "format", "global_scale", "rows", "cols")

    def __init__(self, codes, scales, shape, format, global_scale=None):
        f = _format(format)
        self.codes, self.scales, self.format, self.global_scale = codes, scales, format, global_scale
        self.shape = shape if type(shape) is tuple else tuple(shape)
        if not self.shape or min(self.shape) < 0 or self.shape[-1] == 0:
            _fail("MxTensor: at least one dimension, the last not empty")
        self.cols = self.shape[-1]
        self.rows = self.shape[0] if len(self.shape) == 2 else _rows(self.shape)
        if self.rows > 1 << 31 or self.cols > 1 << 30:
            _fail("MxTensor: at most 2^31 rows and 2^30 columns")
        if not (codes.is_cuda and codes.is_contiguous() and codes.element_size() == 1 and
                codes.numel() == self.rows * _row_bytes(self.cols)):
            _fail("MxTensor: codes are rows x zipnn_mx_row_bytes(cols) contiguous CUDA bytes")
        if not (scales.device == codes.device and scales.is_contiguous() and scales.element_size() == 1 and
                scales.numel() == _scale_bytes(format, self.rows, self.cols)):
            _fail("MxTensor: scales are zipnn_mx_scale_bytes contiguous bytes beside the codes")
        if f == Z.NVFP4:
            g = global_scale
            if g is None or g.dtype != torch.float32 or g.numel() != 1 or g.device != codes.device:
                _fail("MxTensor: nvfp4 has a global_scale, one FP32 value on the codes' device")
        elif global_scale is not None:
            _fail("MxTensor: mxfp4 has no global_scale")

    @classmethod
    def _of(cls, codes, scales, shape, rows, cols, format, global_scale):
        """What a call of this module made, which needs no checks."""
        q = object.__new__(cls)
        q.codes, q.scales, q.shape, q.rows, q.cols, q.format, q.global_scale = codes, scales, shape, rows, cols, format, global_scale
        return q

    @property
    def device(self):
        return self.codes.device

    @property
    def _global(self):
        return None if self.global_scale is None else self.global_scale.data_ptr()

    def block_scales(self):
        """The scales as a (rows, blocks) tensor, one to a block (a copy)."""
        nb = -(-self.cols // BLOCK[self.format])
        t = self.scales.view(torch.uint8).view(-(-self.rows // 128), -(-nb // 4), 32, 4, 4)
        return t.permute(0, 3, 2, 1, 4).reshape(-1, 4 * t.shape[1])[:self.rows, :nb].contiguous().view(self.scales.dtype)


def tile_scales(block_scales):
    """A (rows, blocks) tensor of one-byte scales in the tiles of MxTensor.scales."""
    r, nb = block_scales.shape
    s = torch.nn.functional.pad(block_scales.view(torch.uint8), (0, -nb % 4, 0, -r % 128))
    s = s.view(-(-r // 128), 4, 32, -(-nb // 4), 4).permute(0, 3, 2, 1, 4)
    return s.reshape(-1).view(block_scales.dtype)


def quantize(x, format="mxfp4", global_scale=None, stream=None):
    """Quantise the CUDA tensor x (..., K) in blocks along its last dimension.

    nvfp4: global_scale is a one-element FP32 CUDA tensor (positive and finite; taken as it is,
    and kept by the result, whose values change with it), or None: then it is found from x (its
    largest finite magnitude / 2688). Rounding, saturation and what a block with a NaN gives:
    zipnn_mx_quantize."""
    if stream is not None:
        with _use(stream, x.device):
            return quantize(x, format, global_scale)
    f, type, shape = _format(format), _VALUES.get(x.dtype), tuple(x.shape)
    if type is None or not x.is_cuda or not shape or shape[-1] == 0:
        _fail("mx.quantize: a CUDA tensor (..., K) of BF16, FP16 or FP32")
    _no_gradient(x, "mx.quantize: x")
    if type != Z.VALUE_BF16 and x.is_neg():
        x = x.resolve_neg()  # a part of a conjugated complex tensor (of which BF16 has none)
    dev, cols = x.device, shape[-1]
    if len(shape) == 2:
        m, rows = x, shape[0]
    else:
        m = x.reshape(-1, cols)
        rows = m.shape[0]
    stride = cols
    if not m.is_contiguous():
        stride = m.stride(0) if rows > 1 else cols
        if (cols > 1 and m.stride(1) != 1) or stride < cols:
            m, stride = m.contiguous(), cols
    find = False
    if f == Z.NVFP4:
        find = global_scale is None
        if find:
            global_scale = torch.empty(1, dtype=torch.float32, device=dev)
        elif global_scale.dtype != torch.float32 or global_scale.numel() != 1 or global_scale.device != dev:
            _fail("mx.quantize: global_scale is one FP32 value on x's device")
        else:
            _no_gradient(global_scale, "mx.quantize: global_scale")
    elif global_scale is not None:
        _fail("mx.quantize: mxfp4 has no global_scale")
    if rows > 1 << 31 or cols > 1 << 30:
        _fail("mx.quantize: at most 2^31 rows and 2^30 columns")
    codes = torch.empty(rows, _row_bytes(cols), dtype=torch.float4_e2m1fn_x2, device=dev)
    scales = torch.empty(_scale_bytes(format, rows, cols), dtype=_SCALE_DTYPES[format], device=dev)
    if rows:
        ws = None
        if find and rows * ((cols + 31) // 32) > Z.MX_SMALL:
            ws = torch.empty(Z.MX_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
        _call(Z.zipnn_mx_quantize, "zipnn_mx_quantize", dev, f, type, m.data_ptr(), rows, cols, stride,
              None if global_scale is None else global_scale.data_ptr(), find, codes.data_ptr(), scales.data_ptr(),
              None if ws is None else ws.data_ptr(), Z.MX_WORKSPACE_BYTES)
    elif find:
        global_scale.fill_(1.0)
    return MxTensor._of(codes, scales, shape, rows, cols, format, global_scale)


def _out(out, shape, dtype, device, what):
    """The caller's tensor where it can be written: its last dimension contiguous."""
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device:
        _fail(f"{what}: out is a {dtype} tensor {tuple(shape)} on {device}")
    if out.is_neg():
        _fail(f"{what}: out is a negated view")
    _no_gradient(out, f"{what}: out")
    if not (out.is_contiguous() or (out.dim() == 2 and (out.shape[1] == 1 or out.stride(1) == 1) and out.stride(0) >= out.shape[1])):
        _fail(f"{what}: out's rows are contiguous and do not overlap")
    return out


def dequantize(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values of q as a tensor of its shape (BF16, FP16 or FP32)."""
    if not isinstance(q, MxTensor):
        _fail("mx.dequantize: an MxTensor")
    if stream is not None:
        with _use(stream, q.device):
            return dequantize(q, dtype, out)
    type = _VALUES.get(dtype)
    if type is None:
        _fail("mx.dequantize: to BF16, FP16 or FP32")
    dev, stride = q.codes.device, q.cols
    given = out is not None
    if not given:
        out = torch.empty(*q.shape, dtype=dtype, device=dev)  # sizes one by one: a tuple takes 0.7 us to read
    else:
        _out(out, q.shape, dtype, dev, "mx.dequantize")
        stride = out.stride(0) if out.dim() == 2 and q.rows > 1 else stride
    if q.rows:
        _call(Z.zipnn_mx_dequantize, "zipnn_mx_dequantize", dev, _FORMATS[q.format], type, q.codes.data_ptr(),
              q.scales.data_ptr(), q._global, q.rows, q.cols, out.data_ptr(), stride)
    if given:
        _written((out,))
    return out


def matmul(a, b, dtype=torch.bfloat16, out=None, stream=None):
    """a @ b.T for a (..., K) and b (N, K) of one format, FP32 sums, as BF16, FP16 or FP32
    (..., N). a may be a BF16, FP16 or FP32 tensor: it is then quantised in b's format first
    (activations against a quantised weight); see zipnn_mx_matmul."""
    if stream is not None:
        with _use(stream, b.device):
            return matmul(a, b, dtype, out)
    if not isinstance(b, MxTensor):
        _fail("mx.matmul: b is an MxTensor")
    if not isinstance(a, MxTensor):
        a = quantize(a, b.format)
    dev, type = a.codes.device, _VALUES.get(dtype)
    if a.format != b.format or a.cols != b.cols or len(b.shape) != 2 or b.codes.device != dev or type is None:
        _fail("mx.matmul: a (..., K) and b (N, K) of one format, on one device, to BF16, FP16 or FP32")
    shape, stride = a.shape[:-1] + (b.rows,), b.rows
    given = out is not None
    if not given:
        out = torch.empty(*shape, dtype=dtype, device=dev)
    else:
        _out(out, shape, dtype, dev, "mx.matmul")
        stride = out.stride(0) if out.dim() == 2 and a.rows > 1 else stride
    if a.rows and b.rows:
        _call(Z.zipnn_mx_matmul, "zipnn_mx_matmul", dev, _FORMATS[a.format], a.codes.data_ptr(), a.scales.data_ptr(),
              a._global, b.codes.data_ptr(), b.scales.data_ptr(), b._global, a.rows, b.rows, a.cols, type, out.data_ptr(),
              stride)
    if given:
        _written((out,))
    return out


def status(device=None):
    """Z.OK, or Z.ERR_TIMEOUT if a product on the device gave up since this was last asked
    (waits for the current stream)."""
    with torch.cuda.device(device):
        return Z.zipnn_mx_status(torch.cuda.current_stream().cuda_stream)


class MxContainers:
    """A microscaled tensor compressed: a container of its codes (FP4) and one of its scales
    (as FP8 values), and what it takes to put them together again."""

    def __init__(self, codes, scales, shape, format, global_scale, chunk_bytes):
        self.codes, self.scales, self.shape, self.format = codes, scales, shape, format
        self.global_scale, self.chunk_bytes = global_scale, chunk_bytes

    @property
    def nbytes(self):
        return self.codes.numel() + self.scales.numel()


def compress(q, chunk_bytes=Z.DEFAULT_CHUNK_BYTES, plan=None, stream=None):
    """Compress a microscaled tensor's codes (with `plan`, an FP4 plan, if given) and scales
    with the codec (synchronises)."""
    if q.rows == 0:
        _fail("mx.compress: an empty tensor")
    with torch.cuda.device(q.device):
        codes = Z.compress(q.codes.view(torch.float4_e2m1fn_x2), chunk_bytes, plan, stream=stream)
        scales = Z.compress(q.scales.view(torch.float8_e4m3fn), chunk_bytes, stream=stream)
        # a copy, as of the codes: what becomes of q does not reach what is stored
        g = None if q.global_scale is None else q.global_scale.clone()
    return MxContainers(codes, scales, q.shape, q.format, g, chunk_bytes)


def decompress(c, stream=None):
    """The microscaled tensor of mx.compress, bit for bit (synchronises)."""
    rows, cols = _rows(c.shape), c.shape[-1]
    with torch.cuda.device(c.codes.device):
        codes = Z.decompress(c.codes, torch.float4_e2m1fn_x2, (rows, Z.zipnn_mx_row_bytes(cols)), c.chunk_bytes, stream)
        scales = Z.decompress(c.scales, torch.float8_e4m3fn, (Z.zipnn_mx_scale_bytes(_FORMATS[c.format], rows, cols),),
                              c.chunk_bytes, stream)
        g = None if c.global_scale is None else c.global_scale.clone()
    return MxTensor(codes, scales.view(_SCALE_DTYPES[c.format]), c.shape, c.format, g)
