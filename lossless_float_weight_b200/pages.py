"""Pages of a served K/V cache: copied, shared when a sequence forks, given back, closed up,
and stored compressed.

A pool is one CUDA tensor of shape (planes, pages, ...): page p of a plane holds
`page_tokens` positions of the K or V of one layer. :class:`PagePool` keeps beside it which
sequence holds which page (the references, lengths and tables of include/zipnn.h)::

    pool = pages.PagePool(kv, page_tokens=16, max_seqs=64, max_pages=256)
    pool.fork([0], [-1], [700])          # sequence 0: 700 positions, fresh pages
    pool.fork([1], [0], [650])           # sequence 1: its first 650, shared where whole
    stored = pool.store(0)               # sequence 0's pages through the codec
    pool.free([0], compact=True)         # its references back, and the gaps closed
    pool.load(stored, 2)                 # the same positions in row 2

`fork`, `free`, `compact`, `copy`, `gather` and `scatter` launch kernels on the current stream (or
`stream`), and do no more where their lists are int32 tensors on the device: a Python list is
copied there first, which waits and cannot be captured. What they find wrong is read with
`status()`. `copy` without a workspace, `store` and `load` synchronise. The calls on one pool
share its books and its workspace: on several streams, the caller has them follow one another.
No gradient passes through any of them, and pages that ask for one are refused.
"""
import ctypes
import math

import torch

from . import zipnn as Z
from .mx import _call, _fail, _no_gradient, _use, _written


def _codec_dtype(dtype, what):
    """The codec's type that stores a dtype by its bits."""
    if dtype in Z._TORCH_DTYPES:
        return dtype
    return {1: torch.float8_e4m3fn, 2: torch.bfloat16, 4: torch.float32}.get(dtype.itemsize) or \
        _fail(f"{what}: pages of {dtype}, which the codec has no type for")


def copy_workspace(device="cuda"):
    """A workspace for `copy`, to be kept between calls (making one takes longer than a small
    copy): its status stays at the first error until it is zeroed."""
    return torch.zeros(256, dtype=torch.uint8, device=device)


def _pool_desc(t, what):
    """(descriptor, bytes of a page) of a (planes, pages, ...) CUDA tensor with contiguous pages."""
    if not t.is_cuda or t.dim() < 3:
        _fail(f"{what}: a CUDA tensor (planes, pages, ...)")
    shape, size = t.shape, t.element_size()
    planes, count = shape[0], shape[1]
    if t.is_contiguous():
        n = planes * count
        page = t.numel() * size // n if n else math.prod(shape[2:]) * size
        return Z.PagePoolDesc(t.data_ptr(), page * count, page, planes, count), page
    n = 1
    for d in range(t.dim() - 1, 1, -1):
        if shape[d] != 1 and t.stride(d) != n:
            _fail(f"{what}: pages are contiguous")
        n *= shape[d]
    # the stride of a dimension of one element says nothing
    page = t.stride(1) * size if count > 1 else n * size
    return Z.PagePoolDesc(t.data_ptr(), t.stride(0) * size if planes > 1 else page * count, page, planes, count), n * size


def _ids(v, device, what):
    """A list of int32 numbers on the device; a Python sequence is copied there."""
    if isinstance(v, torch.Tensor):
        if v.dtype != torch.int32 or v.device != device or v.dim() != 1 or not v.is_contiguous():
            _fail(f"{what}: a contiguous 1-D int32 tensor on {device}")
        return v
    return torch.tensor(list(v), dtype=torch.int32, device=device)


def copy(src, src_ids, dst, dst_ids, count=None, ws=None, stream=None):
    """Copy pages of src into dst (both (planes, pages, ...), of one page size): pair i from
    page src_ids[i] to page dst_ids[i]; None for page i itself; negative numbers skip a pair.
    Returns dst. Errors found on the device (zipnn_pages_copy) are in Z.status(ws); without
    `ws` (copy_workspace) the call synchronises and raises them."""
    if stream is not None:
        with _use(stream, dst.device):
            return copy(src, src_ids, dst, dst_ids, count, ws)
    _no_gradient(src, "pages.copy: src")
    _no_gradient(dst, "pages.copy: dst")
    a, na = _pool_desc(src, "pages.copy: src")
    b, nb = _pool_desc(dst, "pages.copy: dst")
    if na != nb or src.device != dst.device or a.planes != b.planes:
        _fail("pages.copy: src and dst have the same planes and page size, on one device")
    n = min(a.pages, b.pages)
    if src_ids is not None:
        src_ids = _ids(src_ids, dst.device, "pages.copy: src_ids")
        n = src_ids.numel()
    if dst_ids is not None:
        dst_ids = _ids(dst_ids, dst.device, "pages.copy: dst_ids")
        if src_ids is not None and dst_ids.numel() != n:
            _fail("pages.copy: as many destinations as sources")
        n = dst_ids.numel()
    if count is not None:
        if not 0 <= count <= n:
            _fail("pages.copy: count is at most the lists' length")
        n = count
    if n == 0 or na == 0 or a.planes == 0:
        return dst
    if ws is not None and ws.device != dst.device:
        _fail("pages.copy: a workspace on the pages' device")
    wait = ws is None
    if wait:
        ws = copy_workspace(dst.device)
    _call(Z.zipnn_pages_copy, "zipnn_pages_copy", dst.device, ctypes.byref(a),
          None if src_ids is None else src_ids.data_ptr(), ctypes.byref(b),
          None if dst_ids is None else dst_ids.data_ptr(), n, na, ws.data_ptr(), ws.numel())
    _written((dst,))
    if wait:
        with torch.cuda.device(dst.device):
            Z.check(Z.status(ws), "pages.copy")
    return dst


class StoredPages:
    """One sequence's pages as a container of the codec, its length, and what its pages were
    (planes, shape, type and positions of a page)."""

    def __init__(self, container, length, chunk_bytes, pages):
        self.container, self.length, self.chunk_bytes, self.pages = container, length, chunk_bytes, pages


class PagePool:
    """The pages of a cache and the sequences that hold them.

    pages: CUDA tensor (planes, P, ...), each page contiguous and a multiple of 16 bytes.
    max_seqs rows of max_pages slots. `meta` is one int32 tensor with refs (P), lens
    (max_seqs) and tables (max_seqs x max_pages) one behind the other; given, it is taken as
    it is (max_pages follows from its length), else it starts with every page free."""

    def __init__(self, pages, page_tokens, max_seqs, max_pages=None, meta=None):
        self._pool, self.page_bytes = _pool_desc(pages, "PagePool: pages")
        P = pages.shape[1]
        if not 1 <= max_seqs <= 1 << 18 or not 1 <= page_tokens < 1 << 31:
            _fail("PagePool: 1 to 2^18 sequences, 1 to 2^31 - 1 positions of a page")
        if meta is None:
            if max_pages is None or max_pages < 1 or max_seqs * max_pages >= 1 << 31:
                _fail("PagePool: max_pages, at least 1 (max_seqs x max_pages below 2^31), or meta")
            meta = torch.full((P + max_seqs * (1 + max_pages),), -1, dtype=torch.int32, device=pages.device)
            meta[:P + max_seqs] = 0
        slots = (meta.numel() - P - max_seqs) // max_seqs
        if meta.dtype != torch.int32 or meta.device != pages.device or meta.dim() != 1 or not meta.is_contiguous() or \
                slots < 1 or meta.numel() != P + max_seqs * (1 + slots) or (max_pages is not None and max_pages != slots):
            _fail("PagePool: meta is int32, pages + max_seqs x (1 + max_pages) long, beside the pages")
        self.pages, self.meta, self.page_tokens, self.device = pages, meta, page_tokens, pages.device
        self._books = (pages, meta)  # what fork and compact write
        self.refs, self.lens = meta[:P], meta[P:P + max_seqs]
        self.tables = meta[P + max_seqs:].view(max_seqs, slots)
        self._table = Z.PageTableDesc(self.refs.data_ptr(), self.lens.data_ptr(), self.tables.data_ptr(), max_seqs, slots,
                                      page_tokens)
        self.ws = torch.zeros(Z.zipnn_pages_workspace_bytes(max_seqs, P), dtype=torch.uint8, device=pages.device)
        self._pool_ref, self._table_ref = ctypes.byref(self._pool), ctypes.byref(self._table)
        self._ws_ptr, self._ws_bytes = self.ws.data_ptr(), self.ws.numel()
        self.live = self.ws[4:8].view(torch.int32)  # pages in use, as the last `compact` counted them

    def fork(self, rows, parents, lens, stream=None):
        """rows[j] becomes a sequence of lens[j] positions: new (parents[j] = -1), the start of
        another row's, or the row itself grown (parents[j] = rows[j]); zipnn_pages_fork."""
        if stream is not None:
            with _use(stream, self.device):
                return self.fork(rows, parents, lens)
        _no_gradient(self.pages, "PagePool.fork: pages")
        rows, parents, lens = (_ids(v, self.device, "PagePool.fork") for v in (rows, parents, lens))
        n = rows.numel()
        if parents.numel() != n or lens.numel() != n or n > self._table.seqs:
            _fail("PagePool.fork: a parent and a length for each row, each row at most once")
        _call(Z.zipnn_pages_fork, "zipnn_pages_fork", self.device, self._pool_ref, self.page_bytes, self._table_ref, rows.data_ptr(),
              parents.data_ptr(), lens.data_ptr(), n, self._ws_ptr, self._ws_bytes)
        _written(self._books)

    def free(self, rows, compact=False, stream=None):
        """The sequences in `rows` give their pages back; with compact, the gaps are closed
        (zipnn_pages_free; `live` then holds how many pages are in use)."""
        if stream is not None:
            with _use(stream, self.device):
                return self.free(rows, compact)
        _no_gradient(self.pages, "PagePool.free: pages")
        rows = None if isinstance(rows, (tuple, list)) and not rows else _ids(rows, self.device, "PagePool.free")
        _call(Z.zipnn_pages_free, "zipnn_pages_free", self.device, self._pool_ref, self.page_bytes, self._table_ref,
              None if rows is None else rows.data_ptr(), 0 if rows is None else rows.numel(), compact, self._ws_ptr,
              self._ws_bytes)
        _written(self._books if compact else (self.meta,))

    def compact(self, stream=None):
        """Close the gaps: afterwards the pages in use are the first `live` ones."""
        self.free((), compact=True, stream=stream)

    def gather(self, ids, out=None, stream=None):
        """The pages `ids` as a contiguous (planes, len(ids), ...) tensor. What a number outside
        the pool (which the status tells of) or below 0 stands for is left as it was in `out`."""
        if stream is not None:
            with _use(stream, self.device):
                return self.gather(ids, out)
        ids = _ids(ids, self.device, "PagePool.gather")
        if out is None:
            out = torch.empty(self.pages.shape[:1] + ids.shape + self.pages.shape[2:], dtype=self.pages.dtype, device=self.device)
        return copy(self.pages, ids, out, None, ids.numel(), self.ws)

    def scatter(self, values, ids, stream=None):
        """The pages of a (planes, len(ids), ...) tensor into the pages `ids`."""
        copy(values, None, self.pages, ids, ws=self.ws, stream=stream)

    def status(self, clear=False):
        """The first error that a call on this pool found on the device since the status was
        cleared (Z.OK if none); waits for the current stream."""
        with torch.cuda.device(self.device):
            s = Z.status(self.ws)
        if clear:
            self.ws[:4].zero_()
        return s

    def _held(self, row):
        """(length, page numbers on the device) of a row; waits."""
        if not 0 <= row < self._table.seqs:
            _fail("PagePool: row out of range")
        n = int(self.lens[row])
        return n, self.tables[row, : -(-n // self.page_tokens)]

    @property
    def _page(self):
        return self.pages.shape[0], tuple(self.pages.shape[2:]), self.pages.dtype, self.page_tokens

    def store(self, row, chunk_bytes=Z.DEFAULT_CHUNK_BYTES, plan=None):
        """The pages of the sequence in `row`, gathered and compressed (synchronises). The row
        keeps them; free it to give them back. A row whose length or page numbers do not fit the
        pool is refused with Z.ERR_CORRUPT."""
        n, ids = self._held(row)
        if n == 0:
            _fail("PagePool.store: an empty row")
        # a row that the pool's own calls would report as damaged: what gather leaves of such
        # pages is whatever was in the memory
        held = -(-n // self.page_tokens)
        if n < 0 or held > self._table.slots or not all(0 <= p < self._pool.pages for p in ids.tolist()):
            raise Z.ZipnnError(Z.ERR_CORRUPT, f"PagePool.store: row {row}")
        flat = self.gather(ids)
        with torch.cuda.device(self.device):
            c = Z.compress(flat.view(_codec_dtype(flat.dtype, "PagePool.store")), chunk_bytes, plan)
        return StoredPages(c, n, chunk_bytes, self._page)

    def load(self, stored, row):
        """A stored sequence back into the empty `row`, in fresh pages (synchronises)."""
        if stored.pages != self._page:
            _fail("PagePool.load: a sequence of pages of another shape, type or length")
        if stored.container.device != self.device:
            _fail(f"PagePool.load: a sequence on {stored.container.device}, pages on {self.device}")
        dt = self.pages.dtype
        codec = _codec_dtype(dt, "PagePool.load")
        Z.check(self.status(), "PagePool.load: an earlier call")
        # decoded before the row takes its pages: what can fail there (a damaged container, no
        # memory) then changes nothing
        shape = self.pages.shape[:1] + (-(-stored.length // self.page_tokens),) + self.pages.shape[2:]
        with torch.cuda.device(self.device):
            flat = Z.decompress(stored.container, codec, shape, stored.chunk_bytes).view(dt)
        mine = _ids([row], self.device, "PagePool.load")  # at hand for the way back, which allocates nothing
        self.fork(mine, [-1], [stored.length])
        Z.check(self.status(clear=True), "PagePool.load: no room")
        try:
            copy(flat, None, self.pages, self._held(row)[1])  # with a status of its own: waits, and raises
        except BaseException:  # whatever it was, the row is empty again
            self.free(mine)
            raise
