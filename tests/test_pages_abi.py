"""Pages of a K/V cache: workspace sizes and the refusals that need no device (CPU)."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # an aligned address, never dereferenced: every case fails before a launch


@pytest.fixture(scope="module")
def Z():
    from lossless_float_weight_b200 import build
    build.build()
    from lossless_float_weight_b200 import zipnn
    return zipnn


def pool(Z, **kw):
    d = dict(base=FAKE, plane_stride=8192, page_stride=1024, planes=4, pages=8)
    d.update(kw)
    return Z.PagePoolDesc(**d)


BAD_POOLS = (dict(base=None), dict(base=FAKE + 8), dict(planes=0), dict(pages=0), dict(page_stride=1000),
             dict(plane_stride=8200), dict(page_stride=512), dict(plane_stride=7168), dict(pages=9),
             dict(planes=1, page_stride=1 << 47), dict(planes=1, page_stride=1 << 45, pages=64), dict(pages=1 << 31))


def test_copy_refusals(Z):
    def copy(src=None, dst=None, si=FAKE, di=FAKE, count=3, nbytes=1024, ws=FAKE, wb=256):
        a = src or pool(Z)
        b = dst or pool(Z, base=FAKE + (1 << 20))
        return Z.zipnn_pages_copy(ctypes.byref(a), si, ctypes.byref(b), di, count, nbytes, ws, wb, None)

    for kw in BAD_POOLS:
        assert copy(src=pool(Z, **kw)) == Z.ERR_INVALID_ARG, kw
    for kw in (dict(nbytes=0), dict(nbytes=1000), dict(si=FAKE + 2), dict(di=FAKE + 1), dict(si=None, count=9),
               dict(di=None, count=9), dict(ws=None), dict(ws=FAKE + 4), dict(dst=pool(Z, base=FAKE + (1 << 20), planes=3)),
               dict(dst=pool(Z, base=FAKE + 4096)), dict(dst=pool(Z, pages=7))):  # overlapping, not the same pool
        assert copy(**kw) == Z.ERR_INVALID_ARG, kw
    assert copy(wb=255) == Z.ERR_OUT_TOO_SMALL
    assert Z.zipnn_pages_copy(None, None, None, None, 1, 1024, FAKE, 256, None) == Z.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        # pages that hold all their planes are a layout too
        inner = pool(Z, plane_stride=1024, page_stride=4096)
        assert copy() == Z.ERR_UNSUPPORTED and copy(src=inner) == Z.ERR_UNSUPPORTED
        assert copy(src=pool(Z, planes=1), dst=pool(Z, planes=1, base=FAKE + 8192)) == Z.ERR_UNSUPPORTED


def test_table_refusals(Z):
    wb = Z.zipnn_pages_workspace_bytes(4, 8)
    assert wb >= 256 and Z.zipnn_pages_workspace_bytes(5, 2 ** 20) > wb

    def table(**kw):
        d = dict(refs=FAKE, lens=FAKE, tables=FAKE, seqs=4, slots=8, page_tokens=16)
        d.update(kw)
        return Z.PageTableDesc(**d)

    def fork(p=None, t=None, rows=FAKE, parents=FAKE, lens=FAKE, count=2, ws=FAKE, w=wb):
        return Z.zipnn_pages_fork(ctypes.byref(p or pool(Z)), 1024, ctypes.byref(t or table()), rows, parents, lens, count, ws, w, None)

    def free(p=None, t=None, rows=FAKE, count=2, ws=FAKE, w=wb):
        return Z.zipnn_pages_free(ctypes.byref(p or pool(Z)), 1024, ctypes.byref(t or table()), rows, count, 1, ws, w, None)

    for call in (fork, free):
        for kw in BAD_POOLS:
            assert call(p=pool(Z, **kw)) == Z.ERR_INVALID_ARG, kw
        for kw in (dict(refs=None), dict(lens=FAKE + 1), dict(tables=None), dict(seqs=0), dict(seqs=(1 << 18) + 1), dict(slots=0),
                   dict(page_tokens=0), dict(seqs=1 << 18, slots=1 << 13)):
            assert call(t=table(**kw)) == Z.ERR_INVALID_ARG, kw
        assert call(ws=None) == Z.ERR_INVALID_ARG and call(ws=FAKE + 8) == Z.ERR_INVALID_ARG and call(rows=None) == Z.ERR_INVALID_ARG
        assert call(w=wb - 1) == Z.ERR_OUT_TOO_SMALL
        if not torch.cuda.is_available():
            assert call() == Z.ERR_UNSUPPORTED
    for kw in (dict(parents=None), dict(lens=FAKE + 2), dict(count=5)):
        assert fork(**kw) == Z.ERR_INVALID_ARG


def test_python_refusals(Z):
    from lossless_float_weight_b200 import pages
    kv = torch.zeros(2, 4, 16, 8)
    for call in (lambda: pages.PagePool(kv, 16, 4, 4), lambda: pages.copy(kv, [0], kv, [1]), lambda: pages.copy(kv[0], [0], kv, [1])):
        with pytest.raises(Z.ZipnnError):
            call()
