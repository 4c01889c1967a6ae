"""Pages of a K/V cache: stores of rows that are damaged, loads that fail, lists of no pages, and
what autograd is told of pages that change."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_float_weight_b200 import pages
    return pages


@pytest.fixture(scope="module")
def Z():
    from lossless_float_weight_b200 import zipnn
    return zipnn


def cache(P, planes=2, pages=20, seed=0):
    kv = torch.randn(planes, pages, 16, 2, 64, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    return P.PagePool(kv, 16, 6, 8)


@pytest.mark.parametrize("number", [99, 20, -7, -1])
def test_a_damaged_row_is_not_stored(P, Z, number):
    """A number outside the pool in the row's table, in the row itself and in a fork of it."""
    pool = cache(P)
    pool.fork([0, 1], [-1, -1], [70, 33])
    whole = pool.store(1)
    pool.tables[0, 2] = number
    pool.fork([2], [0], [64])
    assert pool.status(clear=True) == Z.ERR_CORRUPT
    for row in (0, 2):
        with pytest.raises(Z.ZipnnError) as e:
            pool.store(row)
        assert e.value.status == Z.ERR_CORRUPT
    assert pool.status() == Z.OK and torch.equal(pool.store(1).container, whole.container)


@pytest.mark.parametrize("length", [129, 1 << 30, -5])
def test_a_row_of_an_impossible_length_is_not_stored(P, Z, length):
    pool = cache(P)
    pool.fork([0], [-1], [128])
    pool.lens[0] = length
    with pytest.raises(Z.ZipnnError) as e:
        pool.store(0)
    assert e.value.status == Z.ERR_CORRUPT


def test_a_store_beside_an_earlier_error(P, Z):
    """An error that was not yet taken stays for its caller, and says nothing of the store."""
    pool = cache(P)
    pool.fork([0], [-1], [70])
    pool.fork([0], [-1], [70])  # refused: the row is filled
    stored = pool.store(0)
    assert pool.status(clear=True) == Z.ERR_INVALID_ARG
    want = pool.gather(pool.tables[0, :5]).clone()
    pool.load(stored, 3)
    assert torch.equal(pool.gather(pool.tables[3, :5]), want)


@pytest.mark.parametrize("where", ["decompress", "scatter"])
@pytest.mark.parametrize("error", [torch.cuda.OutOfMemoryError, KeyboardInterrupt, RuntimeError])
def test_a_load_that_fails_leaves_the_books_as_they_were(P, Z, monkeypatch, where, error):
    pool = cache(P)
    pool.fork([0, 1], [-1, -1], [70, 33])
    stored = pool.store(0)
    pool.free([0])
    books = pool.meta.clone()

    def fail(*a, **k):
        raise error("out of memory")

    with monkeypatch.context() as m:
        if where == "decompress":
            m.setattr(Z, "decompress", fail)
        else:
            m.setattr(P, "copy", fail)
        with pytest.raises(error):
            pool.load(stored, 2)
    assert torch.equal(pool.meta, books) and pool.status() == Z.OK
    pool.load(stored, 2)
    assert pool.lens.tolist() == [0, 33, 70, 0, 0, 0]


def test_a_load_that_fails_needs_no_memory_to_undo(P, Z, monkeypatch):
    """As on a device that the cache fills: after the failure nothing can be allocated."""
    pool = cache(P)
    pool.fork([0, 1], [-1, -1], [70, 33])
    stored = pool.store(0)
    pool.free([0])
    books = pool.meta.clone()
    full = []

    def no_memory(*a, **k):
        full.append(1)
        raise torch.cuda.OutOfMemoryError("out of memory")

    ids = P._ids

    def allocating(v, device, what):
        if full and not isinstance(v, torch.Tensor):
            raise torch.cuda.OutOfMemoryError("out of memory")
        return ids(v, device, what)

    with monkeypatch.context() as m:
        m.setattr(P, "copy", no_memory)
        m.setattr(P, "_ids", allocating)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            pool.load(stored, 2)
    assert torch.equal(pool.meta, books) and pool.status() == Z.OK


def test_a_stored_sequence_on_another_device_is_refused(P, Z):
    pool = cache(P)
    pool.fork([0], [-1], [70])
    stored = pool.store(0)
    books = pool.meta.clone()
    away = P.StoredPages(stored.container.cpu(), stored.length, stored.chunk_bytes, stored.pages)
    with pytest.raises(Z.ZipnnError):
        pool.load(away, 2)
    assert torch.equal(pool.meta, books)


def test_lists_of_no_pages(P, Z):
    pool = cache(P)
    pool.fork([0], [-1], [0])
    none = pool.gather(pool.tables[0, :0])
    assert none.shape == (2, 0, 16, 2, 64) and none.dtype == torch.bfloat16
    assert pool.gather([]).shape == none.shape
    before = pool.pages.clone()
    pool.scatter(none, [])
    pool.scatter(none, torch.empty(0, dtype=torch.int32, device="cuda"))
    P.copy(none, None, pool.pages, None)
    P.copy(pool.pages, [], none, [])
    assert torch.equal(pool.pages, before) and pool.status() == Z.OK
    for bad in (lambda: P.copy(none[..., :32], None, pool.pages, None), lambda: pool.scatter(none[:1], [])):
        with pytest.raises(Z.ZipnnError):
            bad()


def test_pages_that_ask_for_gradients_are_refused(P, Z):
    import torch.autograd.forward_ad as fw
    kv = torch.zeros(2, 8, 16, 8, device="cuda")
    leaf = kv.clone().requires_grad_()
    pool = P.PagePool(leaf, 16, 4, 4)
    calls = (lambda: P.copy(leaf, [0], kv, [1]), lambda: P.copy(kv, [0], leaf, [1]), lambda: pool.fork([0], [-1], [20]),
             lambda: pool.free([0], compact=True), lambda: pool.gather([0]))
    for call in calls:
        with pytest.raises(Z.ZipnnError):
            call()
    with torch.no_grad():
        for call in calls:
            call()
    assert pool.status() == Z.OK
    with fw.dual_level():
        with pytest.raises(Z.ZipnnError):
            P.copy(fw.make_dual(kv, torch.ones_like(kv)), [0], kv.clone(), [1])


def test_pages_saved_for_backward_are_seen_to_change(P):
    def fork(pool):
        pool.fork([1], [0], [20])

    def scatter(pool):
        pool.scatter(torch.zeros(2, 1, 16, 2, 64, dtype=torch.bfloat16, device="cuda"), [3])

    def compact(pool):
        pool.free([], compact=True)

    def copy(pool):
        P.copy(pool.pages, [0], pool.pages, [5])

    for change in (fork, scatter, compact, copy):
        pool = cache(P)
        pool.fork([0], [-1], [40])
        w = torch.ones_like(pool.pages, requires_grad=True)
        y = (w * pool.pages).sum()  # the pages are saved
        change(pool)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    pool = cache(P)
    pool.fork([0], [-1], [40])
    w = torch.ones_like(pool.pages, requires_grad=True)
    y = (w * pool.pages).sum()
    pool.free([0])  # changes no page
    y.backward()
    assert torch.equal(w.grad, pool.pages)
    pool.fork([0], [-1], [40])
    w = torch.ones(20, requires_grad=True, device="cuda")
    y = w[pool.refs].sum()  # the references are saved as indexes
    pool.free([0])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_a_workspace_elsewhere_is_refused(P, Z):
    src, dst = torch.ones(2, 4, 16, 8, device="cuda"), torch.zeros(2, 4, 16, 8, device="cuda")
    for ws in (torch.zeros(256, dtype=torch.uint8), torch.zeros(255, dtype=torch.uint8, device="cuda"),
               torch.zeros(264, dtype=torch.uint8, device="cuda")[8:], torch.zeros(256, dtype=torch.uint8, device="meta")):
        with pytest.raises(Z.ZipnnError):
            P.copy(src, [0], dst, [1], ws=ws)
    assert not dst.any()


@pytest.mark.parametrize("tokens", [-1, 1 << 31, (1 << 32) + 16])
def test_page_tokens_out_of_range_are_refused(P, Z, tokens):
    with pytest.raises(Z.ZipnnError):
        P.PagePool(torch.zeros(2, 4, 16, 8, device="cuda"), tokens, 4, 4)
    pool = P.PagePool(torch.zeros(2, 4, 16, 8, device="cuda"), (1 << 31) - 1, 4, 4)
    pool.fork([0], [-1], [(1 << 31) - 1])
    assert pool.status() == Z.OK and pool.tables[0].tolist() == [0, -1, -1, -1]
