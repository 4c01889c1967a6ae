"""Pages of a K/V cache on the GPU: every page, reference, length and table equal to a pool
kept one page at a time on the host, and the calls that are refused."""
import random

import numpy as np
import pytest
import torch

import pages_util as U

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


def values(planes, pages, inner, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2 ** 31, 2 ** 31 - 1, (planes, pages) + inner, generator=g, dtype=torch.int64).to(torch.int32)


SHAPES = [(1, 2, (4,)), (3, 17, (1, 4)), (2, 40, (5, 3, 4)), (5, 9, (16, 8, 32)), (2, 33, (16, 8, 37 * 4)), (64, 6, (1, 20)),
          (1, 300, (7, 12)), (2, 8, (4096, 4)), (1, 5, (16389, 4))]


@pytest.mark.parametrize("planes,count,inner", SHAPES)
def test_copy_each_way(P, Z, planes, count, inner):
    src = values(planes, count, inner).cuda()
    perm = torch.randperm(count, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    n = max(1, count * 2 // 3)
    ids = perm[:n].cuda()
    guard = torch.full((planes, count + 2) + inner, 7, dtype=torch.int32, device="cuda")
    ws = P.copy_workspace()
    # gather, into the middle of a guarded tensor
    P.copy(src, ids, guard[:, 1:n + 1], None, ws=ws)
    assert torch.equal(guard[:, 1:n + 1], src[:, ids.long()])
    assert (guard[:, 0] == 7).all() and (guard[:, n + 1:] == 7).all()
    # scatter
    dst = values(planes, count, inner, 5).cuda()
    want = dst.clone()
    want[:, ids.long()] = guard[:, 1:n + 1]
    P.copy(guard[:, 1:n + 1], None, dst, ids, ws=ws)
    assert torch.equal(dst, want)
    # lists on both sides, some pairs skipped, a page read twice
    a, b = torch.randint(0, count, (n,), dtype=torch.int32), perm[:n].clone()
    a[::3] = -1
    if n > 1:
        b[1] = -5
    keep = (a >= 0) & (b >= 0)
    want[:, b[keep].long().cuda()] = src[:, a[keep].long().cuda()]
    P.copy(src, a.cuda(), dst, b.cuda(), ws=ws)
    assert torch.equal(dst, want)
    # within one pool
    half = count // 2
    if half:
        a, b = perm[:half].cuda(), perm[half:2 * half].cuda()
        want = src.clone()
        want[:, b.long()] = src[:, a.long()]
        P.copy(src, a, src, b, ws=ws)
        assert torch.equal(src, want)
    assert Z.status(ws) == Z.OK


def test_copy_strided_pools(P):
    big = values(6, 20, (8, 4)).cuda()
    ids = torch.tensor([7, 0, 3], dtype=torch.int32, device="cuda")
    assert torch.equal(P.copy(big[::2, 1:9], ids, torch.empty(3, 3, 8, 4, dtype=torch.int32, device="cuda"), None),
                       big[::2, 1:9][:, ids.long()])
    inner = big.transpose(0, 1)  # pages that hold all their planes: planes are the second dimension in memory
    out = torch.zeros(20, 6, 8, 4, dtype=torch.int32, device="cuda")
    P.copy(inner, None, out, None)
    assert torch.equal(out, inner.contiguous())


def test_copy_refused_on_the_device(P, Z):
    src = values(2, 12, (4, 4)).cuda()
    dst = values(2, 12, (4, 4), 3).cuda()
    for a, b, x, y in (([0, 1], [5, 5], src, dst), ([0, 1, 2], [3, 2, 5], src, src), ([4], [4], src, src),
                       ([0, 1], [3, 12], src, dst), ([12, 1], [3, 4], src, dst), ([0, 1, 2], [9, 10, 9], src, dst)):
        before = (x.clone(), y.clone())
        ws = P.copy_workspace()
        P.copy(x, a, y, b, ws=ws)
        assert Z.status(ws) == Z.ERR_INVALID_ARG
        assert torch.equal(x, before[0]) and torch.equal(y, before[1])
        P.copy(src, [1], dst, [2], ws=ws)  # a call after it works, and the first error stays
        assert Z.status(ws) == Z.ERR_INVALID_ARG and torch.equal(dst[:, 2], src[:, 1])
        with pytest.raises(Z.ZipnnError):
            P.copy(x, a, y, b)
    out = torch.zeros(2, 3, 4, 4, dtype=torch.int32, device="cuda")
    ws = P.copy_workspace()
    P.copy(src, [1, 99, 2], out, None, ws=ws)  # without a list of destinations the others are copied
    assert Z.status(ws) == Z.ERR_INVALID_ARG
    assert torch.equal(out[:, 0], src[:, 1]) and torch.equal(out[:, 2], src[:, 2]) and not out[:, 1].any()


def test_copy_more_pages_than_one_window(P, Z):
    """Page numbers past 2^18, where the check takes a second window."""
    n = (1 << 18) + 70
    src = torch.arange(n * 4, dtype=torch.int32, device="cuda").view(1, n, 4)
    dst = torch.zeros_like(src)
    ids = torch.tensor([n - 1, 5, (1 << 18) - 1, 1 << 18], dtype=torch.int32, device="cuda")
    to = torch.tensor([3, n - 2, 1 << 18, (1 << 18) - 1], dtype=torch.int32, device="cuda")
    P.copy(src, ids, dst, to)
    want = torch.zeros_like(src)
    want[:, to.long()] = src[:, ids.long()]
    assert torch.equal(dst, want)
    for a, b in (([1, 2], [n - 1, n - 1]), ([n - 1, 2], [4, n - 1])):
        with pytest.raises(Z.ZipnnError):
            P.copy(dst, a, dst, b)
    assert torch.equal(dst, want)


class Both:
    """A pool on the GPU and its books on the host, the same calls made on both."""

    def __init__(self, P, planes, pages, page_tokens, inner, seqs, slots, seed=0):
        v = values(planes, pages, inner, seed)
        self.pool = P.PagePool(v.cuda(), page_tokens, seqs, slots)
        self.books = U.empty(v.numpy().copy(), page_tokens, seqs, slots)

    def same(self):
        assert np.array_equal(self.pool.refs.cpu().numpy(), self.books.refs)
        assert np.array_equal(self.pool.lens.cpu().numpy(), self.books.lens)
        assert np.array_equal(self.pool.tables.cpu().numpy(), self.books.tables)
        assert np.array_equal(self.pool.pages.cpu().numpy(), self.books.pages)

    def fork(self, rows, parents, lens):
        ok = self.books.fork(rows, parents, lens)
        self.pool.fork(rows, parents, lens)
        assert (self.pool.status(clear=True) == 0) == ok
        self.same()
        return ok

    def free(self, rows, compact=False):
        self.books.free(rows)
        live = self.books.compact() if compact else None
        self.pool.free(rows, compact=compact)
        assert self.pool.status() == 0
        if compact:
            assert self.pool.live.item() == live
        self.same()


@pytest.mark.parametrize("page_tokens", [1, 7, 16])
def test_fork_at_every_kind_of_length(P, page_tokens):
    pt = page_tokens
    b = Both(P, 2, 120, pt, (pt, 4), 24, 8)
    assert b.fork([3], [-1], [5 * pt])
    assert b.fork([0], [-1], [0])                              # an empty sequence
    assert b.fork([5, 1], [-1, -1], [1, 3 * pt + 1])
    row = 6
    for n in sorted({0, 1, pt - 1, pt, pt + 1, 2 * pt - 1, 3 * pt, 5 * pt, 5 * pt + 1, 8 * pt} - {-1}):  # of a whole parent, past it
        assert b.fork([row], [3], [n])
        row += 1
    assert b.fork([row, row + 1, row + 2], [1, 1, 5], [3 * pt + 1, 3 * pt, pt + 2])  # several at once, of a ragged one
    assert b.fork([1, 5, row + 3], [1, 5, 1], [3 * pt + 1, 2 * pt + 1, 3 * pt + 1])    # staying, growing, and forked meanwhile
    assert b.fork([row + 4, row + 5], [0, row + 4], [pt + 1, 2])                       # empty parents give nothing
    b.free([3, 1], compact=True)
    assert b.fork([1, 3], [5, -1], [2, pt])


def test_fork_refused(P, Z):
    b = Both(P, 1, 10, 4, (4, 4), 5, 6)
    assert b.fork([0, 1], [-1, -1], [9, 4])
    for rows, parents, lens in (([2, 2], [-1, -1], [4, 4]), ([5], [-1], [4]), ([-1], [-1], [4]), ([2], [5], [4]), ([2], [-2], [4]),
                                ([2], [-1], [25]), ([2], [-1], [-1]), ([1], [-1], [4]), ([1], [0], [4]), ([0], [0], [8]),
                                ([2, 3], [0, 9], [4, 4])):
        assert not b.fork(rows, parents, lens)
    pool = b.pool
    pool.fork([2, 3], [-1, -1], [16, 9])  # 7 fresh pages of the 6 left
    assert pool.status(clear=True) == Z.ERR_OUT_TOO_SMALL
    b.same()
    assert b.fork([2, 3], [-1, -1], [16, 8])  # all of them
    assert not b.fork([4], [-1], [1])
    assert b.fork([4], [2], [16])             # shared pages cost none
    for bad in (lambda: pool.fork([0], [0], [0, 1]), lambda: pool.fork(torch.zeros(1, device="cuda"), [0], [1]),
                lambda: pool.fork([0] * 6, [0] * 6, [0] * 6), lambda: pool.free(torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(Z.ZipnnError):
            bad()


def test_free_twice_empty_and_out_of_range(P, Z):
    b = Both(P, 1, 12, 4, (4, 4), 4, 6)
    b.fork([0, 1], [-1, -1], [9, 5])
    b.fork([2], [0], [8])
    b.pool.free([0, 0, 3, 0])
    b.books.free([0])
    assert b.pool.status() == Z.OK
    b.same()
    b.pool.free([4, 1, -1])
    b.books.free([1])
    assert b.pool.status(clear=True) == Z.ERR_INVALID_ARG
    b.same()
    b.pool.free([])
    b.same()


def test_damaged_books_are_reported(P, Z):
    b = Both(P, 1, 12, 4, (4, 4), 4, 6)
    b.fork([0], [-1], [20])
    t = b.pool.tables
    t[0, 1], t[0, 2] = 99, -7
    b.pool.fork([1], [0], [18])
    assert b.pool.status(clear=True) == Z.ERR_CORRUPT
    b.pool.compact()
    t[0, 0] = 11  # a page without references
    b.pool.free([0])
    assert b.pool.status(clear=True) == Z.ERR_CORRUPT
    assert (b.pool.refs >= 0).all()
    b.pool.lens[2] = 1 << 30
    b.pool.free([2])
    assert b.pool.status(clear=True) == Z.ERR_CORRUPT
    b.pool.lens[2] = -3
    b.pool.fork([3], [2], [4])
    assert b.pool.status(clear=True) == Z.ERR_INVALID_ARG
    b.pool.lens[2] = 0
    b.pool.refs[:] = 1
    b.pool.refs[5] = 0
    t[3, 0] = 11
    b.pool.free([], compact=True)  # 11 moves to 5; what the other tables name is in range
    assert b.pool.tables[3, 0].item() == 5


@pytest.mark.parametrize("seed", range(6))
def test_a_served_cache_step_by_step(P, seed):
    """Random forks, growth, frees and compactions, everything compared after each."""
    rng = random.Random(seed)
    pt = rng.choice((1, 3, 16))
    seqs, slots = rng.choice(((5, 9), (40, 30), (1100, 4)))
    pages = rng.choice((16, 200, 1500))
    b = Both(P, rng.choice((1, 3)), pages, pt, (pt, 4), seqs, slots, seed)
    refused = 0
    for _ in range(25):
        lens = b.books.lens
        filled, empty = [r for r in range(seqs) if lens[r]], [r for r in range(seqs) if not lens[r]]
        if rng.random() < 0.6:
            n = rng.choice((1, 2, 5, seqs))
            rows, parents, want = [], [], []
            for r in rng.sample(range(seqs), min(n, seqs)):
                if lens[r]:
                    rows.append(r), parents.append(r), want.append(min(slots * pt, int(lens[r]) + rng.randint(0, pt)))
                else:
                    p = rng.choice(filled) if filled and rng.random() < 0.6 else -1
                    rows.append(r), parents.append(p), want.append(rng.randint(0, slots * pt // 2 + 1))
            refused += not b.fork(rows, parents, want)
        elif filled:
            b.free(rng.sample(filled, rng.randint(1, len(filled))), compact=rng.random() < 0.5)
        else:
            b.free([], compact=True)
    assert refused < 25


@pytest.mark.parametrize("pages", [1, 31, 32, 33, 1023, 1025, 5000, 140_000])
def test_books_of_every_size(P, pages):
    """Scans over few and many pages: every other sequence freed, the pool closed up, and the
    room found again."""
    seqs = min(pages, 37)
    slots = -(-pages // seqs)
    b = Both(P, 1, pages, 1, (1, 4), seqs, slots)
    per = pages // seqs
    assert b.fork(list(range(seqs)), [-1] * seqs, [per] * seqs)
    b.free(list(range(0, seqs, 2)))
    b.free([], compact=True)
    b.free([seqs - 1], compact=True)
    assert b.fork([0], [-1], [per])


def test_the_longest_lists(P):
    """2^18 rows, forked, freed and closed up in one call each, and 200,000 pairs copied."""
    seqs = 1 << 18
    b = Both(P, 1, 300_000, 1, (1, 4), seqs, 2)
    rng = np.random.RandomState(1)
    assert b.fork(rng.permutation(seqs).tolist(), [-1] * seqs, [1] * seqs)
    assert not b.fork([0, seqs], [0, -1], [2, 1])
    b.free(rng.permutation(seqs)[: seqs // 2].tolist(), compact=True)
    filled = np.nonzero(b.books.lens)[0]
    assert b.fork(filled[:1000].tolist(), filled[:1000].tolist(), [2] * 1000)
    perm = torch.from_numpy(rng.permutation(300_000).astype(np.int32)).cuda()
    src = b.pool.pages.clone()
    out = P.copy(src, perm[:200_000], torch.zeros_like(src), perm[100_000:])
    assert torch.equal(out[:, perm[100_000:].long()], src[:, perm[:200_000].long()])


def test_two_pools_two_streams_and_graphs(P, Z):
    pools = [Both(P, 2, 64, 4, (4, 8), 8, 10, s) for s in range(2)]
    for b in pools:
        b.fork([0, 1], [-1, -1], [30, 17])
    rows, parents, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([2, 3], [0, 1], [29, 17]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pools]
    graphs = []
    for b, s in zip(pools, streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b.pool.fork(rows, parents, lens)
            b.pool.free(rows, compact=True)
            b.pool.fork(rows, parents, lens)
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b in pools:
            b.books.fork([2, 3], [0, 1], [29, 17])
            b.books.free([2, 3])
            b.books.compact()
            b.books.fork([2, 3], [0, 1], [29, 17])
            b.same()
            assert b.pool.status() == Z.OK
            b.pool.free([2, 3])
            b.books.free([2, 3])
    b = pools[0]
    b.pool.fork(rows, parents, lens, stream=streams[0])
    streams[0].synchronize()
    b.books.fork([2, 3], [0, 1], [29, 17])
    b.same()


def test_copies_captured_and_replayed(P, Z):
    """A checked copy in a graph: the lists are read at each replay, and a bad one copies nothing
    and is seen in the status."""
    src, dst = values(3, 20, (8, 4)).cuda(), torch.zeros(3, 20, 8, 4, dtype=torch.int32, device="cuda")
    a, b = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([1, 2, 3], [4, 5, 6]))
    ws = P.copy_workspace()
    P.copy(src, a, dst, b, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.copy(src, a, dst, b, ws=ws)
        P.copy(dst, b, dst, a, ws=ws)
    for x, y in (([1, 2, 3], [4, 5, 6]), ([7, 7, 19], [0, 9, 18]), ([0, 1, 2], [3, 3, 4]), ([5, 6, 8], [11, 12, 13])):
        a.copy_(torch.tensor(x, dtype=torch.int32))
        b.copy_(torch.tensor(y, dtype=torch.int32))
        want = dst.clone()
        if len(set(y)) == 3:  # a page named twice is refused as a destination, not as a source
            want[:, y] = src[:, x]
        if len(set(x)) == 3:
            want[:, x] = want[:, y].clone()
        g.replay()
        assert torch.equal(dst, want)
    assert Z.status(ws) == Z.ERR_INVALID_ARG


def test_offsets_past_32_bits(P):
    """A pool of 9.7 GB: its last pages, gathered, moved and scattered."""
    kv = torch.empty(3, 100_000, 16, 1024, dtype=torch.bfloat16, device="cuda")
    kv[:, -5:] = torch.randn(3, 5, 16, 1024, device="cuda").to(torch.bfloat16)
    want = kv[:, -5:].clone()
    kv[:, :5] = 0
    ids = torch.arange(99_995, 100_000, dtype=torch.int32, device="cuda")
    to = torch.arange(5, dtype=torch.int32, device="cuda")
    got = P.copy(kv, ids, torch.empty_like(want), None)
    assert torch.equal(got, want)
    P.copy(kv, ids, kv, to)
    assert torch.equal(kv[:, :5], want)
    kv[:, -5:] = 0
    P.copy(got, None, kv, ids)
    assert torch.equal(kv[:, -5:], want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp8", "fp32", "uint8", "int32"])
def test_store_and_load_through_the_codec(P, Z, dtype):
    """A sequence leaves the cache compressed, its pages go to others, and it comes back."""
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn, "fp32": torch.float32, "uint8": torch.uint8,
          "int32": torch.int32}[dtype]
    g = torch.Generator().manual_seed(2)
    kv = (torch.randn(4, 50, 16, 2, 64, generator=g) * 20).to(dt).cuda()
    pool = P.PagePool(kv, 16, 6, 20)
    pool.fork([0, 1], [-1, -1], [300, 77])
    pool.fork([2], [0], [200])
    ids = pool.tables[2, :13].long()
    before = kv.view(torch.uint8)[:, ids].clone()
    stored = pool.store(2, chunk_bytes=65536)
    assert stored.length == 200
    pool.free([0, 2], compact=True)
    assert pool.live.item() == 5
    pool.fork([3], [-1], [300])
    kv.view(torch.uint8)[:, pool.tables[3, :19].long()] = 0
    pool.load(stored, 2)
    assert pool.lens.tolist() == [0, 77, 200, 300, 0, 0]
    assert torch.equal(kv.view(torch.uint8)[:, pool.tables[2, :13].long()], before)
    with pytest.raises(Z.ZipnnError):
        pool.load(stored, 2)      # not empty
    with pytest.raises(Z.ZipnnError):
        pool.store(5)             # nothing there
    pool.fork([0], [-1], [13 * 16])
    with pytest.raises(Z.ZipnnError):
        pool.load(stored, 4)      # no room
    assert pool.status() == Z.OK
    pool.free([0, 3])
    other = P.PagePool(kv.view(4, 100, 8, 2, 64), 8, 6, 40)
    with pytest.raises(Z.ZipnnError):
        other.load(stored, 0)     # pages of another shape
    bad = P.StoredPages(stored.container.clone(), stored.length, stored.chunk_bytes, stored.pages)
    bad.container[:4] = 0
    books = pool.meta.clone()
    with pytest.raises(Z.ZipnnError):
        pool.load(bad, 4)         # a damaged container: the row is empty again
    assert torch.equal(pool.meta, books) and pool.status() == Z.OK
    wide = P.PagePool(torch.zeros(1, 2, 4, dtype=torch.int64, device="cuda"), 4, 2, 2)
    wide.fork([0], [-1], [4])
    with pytest.raises(Z.ZipnnError):
        wide.store(0)             # no type of the codec


def test_a_cache_in_four_bits_through_the_codec(P):
    """The operators together: pages gathered, quantised, compressed and given back; later
    decompressed, read back and scattered into the pages of a new row."""
    from lossless_float_weight_b200 import mx
    g = torch.Generator().manual_seed(6)
    kv = torch.randn(4, 40, 16, 2, 64, generator=g).to(torch.bfloat16).cuda()
    pool = P.PagePool(kv, 16, 4, 16)
    pool.fork([0], [-1], [170])
    flat = pool.gather(pool.tables[0, :11])
    for fmt in ("mxfp4", "nvfp4"):
        q = mx.quantize(flat, fmt)
        stored = mx.compress(q)
        pool.free([0], compact=True)
        pool.fork([1], [-1], [170])
        back = mx.dequantize(mx.decompress(stored))
        assert torch.equal(back, mx.dequantize(q))
        pool.scatter(back, pool.tables[1, :11])
        assert torch.equal(kv[:, pool.tables[1, :11].long()], back)
        pool.free([1])
        assert pool.status() == 0


def test_pool_refusals(P, Z):
    kv = torch.zeros(2, 8, 16, 8, dtype=torch.bfloat16, device="cuda")
    meta = torch.zeros(8 + 4 * 5, dtype=torch.int32, device="cuda")
    P.PagePool(kv, 16, 4, meta=meta)
    for bad in (lambda: P.PagePool(kv, 0, 4, 4), lambda: P.PagePool(kv, 16, 0, 4), lambda: P.PagePool(kv, 16, 4),
                lambda: P.PagePool(kv, 16, 4, 5, meta=meta), lambda: P.PagePool(kv, 16, 4, meta=meta[:-1]),
                lambda: P.PagePool(kv, 16, 4, meta=meta.long()), lambda: P.PagePool(kv.transpose(2, 3), 16, 4, 4),
                lambda: P.copy(kv, [0], kv[..., :4], [1]), lambda: P.copy(kv, [0], kv[:1], [1]),
                lambda: P.copy(kv, [0, 1], kv, [2]), lambda: P.copy(kv, [0], kv, [1], count=2),
                lambda: P.copy(kv[:, :4], [0], kv, [5]), lambda: P.copy(kv[:1].expand(2, 8, 16, 8), [0], kv.clone(), [1]),
                lambda: P.copy(kv[..., :3], [0], kv[..., :3].contiguous(), [1])):
        with pytest.raises(Z.ZipnnError):
            bad()
