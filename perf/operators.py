"""The low-precision operators beside the codec, as calls of a user's program.

Three groups: tensors held as microscaled 4-bit values (their quantisation, what they read
back as, and the product of two of them); the copying of K/V-cache pages; and the pages of
sequences (sharing them when a sequence forks, giving them back, closing the gaps).

``own`` False computes everything in elementary torch operations; True makes the calls of
the library. Sizes come from the codec's own workloads (hidden 4096, MLP 11008, vocabulary
32000; a K/V cache of 32 layers x (K, V), 8 heads, 4096 positions, 128 dims) and from
ragged ones around them.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden state, quantised in front of a product (a decode step)
        dict(name="quantize_token_mxfp4", op="quantize", format="mxfp4", dtype="bf16", rows=1, cols=4096),
        # the K of one layer of one sequence leaving the cache, rows of one head each
        dict(name="quantize_kv_fp16_mxfp4", op="quantize", format="mxfp4", dtype="fp16", rows=32760, cols=128),
        # an MLP weight of the 7B shape, quantised when it is loaded (its own global scale)
        dict(name="quantize_mlp_nvfp4", op="quantize", format="nvfp4", dtype="bf16", rows=11008, cols=4096),
        # a decode step: one token through the MLP's wide matrix
        dict(name="matmul_token_mxfp4", op="matmul", format="mxfp4", out="bf16", m=1, n=11008, k=4096),
        # a small ragged batch through an attention matrix, FP32 out
        dict(name="matmul_batch_nvfp4", op="matmul", format="nvfp4", out="fp32", m=77, n=4096, k=4080),
        # a prompt of 4096 tokens through the MLP's wide matrix
        dict(name="matmul_prompt_mxfp4", op="matmul", format="mxfp4", out="bf16", m=4096, n=11008, k=4096),
        # the pages of one short sequence collected for the codec
        dict(name="copy_gather_small", op="copy", way="gather", dtype="bf16", planes=64, pages=256, n=5, tokens=16,
             heads=8, dim=128),
        # a cache of many sequences coming back into its pages
        dict(name="copy_scatter_large", op="copy", way="scatter", dtype="bf16", planes=64, pages=768, n=640,
             tokens=16, heads=8, dim=128),
        # one sequence forked once (a second answer to a prompt that ends inside a page)
        dict(name="fork_one", op="fork", dtype="bf16", planes=64, pages=512, tokens=16, heads=8, dim=128, seqs=8,
             n=1, max_len=500),
        # a batch step: forks, new sequences and longer ones in one call, 16-token FP8 pages
        dict(name="fork_batch", op="fork", dtype="fp8", planes=64, pages=2048, tokens=16, heads=8, dim=128,
             seqs=64, n=48, max_len=900),
        # two finished sequences give their pages back
        dict(name="free_two", op="free", dtype="bf16", planes=2, pages=4096, tokens=16, heads=8, dim=128, seqs=64,
             n=2, max_len=1000, compact=False),
        # half of the sequences gone, and the pool closed up
        dict(name="free_compact", op="free", dtype="bf16", planes=64, pages=1024, tokens=16, heads=8, dim=128,
             seqs=32, n=16, max_len=500, compact=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "quantize", "matmul", "matmul", "matmul", "copy", "fork", "free"))
    if op == "quantize":
        cols = _log(rng, 1, 11008)
        rows = _log(rng, 1, min(32768, 45088768 // cols))
        return dict(op=op, format=rng.choice(("mxfp4", "nvfp4")), dtype=rng.choice(("bf16", "fp16", "fp32")),
                    rows=rows, cols=cols)
    if op == "matmul":
        m, n, k = _log(rng, 1, 4096), _log(rng, 1, 32000), _log(rng, 1, 11008)
        while m * n * k > 4096 * 4096 * 11008:
            m, n, k = (m + 1) // 2, (2 * n + 2) // 3, k
        return dict(op=op, format=rng.choice(("mxfp4", "nvfp4")), out=rng.choice(("bf16", "fp16", "fp32")),
                    m=m, n=n, k=k)
    shape = dict(dtype=rng.choice(("bf16", "fp8", "fp16")), tokens=rng.choice((1, 8, 16, 32, 64)),
                 heads=rng.choice((1, 2, 4, 8)), dim=rng.choice((64, 128)))
    page = _SIZE[shape["dtype"]] * shape["tokens"] * shape["heads"] * shape["dim"]
    planes = _log(rng, 1, 64)
    most = max(2, min(8192, (1 << 31) // (page * planes)))
    if op == "copy":
        pages = _log(rng, 2, min(most, 2048))
        return dict(op=op, way=rng.choice(("gather", "scatter", "move")), planes=planes, pages=pages,
                    n=_log(rng, 1, max(1, pages // 2)), **shape)
    seqs = _log(rng, 2, 128)
    pages = _log(rng, min(most, 2 * seqs), most)
    per_seq = max(1, pages // (2 * seqs))
    case = dict(op=op, planes=planes, pages=pages, seqs=seqs, n=max(1, int(seqs * rng.uniform(0.01, 0.75))),
                max_len=max(1, int(per_seq * shape["tokens"] * rng.uniform(0.5, 1.0))), **shape)
    if op == "free":
        case["compact"] = rng.random() < 0.7
    return case


# ------------------------------------------------------- microscaled tensors, plain form

def _tiles(scales):
    """Row-major block scales (rows, blocks) in the order the products read them: 128 rows x
    4 blocks make a tile of 512 bytes, row r at 16 (r % 32) + 4 (r // 32 % 4)."""
    r, b = scales.shape
    rt, bt = -(-r // 128), -(-b // 4)
    s = torch.nn.functional.pad(scales.view(torch.uint8), (0, bt * 4 - b, 0, rt * 128 - r))
    return s.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(-1).view(scales.dtype)


def _untile(tiles, r, b):
    rt, bt = -(-r // 128), -(-b // 4)
    s = tiles.view(torch.uint8).view(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)
    return s[:r, :b].contiguous().view(tiles.dtype)


def _round_e2m1(a):
    """Magnitudes to the E2M1 grid, ties to the even code, saturating at 6."""
    a = a.clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step) * step


def _pow2(e):
    """2^e in 64 bits, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _plain_quantize(x, fmt):
    """(values in units of the scales (rows, blocks, block), scales (rows, blocks), global scale)."""
    rows, cols = x.shape
    blk = _BLOCK[fmt]
    xd = torch.nn.functional.pad(x.double(), (0, -cols % blk)).view(rows, -1, blk)
    amax = xd.abs().amax(-1)
    if fmt == "mxfp4":
        # floor(log2(amax)) - 2, kept in the range of E8M0
        _, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 3, -127).clamp(-127, 127)
        sc, g = _pow2(e), None
        s8 = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        inv = 1 / sc
    else:
        g = (amax.max() / 2688).float()
        g = torch.where(g > 0, g, torch.ones_like(g))
        gd = g.double()
        want = (amax / (6 * gd)).clamp(max=448.0)
        # to E4M3, ties to even: steps of 2^(e-3), 2^-9 below 2^-6
        _, e = torch.frexp(want)
        step = _pow2(e.clamp(min=-5) - 4)
        sv = torch.round(want / step) * step
        s8 = sv.float().to(torch.float8_e4m3fn)
        sc = sv * gd
        inv = torch.where(sv > 0, 1 / sc, torch.zeros_like(sc))
    # a quotient by 1 / scale may round across a border: divide
    q = torch.where(inv[..., None] > 0, xd.abs() / torch.where(inv > 0, sc, torch.ones_like(sc))[..., None], 0.0)
    q = torch.copysign(_round_e2m1(q), xd)
    return q, sc, s8, g


def _pack(q, rows):
    """E2M1 values (rows, blocks, block) as bytes, the first value of a pair in the low nibble,
    rows padded to whole 32 values."""
    grid = torch.tensor(_E2M1, device=q.device, dtype=q.dtype)
    code = torch.searchsorted(grid, q.abs().reshape(rows, -1).contiguous())
    code = code | (torch.signbit(q.reshape(rows, -1)).to(code.dtype) << 3)
    code = torch.nn.functional.pad(code, (0, -code.shape[1] % 32))
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)


def _values32(codes, tiles, shape, fmt, g):
    """FP32 values of a packed tensor."""
    rows, cols = shape
    blk = _BLOCK[fmt]
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    c = codes.to(torch.int32)
    v = torch.stack((lut[c & 15], lut[c >> 4]), -1).reshape(rows, -1)
    s = _untile(tiles, rows, -(-cols // blk)).float()
    s = s if g is None else s * g
    v = v[:, : s.shape[1] * blk].reshape(rows, -1, blk) * s[..., None]
    return v.reshape(rows, -1)[:, :cols]


# --------------------------------------------------------------------------- preparation

def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed & 0x7FFFFFFF)


def _rows(g, rows, cols):
    """Normal values whose scale differs from row to row by a factor of 16, as weights of
    different channels have, and a few values far out, as activations have."""
    scale = torch.exp((torch.rand(rows, 1, generator=g, device="cuda") - 0.5) * math.log(16.0))
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    far = torch.rand(rows, cols, generator=g, device="cuda") < 0.002
    return torch.where(far, x * 20, x)


def _packed(g, rows, cols, fmt):
    q, _, s8, gs = _plain_quantize(_rows(g, rows, cols).to(torch.bfloat16), fmt)
    return dict(codes=_pack(q, rows), scales=_tiles(s8), shape=(rows, cols), gs=gs)


def _cache_meta(case, seed):
    """References, lengths and tables of a cache in use, as one int32 array: `seqs` rows,
    about half of them filled, some sharing their first pages with another."""
    rng = np.random.RandomState(seed & 0x7FFFFFFF)
    P, B, pt = case["pages"], case["seqs"], case["tokens"]
    T = -(-2 * case["max_len"] // pt) + 1
    live = B // 2 if case["op"] == "fork" else B
    live = max(1, live)
    refs, lens, tab = np.zeros(P, np.int32), np.zeros(B, np.int32), np.full((B, T), -1, np.int32)
    order, at = rng.permutation(P), 0
    for b in range(live):
        want = int(rng.randint(1, case["max_len"] + 1))
        used = -(-want // pt)
        first = 0
        if b and rng.rand() < 0.25:
            first = min(used, int(lens[b - 1]) // pt) // 2
            tab[b, :first] = tab[b - 1, :first]
        if at + used - first > P - (P // 4):
            break
        tab[b, first:used] = order[at:at + used - first]
        at += used - first
        lens[b] = want
        np.add.at(refs, tab[b, :used], 1)
    return refs, lens, tab, rng, P - at


def _fork_requests(case, refs, lens, tab, rng, room):
    """Rows, parents and lengths of one call: forks of filled rows at a point of theirs or
    past it, new sequences (parent -1), rows that grow (parent = row)."""
    pt, T = case["tokens"], tab.shape[1]
    filled, empty = np.nonzero(lens > 0)[0], list(np.nonzero(lens == 0)[0])
    grow = list(rng.permutation(filled))
    out = []
    for j in range(case["n"]):
        kind = 0 if j == 0 else int(rng.randint(0, 3))
        if kind == 2 and grow:
            row = parent = int(grow.pop())
            L = int(min(lens[row] + rng.randint(1, pt + 2), T * pt))
        elif empty:
            row, parent = int(empty.pop(0)), -1 if kind == 1 or not len(filled) else int(rng.choice(filled))
            base = case["max_len"] // 4 + 1 if parent < 0 else int(lens[parent])
            L = int(rng.randint(1, base + pt + 1))
        else:
            break
        have = 0 if parent < 0 else int(lens[parent])
        first = -(-have // pt) if parent == row else min(L, have) // pt
        cost = -(-L // pt) - first
        if cost > room:
            break
        room -= cost
        out.append((row, parent, L))
    if not out:
        row = int(filled[0])
        out.append((row, row, int(lens[row])))
    return np.array(out, np.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        return dict(case=case, x=_rows(g, case["rows"], case["cols"]).to(_DT[case["dtype"]]))
    if op == "matmul":
        return dict(case=case, a=_packed(g, case["m"], case["k"], case["format"]),
                    b=_packed(g, case["n"], case["k"], case["format"]))
    planes, P = case["planes"], case["pages"]
    inner = (case["tokens"], case["heads"], case["dim"])

    def values(count):
        out = torch.empty((planes, count) + inner, dtype=_DT[case["dtype"]], device="cuda")
        for p in range(planes):
            out[p] = torch.randn((count,) + inner, generator=g, device="cuda").to(out.dtype)
        return out

    st = dict(case=case, pages=values(P))
    if op == "copy":
        rng = np.random.RandomState(seed & 0x7FFFFFFF)
        perm = rng.permutation(P).astype(np.int32)
        st["ids"] = torch.from_numpy(perm[:case["n"]].copy()).cuda()
        if case["way"] == "move":
            st["to"] = torch.from_numpy(perm[case["n"]:2 * case["n"]].copy()).cuda()
        else:
            st["flat"] = values(case["n"])
        return st
    refs, lens, tab, rng, room = _cache_meta(case, seed)
    meta = np.concatenate((refs, lens, tab.reshape(-1)))
    st["meta0"] = torch.from_numpy(meta).cuda()
    st["meta"] = st["meta0"].clone()
    if op == "fork":
        rows = _fork_requests(case, refs, lens, tab, rng, room)
        st["rows"], st["parents"], st["lens"] = (torch.from_numpy(rows[:, i].copy()).cuda() for i in range(3))
    else:
        st["rows"] = torch.from_numpy(rng.permutation(case["seqs"])[:case["n"]].astype(np.int32)).cuda()
    return st


# -------------------------------------------------------------------------------- passes

def _views(st):
    P, B = st["case"]["pages"], st["case"]["seqs"]
    m = st["meta"]
    return m[:P], m[P:P + B], m[P + B:].view(B, -1)


def _plain_fork(st):
    refs, lens, tab = _views(st)
    pages, pt = st["pages"], st["case"]["tokens"]
    rows, parents, want = (st[k].long() for k in ("rows", "parents", "lens"))
    same = parents == rows
    src = tab[parents.clamp(min=0)].long()
    have = torch.where(parents >= 0, lens[parents.clamp(min=0)].long(), 0)
    upto = torch.minimum(have, want)
    first = torch.where(same, (have + pt - 1) // pt, upto // pt)
    total = (want + pt - 1) // pt
    new = total - first
    base = torch.cumsum(new, 0) - new
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    slot = torch.arange(tab.shape[1], device=tab.device)[None]
    fresh = (slot >= first[:, None]) & (slot < total[:, None])
    ids = free[(base[:, None] + slot - first[:, None]).clamp(0, free.numel() - 1)]
    table = torch.where(slot < first[:, None], src, torch.where(fresh, ids, -1))
    shared = (slot < first[:, None]) & ~same[:, None]
    refs.index_add_(0, table[shared], torch.ones_like(table[shared], dtype=torch.int32))
    refs[table[fresh]] = 1
    part = ~same & (upto % pt != 0)
    at = first.clamp(max=tab.shape[1] - 1)[:, None]
    raw = pages.view(torch.int64)
    raw.index_copy_(1, table.gather(1, at)[:, 0][part], raw.index_select(1, src.gather(1, at)[:, 0][part]))
    tab[rows] = table.to(torch.int32)
    lens[rows] = want.to(torch.int32)
    return dict(meta=st["meta"], pages=pages)


def _plain_free(st):
    refs, lens, tab = _views(st)
    pages, pt = st["pages"], st["case"]["tokens"]
    rows = st["rows"].long()
    slot = torch.arange(tab.shape[1], device=tab.device)[None]
    held = tab[rows][slot < ((lens[rows] + pt - 1) // pt)[:, None]].long()
    refs.index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    tab[rows] = -1
    lens[rows] = 0
    if not st["case"]["compact"]:
        return dict(meta=st["meta"])
    used = refs > 0
    live = used.sum()
    page = torch.arange(refs.numel(), device=refs.device)
    movers, holes = page[used & (page >= live)], page[~used & (page < live)]
    to = page.clone()
    to[movers] = holes
    refs[holes] = refs[movers]
    refs[movers] = 0
    tab.copy_(torch.where(tab >= 0, to[tab.clamp(min=0).long()].to(torch.int32), -1))
    raw = pages.view(torch.int64)
    raw.index_copy_(1, holes, raw.index_select(1, movers))
    return dict(meta=st["meta"], pages=pages, live=live.to(torch.int32).reshape(1))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q, sc, s8, _ = _plain_quantize(st["x"], case["format"])
        values = (q * sc[..., None]).reshape(case["rows"], -1)[:, :case["cols"]]
        return dict(values=values.to(torch.bfloat16).contiguous(), scales=_tiles(s8))
    if op == "matmul":
        a, b = (_values32(t["codes"], t["scales"], t["shape"], case["format"], t["gs"]) for t in (st["a"], st["b"]))
        return (a @ b.t()).to(_DT[case["out"]])
    if op == "copy":
        ids, raw = st["ids"].long(), st["pages"].view(torch.int64)  # 8 bytes at a time
        if case["way"] == "gather":
            torch.index_select(raw, 1, ids, out=st["flat"].view(torch.int64))
            return st["flat"]
        if case["way"] == "scatter":
            raw.index_copy_(1, ids, st["flat"].view(torch.int64))
        else:
            raw.index_copy_(1, st["to"].long(), raw.index_select(1, ids))
        return st["pages"]
    st["meta"].copy_(st["meta0"])  # the same call again: from the cache as it was
    return _plain_fork(st) if op == "fork" else _plain_free(st)


def _run_own(st):
    case = st["case"]
    op = case["op"]
    if op in ("quantize", "matmul"):
        from lossless_float_weight_b200 import mx
        if op == "quantize":
            q = mx.quantize(st["x"], case["format"])
            return dict(values=mx.dequantize(q, torch.bfloat16), scales=q.scales)
        a, b = (mx.MxTensor(t["codes"], t["scales"], t["shape"], case["format"], t["gs"]) for t in (st["a"], st["b"]))
        return mx.matmul(a, b, _DT[case["out"]])
    from lossless_float_weight_b200 import pages
    if op == "copy":
        if "ws" not in st:  # scratch that a program keeps
            st["ws"] = pages.copy_workspace(st["pages"].device)
        if case["way"] == "gather":
            return pages.copy(st["pages"], st["ids"], st["flat"], None, ws=st["ws"])
        if case["way"] == "scatter":
            return pages.copy(st["flat"], None, st["pages"], st["ids"], ws=st["ws"])
        return pages.copy(st["pages"], st["ids"], st["pages"], st["to"], ws=st["ws"])
    if "pool" not in st:  # the handle that a program keeps for its cache
        st["pool"] = pages.PagePool(st["pages"], case["tokens"], case["seqs"], meta=st["meta"])
    pool = st["pool"]
    st["meta"].copy_(st["meta0"])
    if op == "fork":
        pool.fork(st["rows"], st["parents"], st["lens"])
        return dict(meta=st["meta"], pages=st["pages"])
    pool.free(st["rows"], compact=case["compact"])
    if not case["compact"]:
        return dict(meta=st["meta"])
    return dict(meta=st["meta"], pages=st["pages"], live=pool.live)


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# -------------------------------------------------------------------------- work, 64 bits

def work(case):
    op = case["op"]
    if op == "quantize":
        rows, cols, blk = case["rows"], case["cols"], _BLOCK[case["format"]]
        n = rows * cols
        # the values in, the values they stand for out, the scales out; a comparison, a
        # division and a rounding a value
        return dict(bytes=n * _SIZE[case["dtype"]] + n * 2 + rows * -(-cols // blk), flops=3 * n)
    if op == "matmul":
        m, n, k, blk = case["m"], case["n"], case["k"], _BLOCK[case["format"]]
        held = (m + n) * (-(-k // 2) + -(-k // blk))
        return dict(bytes=held + m * n * _SIZE[case["out"]], flops=2 * m * n * k)
    page = case["planes"] * _SIZE[case["dtype"]] * case["tokens"] * case["heads"] * case["dim"]
    if op == "copy":
        return dict(bytes=2 * case["n"] * page + 4 * case["n"] * (2 if case["way"] == "move" else 1), flops=0)
    # the tables are read and written; how many pages move depends on the sequences: half
    # of the forks end inside a page, and the freed share of the live ones has to close up
    table = 8 * (case["pages"] + case["seqs"] * (2 + -(-2 * case["max_len"] // case["tokens"])))
    if op == "fork":
        return dict(bytes=table + case["n"] * page, flops=0)
    moved = 0
    if case["compact"]:
        held = min(case["pages"] * 3 // 4, case["seqs"] * (case["max_len"] // (2 * case["tokens"]) + 1))
        moved = held * (case["seqs"] - min(case["n"], case["seqs"])) // case["seqs"] // 2
    return dict(bytes=table + 2 * moved * page, flops=0)


def _exact_quantize(x, fmt):
    """By the definition: every value to the nearest of the grid's, by comparison with the
    midpoints times the scale (exact in 64 bits)."""
    rows, cols = x.shape
    blk = _BLOCK[fmt]
    nb = -(-cols // blk)
    xd = torch.zeros(rows, nb * blk, dtype=torch.float64, device=x.device)
    xd[:, :cols] = x
    xd = xd.view(rows, nb, blk)
    top = xd.abs().max(-1).values
    if fmt == "mxfp4":
        powers = torch.tensor([math.ldexp(1.0, i - 127) for i in range(257)], dtype=torch.float64, device=x.device)
        e = (torch.searchsorted(powers[2:], top, right=True) - 1).clamp(0, 254)  # from 2^(e + 2), e >= -127
        s = powers[e]
        g = 1.0
        shown = s
    else:
        g = float(np.float32(float(top.max()) / 2688.0)) or 1.0
        grid = torch.tensor([m * 2.0 ** -9 if ex == 0 else (8 + m) * 2.0 ** (ex - 10) for ex in range(16) for m in range(8)][:127],
                            dtype=torch.float64, device=x.device)
        mid = (grid[1:] + grid[:-1]) / 2 * (6 * g)
        up, down = torch.searchsorted(mid, top, right=True), torch.searchsorted(mid, top)
        s = grid[torch.where(down % 2 == 0, down, up)]  # a tie (up = down + 1) takes the even code
        shown = s
    unit = s * g
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    code = torch.zeros(xd.shape, dtype=torch.int64, device=x.device)
    for i in range(7):  # an even code below the midpoint keeps a tie
        m = mid[i] * unit[..., None]
        code += (xd.abs() > m) if i % 2 == 0 else (xd.abs() >= m)
    code = torch.where(unit[..., None] > 0, code, 0)
    v = torch.where(xd < 0, -grid[code], grid[code]) * unit[..., None]
    return v.reshape(rows, -1)[:, :cols].contiguous(), shown


def _exact_values(t, fmt):
    rows, cols = t["shape"]
    blk = _BLOCK[fmt]
    c = torch.empty(rows, 2 * t["codes"].shape[1], dtype=torch.int64, device="cuda")
    c[:, 0::2], c[:, 1::2] = t["codes"] % 16, t["codes"] // 16
    c = c[:, :cols]
    e = c % 8 // 2
    mag = torch.where(e == 0, (c % 2).double() / 2, (2 + c % 2).double() * 0.25 * (1 << e).double())
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(cols, device="cuda")[None] // blk
    at = ((r // 128) * -(-(-(-cols // blk)) // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    byte = t["scales"].view(torch.uint8)[at].long()
    if fmt == "mxfp4":
        s = torch.tensor([math.ldexp(1.0, i - 127) for i in range(255)], dtype=torch.float64, device="cuda")[byte]
    else:
        ex, m = byte // 8, byte % 8
        s = torch.where(ex == 0, 2 * m, (8 + m) << ex).double() * 2.0 ** -10 * t["gs"].double()
    return torch.where(c >= 8, -mag, mag) * s


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v, s = _exact_quantize(st["x"], case["format"])
        rows, nb = s.shape
        rt, bt = -(-rows // 128), -(-nb // 4)
        full = torch.zeros(rt * 128, bt * 4, dtype=torch.float64, device="cuda")
        if case["format"] == "mxfp4":
            full += 2.0 ** -127  # a scale byte of 0
        full[:rows, :nb] = s
        tiles = torch.stack([full[:, 4 * i:4 * i + 4].reshape(rt, 4, 32, 4).transpose(1, 2).reshape(rt, 512)
                             for i in range(bt)], 1)
        return dict(values=v, scales=tiles.reshape(-1))
    if op == "matmul":
        return _exact_values(st["a"], case["format"]) @ _exact_values(st["b"], case["format"]).t()
    if op == "copy":
        ids = st["ids"].tolist()
        if case["way"] == "gather":
            return torch.stack([st["pages"][:, i] for i in ids], 1)
        raw = st["pages"].view(torch.uint8)
        for j, i in enumerate(ids):
            raw[:, i if case["way"] == "scatter" else int(st["to"][j])] = \
                st["flat"].view(torch.uint8)[:, j] if case["way"] == "scatter" else raw[:, i]
        return st["pages"]
    if op == "free" and not case["compact"]:
        return None  # whole numbers alone
    # request by request, page by page
    P, B, pt = case["pages"], case["seqs"], case["tokens"]
    meta, raw = st["meta0"].cpu().numpy(), st["pages"].view(torch.uint8)
    refs, lens, tab = meta[:P].copy(), meta[P:P + B].copy(), meta[P + B:].reshape(B, -1).copy()
    if op == "fork":
        free = [p for p in range(P) if refs[p] == 0]
        for row, parent, L in zip(*(st[k].tolist() for k in ("rows", "parents", "lens"))):
            have = int(lens[parent]) if parent >= 0 else 0
            first = -(-have // pt) if parent == row else min(L, have) // pt
            for s in range(first, -(-L // pt)):
                p = free.pop(0)
                if s == first and parent != row and min(L, have) % pt:
                    raw[:, p] = raw[:, int(tab[parent, s])]
        return dict(pages=st["pages"])
    for row in st["rows"].tolist():
        for s in range(-(-int(lens[row]) // pt)):
            refs[tab[row, s]] -= 1
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] == 0]
    for p in range(live, P):
        if refs[p] > 0:
            raw[:, holes.pop(0)] = raw[:, p]
    return dict(pages=st["pages"])
