"""GPU parity of the pair kernel of csa_paged_attention (prompt chunks on pairs of
SMs) where its clusters take several items each, and where tables are wider than
the rows in them.  Every token is compared with its definition in float64, with
the tolerance of test_gpu_paged.py:
(2^-8 + 2^-9) sum_i p_i |row_i| + half a step of the output.
"""
import math

import pytest
import torch

from gpu_util import lib_loaded
from test_gpu_paged import ATTN, BF, F32, Case, half

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def csa():
    lib_loaded()
    import long_context_compressed_02_b200 as m
    return m


def widen(table, pages):
    """The table with columns of -1 up to `pages`: what a server keeps for the longest context it allows."""
    out = torch.full((table.shape[0], pages), -1, dtype=torch.int32, device=table.device)
    out[:, :table.shape[1]] = table
    return out


def widened(c, rows=4096):
    """The case with tables of `rows` rows; what its calls take."""
    for name, ps in (("tok", "tok_pages"), ("kv", "kv_pages")):
        if ps in c.kw:
            c.kw[name + "_table"] = widen(c.kw[name + "_table"], rows // c.kw[ps].shape[1])
    return c


def on_pairs(csa, c):
    return csa.csa_paged_attention_pairs(c.q, c.qp, **{k: v for k, v in c.kw.items() if k in (
        "tok_pages", "tok_table", "W", "kv_pages", "kv_table")})


def definition(c):
    """(token rows, float64 results, sum_i p_i |row_i|) of the tokens, some of a sequence at a time."""
    ends = {}
    for i, b, p in c.toks:
        ends.setdefault(b, []).append((i, p))

    def gather(store, table, b, lo, hi):
        r = torch.arange(lo, hi, device="cuda")
        ps = store.shape[1]
        return store[table[b][r // ps].long(), r % ps].double()
    for b, toks in ends.items():
        idx = torch.tensor([i for i, _ in toks], device="cuda")
        pos = torch.tensor([p for _, p in toks], device="cuda")
        keep = pos >= 0
        idx, pos = idx[keep], pos[keep]
        if len(idx) == 0:
            continue
        first, last = int(pos[0]), int(pos[-1])
        rows, lo, hi = [], [], []                              # a row is seen at positions lo .. hi - 1
        if c.W is not None:
            r0 = 0 if c.W == 0 else max(0, first - c.W + 1)
            rows.append(gather(c.kw["tok_pages"], c.kw["tok_table"], b, r0, last + 1))
            at = torch.arange(r0, last + 1, device="cuda")
            lo.append(at)
            hi.append(at + (c.W or 1 << 40))
        if c.m:
            ne = (last + 1) // c.m
            rows.append(gather(c.kw["kv_pages"], c.kw["kv_table"], b, 0, ne))
            at = (torch.arange(ne, device="cuda") + 1) * c.m - 1
            lo.append(at)
            hi.append(at + (1 << 40))
        rows, lo, hi = torch.cat(rows), torch.cat(lo), torch.cat(hi)
        step = max(1, (1 << 25) // (c.H * max(1, len(rows))))
        for t in range(0, len(idx), step):
            p = pos[t:t + step, None]
            z = torch.einsum("thd,kd->thk", c.q[idx[t:t + step]].double(), rows) / math.sqrt(c.D)
            z.masked_fill_(((p < lo) | (p >= hi))[:, None], -math.inf)
            if c.sink is not None:
                z = torch.cat((z, c.sink.double()[None, :, None].expand(len(p), -1, 1)), -1)
            none = (z == -math.inf).all(-1, keepdim=True)      # no row and no sink: zeros
            w = torch.softmax(z, -1).masked_fill_(none, 0.0)[..., :len(rows)]
            yield idx[t:t + step], torch.einsum("thk,kd->thd", w, rows), torch.einsum("thk,kd->thd", w, rows.abs())


def check_all(c, out):
    worst = 0.0
    for idx, ref, mag in definition(c):
        got = out[idx].double()
        tol = (2.0 ** -8 + 2.0 ** -9) * mag + half(out.dtype) * ref.abs()
        worst = max(worst, float(((got - ref).abs() / tol.clamp(min=1e-300)).nan_to_num(nan=math.inf).max()))
    assert worst <= 1.0, f"an element is off by {worst} tolerances"


# 148 SMs make 74 clusters; an item is 2 tokens of 64 heads, 4 of 32, 128 of one
MANY = [
    # one-tile items from one to five blocks: 8 a cluster
    dict(lens=[40] * 32, pos=[0, 20, 61, 130] * 8, H=64, D=512, W=0),
    # one chunk: one tile an item at its start, six at its end; 10 items a cluster
    dict(lens=[1481], pos=[0], H=64, D=512, W=0),
    # short sequences by the hundred, empty ones between them
    dict(lens=[2, 0, 4, 2] * 150, pos=[0, 7, 63, 190] * 150, H=64, D=512, W=0, ps=16),
    # single tokens among them: items of one token
    dict(lens=[1, 3, 2, 5] * 90, pos=[5, 62, 255, 319] * 90, H=64, D=512, W=0, ps=128, sink=False),
    # a window and entries, whose blocks are patched at both ends
    dict(lens=[500, 301], pos=[10, 700], H=64, D=512, W=100, m=4),
    # entries only, the first tokens without any
    dict(lens=[330, 340], pos=[0, 100], H=64, D=512, W=None, m=2, sink=False),
    # more tokens an item
    dict(lens=[900, 800], pos=[0, 33], H=32, D=512, W=0),
    dict(lens=[130] * 10, pos=[64 * i for i in range(10)], H=20, D=512, W=0, ps=32),
    dict(lens=[300] * 100, pos=[3 * i for i in range(100)], H=1, D=512, W=0),
]


@pytest.mark.parametrize("k", range(len(MANY)))
def test_several_items_for_each_cluster(csa, k):
    c = widened(Case(seed=200 + k, pad=1, **MANY[k]))
    assert on_pairs(csa, c)
    out = torch.full_like(c.q, 9.0)
    csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, **c.kw)
    csa.check_device_error()
    check_all(c, out)
    assert bool((out[-1] == 9.0).all())
    # again while copies on another stream fill the memory, so that loads take longer
    src = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    dst = torch.empty_like(src)
    side = torch.cuda.Stream()
    for _ in range(4):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):
                dst.copy_(src)
        again = csa.csa_paged_attention(c.q, c.cu, c.qp, out=torch.full_like(c.q, 9.0), **c.kw)
        assert torch.equal(again, out)
    csa.check_device_error()


# ---------------------------------------------------------------- one kernel and the other

CHUNKS = [kw for kw in ATTN if sum(kw["lens"]) > 74 and kw["D"] == 512 and kw.get("kind") != "e4m3"
          and sum(kw["lens"]) >= 2 * len(kw["lens"]) and (kw.get("W") in (0, None) and "W" in kw or "m" in kw)]


@pytest.mark.parametrize("k", range(len(CHUNKS)))
def test_chunks_with_wide_tables(csa, k):
    """Short contexts on pairs, where only the width of the table sends them; every dtype of the output."""
    c = widened(Case(seed=300 + k, pad=2, **CHUNKS[k]))
    assert on_pairs(csa, c)
    out = torch.full_like(c.q, 9.0)
    csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, **c.kw)
    full = torch.full(c.q.shape, 9.0, device="cuda")
    csa.csa_paged_attention(c.q, c.cu, c.qp, out=full, **c.kw)
    csa.check_device_error()
    check_all(c, out)
    check_all(c, full)
    assert torch.equal(full.to(BF), out) and bool((out[-2:] == 9.0).all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,W,m", [(64, 0, 0), (16, 100, 0), (24, 0, 0), (64, 40, 4), (64, None, 4)])
def test_rows_that_some_tokens_see(csa, H, W, m, wide):
    """A row with a NaN or an infinity, whole or in one element, reaches the tokens that see it and no others."""
    n, p0 = 110, 90
    c = Case(lens=[n], pos=[p0], H=H, D=512, W=W, m=m)
    if wide:
        widened(c)
    assert on_pairs(csa, c) == (wide or H < 64)
    clean = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    for store, tab, rows in (("tok_pages", "tok_table", (95, 127, 128, 150, 199)), ("kv_pages", "kv_table", (22, 31, 49))):
        if store not in c.kw:
            continue
        for row in rows:
            # tokens first .. last - 1 see the row
            first = row - p0 if store == "tok_pages" else 4 * row + 3 - p0
            last = min(n, row + c.W - p0) if store == "tok_pages" and c.W else n
            first = max(0, first)
            ps = c.kw[store].shape[1]
            at = int(c.kw[tab][0, row // ps]), row % ps
            for bad in (math.nan, math.inf, -math.inf):
                for dims in (slice(None), slice(300, 301)):
                    pages = c.kw[store].clone()
                    pages[at][dims] = bad
                    out = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, **{store: pages}))
                    what = (store, row, bad, dims)
                    assert torch.equal(out[:first], clean[:first]) and torch.equal(out[last:], clean[last:]), what
                    assert bool(torch.isnan(out[first:last]).any(-1).all()), what
    csa.check_device_error()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,W", [(64, 0), (16, 128)])
def test_negative_positions_on_pairs(csa, H, W, wide):
    """Rows at negative positions are left as they were, a pair that has one of each kind among them."""
    for n, back in ((90, 3), (91, 40)):
        c = Case(lens=[n], pos=[0], H=H, D=512, W=W)
        if wide:
            widened(c)
        assert on_pairs(csa, c) == (wide or H < 64)
        c.qp -= back
        c.toks = [(i, b, p - back) for i, b, p in c.toks]
        for dt in (BF, F32):
            out = torch.full(c.q.shape, 3.0, dtype=dt, device="cuda")
            csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, **c.kw)
            csa.check_device_error()
            assert bool((out[:back] == 3.0).all())
            check_all(c, out)


@pytest.mark.parametrize("wide", [False, True])
def test_batch_that_ends_inside_a_sequence_on_pairs(csa, wide):
    n = 91                                                     # inside a pair of the second sequence
    c = Case(lens=[45, 90], pos=[100, 40], H=64, D=512, W=0)
    if wide:
        widened(c)
    room = torch.full(c.q.shape, 9.0, dtype=BF, device="cuda")
    short = c.q[:n]
    assert csa.csa_paged_attention_pairs(short, c.qp, W=0, tok_pages=c.kw["tok_pages"], tok_table=c.kw["tok_table"]) == wide
    csa.csa_paged_attention(short, c.cu, c.qp, out=room[:n], **c.kw)
    csa.check_device_error()
    c.toks = c.toks[:n]
    check_all(c, room)
    assert bool((room[n:] == 9.0).all())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ps", [16, 64])
def test_missing_page_on_pairs(csa, ps, wide):
    """Recorded where a token sees rows of the page; the tokens that do not keep their results."""
    c = Case(lens=[100], pos=[60], H=64, D=512, W=0, ps=ps)
    if wide:
        widened(c)
    assert on_pairs(csa, c) == wide
    clean = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    csa.check_device_error()
    for page in (-1, c.pages.shape[0]):
        tab = c.kw["tok_table"].clone()
        tab[0, 128 // ps] = page
        out = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, tok_table=tab))
        with pytest.raises(csa.CsaError, match="page"):
            csa.check_device_error()
        csa.check_device_error()
        assert torch.equal(out[:68], clean[:68])               # positions 60 .. 127


def test_large_logits_on_pairs(csa):
    """Logits that grow along many tiles, for one item and for several a cluster."""
    for lens, H in (([90], 64), ([400], 64), ([700], 16)):
        c = widened(Case(lens=lens, pos=[900], H=H, D=512, W=0, sink=False))
        assert on_pairs(csa, c)
        ramp = torch.linspace(0.2, 4.0, 900 + lens[0])
        for u in range(len(ramp)):
            c.pages[c.tab[0, u // 64], u % 64] *= ramp[u]
        c.kw["tok_pages"] = c.pages.cuda()
        out = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
        csa.check_device_error()
        check_all(c, out)


def test_replayed_pairs_follow_positions_and_lengths(csa):
    """A captured call over many items reads lengths, positions and tables at replay."""
    c = widened(Case(lens=[300, 200, 0, 100], pos=[0, 50, 3, 200], H=64, D=512, W=0))
    assert on_pairs(csa, c)
    csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    out = torch.full_like(c.q, 9.0)
    with torch.cuda.graph(g):
        csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, **c.kw)
    cu = c.cu.clone()
    for lens, back in (([300, 200, 0, 100], 0), ([20, 200, 0, 1], 0), ([0, 0, 0, 0], 0), ([299, 150, 0, 33], 30)):
        c.cu.copy_(torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32))
        out.fill_(9.0)
        c.qp[1:] -= back
        g.replay()
        torch.cuda.synchronize()
        want = csa.csa_paged_attention(c.q, c.cu, c.qp, out=torch.full_like(c.q, 9.0), **c.kw)
        assert torch.equal(out, want)
        assert bool((out[sum(lens):] == 9.0).all())
    c.cu.copy_(cu)
    csa.check_device_error()
