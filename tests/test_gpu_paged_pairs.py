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
from test_gpu_paged import BF, Case, half

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


def definition(c, seqs=None):
    """(token rows, float64 results, sum_i p_i |row_i|) of the sequences' tokens, a sequence at a time."""
    ends = {}
    for i, b, p in c.toks:
        ends.setdefault(b, []).append((i, p))

    def gather(store, table, b, lo, hi):
        r = torch.arange(lo, hi, device="cuda")
        ps = store.shape[1]
        return store[table[b][r // ps].long(), r % ps].double()
    for b, toks in ends.items():
        if seqs is not None and b not in seqs:
            continue
        idx = torch.tensor([i for i, _ in toks], device="cuda")
        pos = torch.tensor([p for _, p in toks], device="cuda")
        keep = pos >= 0
        idx, pos = idx[keep], pos[keep]
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
    c = Case(seed=200 + k, pad=1, **MANY[k])
    for name, ps in (("tok", "tok_pages"), ("kv", "kv_pages")):
        if ps in c.kw:
            c.kw[name + "_table"] = widen(c.kw[name + "_table"], 4096 // c.kw[ps].shape[1])
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
