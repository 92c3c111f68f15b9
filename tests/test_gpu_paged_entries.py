"""GPU parity of the ways in which finished entries get into pages that
csa_paged_attention reads: csa_paged_append of rows that are not to be turned, and
dense caches seen as pages."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import lib_loaded
from test_gpu_paged import BF, F32, half, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def csa():
    lib_loaded()
    import long_context_compressed_02_b200 as m
    return m


def rows_of(store, kind, table, n):
    """The first n rows of a sequence as the attention reads them, float64."""
    if kind == "bf16":
        return O.page_rows(np64(store[0]), table, 0, n)
    return O.e4m3_page_rows(store[0].cpu().numpy(), np64(store[1]), store[2].cpu().numpy(), table, 0, n)


def check(out, q, rows, sink, seq):
    """Tolerance of test_gpu_paged.py; q, out [n, H, D], rows of sequence seq[i]."""
    for i, b in enumerate(seq):
        ref, mag = O.paged_attention_row(np64(q[i]), rows[b], 1 / math.sqrt(q.shape[-1]), np64(sink))
        assert np.all(np.abs(np64(out[i]) - ref) <= (2.0 ** -8 + 2.0 ** -9) * mag + half(out.dtype) * np.abs(ref)), (i, b)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,dt", [(512, BF), (128, F32)])
def test_append_of_finished_entries(csa, kind, D, dt):
    """Entries that the compressor has normalised and turned go in as rows of their own batch (position: the
    entry's number): bf16 with inv_freq None, e4m3 (whose rows need a rotated part) with frequencies of zero."""
    m, ps, H = 4, 16, 8
    n_e, first = [37, 5], [0, 20]                              # entries now, entries before them
    g = torch.Generator(device="cuda").manual_seed(D)
    ent = [torch.randn(f + n, D, generator=g, device="cuda").to(dt) for n, f in zip(n_e, first)]
    total = sum(-(-len(e) // ps) for e in ent)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    order, at = torch.randperm(total, generator=g, device="cuda").to(torch.int32), 0
    for b, e in enumerate(ent):
        k = -(-len(e) // ps)
        table[b, :k] = order[at:at + k]
        at += k
    if kind == "bf16":
        store = (torch.zeros(total, ps, D, dtype=BF, device="cuda"),)
        kw, still = {}, None
    else:
        store = (torch.zeros(total, ps, D - 64, dtype=torch.uint8, device="cuda"), torch.zeros(total, ps, 64, dtype=BF, device="cuda"),
                 torch.zeros(total, ps, device="cuda"))
        kw, still = dict(pages_rope=store[1], pages_scale=store[2]), torch.zeros(32, dtype=torch.float64, device="cuda")
    cu = lambda n: torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32, device="cuda")  # noqa: E731
    pos = lambda p: torch.tensor(p, dtype=torch.int64, device="cuda")                      # noqa: E731
    if any(first):
        csa.csa_paged_append(torch.cat([e[:f] for e, f in zip(ent, first)]), cu(first), pos([0, 0]), table, store[0], still, norm=False, **kw)
    csa.csa_paged_append(torch.cat([e[f:] for e, f in zip(ent, first)]), cu(n_e), pos(first), table, store[0], still, norm=False, **kw)
    csa.check_device_error()
    tab = table.cpu().numpy()
    for b, e in enumerate(ent):
        x = np64(e)
        if kind == "bf16":
            assert np.array_equal(O.page_rows(np64(store[0]), tab[b], 0, len(e)), np64(e.to(BF)))
            continue
        s = O.page_rows(store[2].double().cpu().numpy(), tab[b], 0, len(e))[:, None]
        want = np.abs(x[:, :-64]).max(-1, keepdims=True) / 448
        assert np.all(np.abs(s - want) <= want * 2.0 ** -22)   # a division and a rounding in float32
        # turned by an angle of zero: the elements themselves, rounded once
        assert np.array_equal(O.page_rows(np64(store[1]), tab[b], 0, len(e)), np64(e[:, -64:].to(BF)))
        deq = O.e4m3_decode(O.page_rows(store[0].cpu().numpy(), tab[b], 0, len(e))) * s
        assert np.all(np.abs(deq - x[:, :-64]) <= np.maximum(2.0 ** -4 * np.abs(x[:, :-64]), s * 2.0 ** -10) + 2.0 ** -20 * s * 448)
    q = torch.randn(2, H, D, generator=g, device="cuda").to(BF)
    sink = torch.randn(H, generator=g, device="cuda")
    last = [len(e) * m - 1 for e in ent]
    out = csa.csa_paged_attention(q, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), pos(last), W=0, m=m, sink=sink,
                                  kv_pages=store[0], kv_table=table, **(dict(kv_rope=store[1], kv_scale=store[2]) if kind == "e4m3" else {}))
    csa.check_device_error()
    check(out, q, [rows_of(store, kind, tab[b], len(e)) for b, e in enumerate(ent)], sink, [0, 1])


def test_dense_caches_seen_as_pages(csa):
    """What csa_compress_append writes into a dense e4m3 cache whose capacity is a multiple of the page is read
    through a table of consecutive pages, and gives what the dense call gives."""
    n_seq, m, cap, D, H, ps = 3, 4, 64, 512, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    nope = torch.zeros(n_seq, cap, D - 64, dtype=torch.uint8, device="cuda")
    rope = torch.zeros(n_seq, cap, 64, dtype=BF, device="cuda")
    scale = torch.zeros(n_seq, cap, device="cuda")
    rings = [torch.zeros(n_seq, 2 * m, D, dtype=BF, device="cuda") for _ in range(2)]
    B = torch.randn(2 * m, D, generator=g, device="cuda")
    start = torch.tensor([0, 3, 40], dtype=torch.int64, device="cuda")
    steps = 30
    for t in range(steps):
        c, z = (torch.randn(n_seq, D, generator=g, device="cuda").to(BF) for _ in range(2))
        csa.csa_compress_append(c, z, B, m, True, start + t, *rings, nope, rope, scale)
    pos = start + steps - 1
    first = [0, 0, 10]                                         # entries before the first appended token are zeros
    table = torch.arange(n_seq * cap // ps, dtype=torch.int32, device="cuda").reshape(n_seq, -1)
    q = torch.randn(n_seq, 1, H, D, generator=g, device="cuda").to(BF)
    sink = torch.randn(H, generator=g, device="cuda")
    pages = (nope.view(-1, ps, D - 64), rope.view(-1, ps, 64), scale.view(-1, ps))
    out = csa.csa_paged_attention(q[:, 0], torch.arange(n_seq + 1, dtype=torch.int32, device="cuda"), pos, W=0, m=m, sink=sink,
                                  kv_pages=pages[0], kv_rope=pages[1], kv_scale=pages[2], kv_table=table)
    csa.check_device_error()
    rows = [rows_of(pages, "e4m3", table[b].cpu().numpy(), int(pos[b] + 1) // m) for b in range(n_seq)]
    assert all(len(r) > f and np.abs(r[f:]).max() > 0 for r, f in zip(rows, first))
    check(out, q[:, 0], rows, sink, range(n_seq))
    dense, lse = csa.hca_dense_attn(q, nope, pos, m, kv_rope=rope, kv_scale=scale)
    # its own sink: weights of the rows against e^sink; the dense call rounds codes * scale to bf16, 2^-8 of each
    # element, which moves a logit by 2^-8 sum |q||row| / sqrt(D) at most
    for b in range(n_seq):
        share = 1 / (1 + np.exp(np64(sink) - np64(lse[b, 0])))
        ref, mag = O.paged_attention_row(np64(q[b, 0]), rows[b], 1 / math.sqrt(D), np64(sink))
        e = 2.0 ** -8 / math.sqrt(D) * (np.abs(np64(q[b, 0])) @ np.abs(rows[b]).T).max(-1, keepdims=True)
        tol = (2 * (2.0 ** -8 + 2.0 ** -9) + 2.0 ** -8 + 2.02 * e) * mag + half(BF) * np.abs(ref)
        assert np.all(np.abs(np64(out[b]) - np64(dense[b, 0]) * share[:, None]) <= tol), b
