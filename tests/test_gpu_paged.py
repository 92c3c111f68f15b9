"""GPU parity of the paged serving step against float64 definitions: rotary
positions, the norm of queries and keys with the rotation, the append to a paged
cache, the attention of a ragged batch's new tokens, and a run of them together.

Tolerances.  A result is rounded once to its dtype, by at most HALF of its value
(torch.finfo(t).eps / 2).  Before that a row element carries float32 arithmetic:
the reduced angle (up to pi) rounds by 2^-23, cos and sin are within 2 units
(2^-22), the scaling, two products and an addition add 4 * 2^-24; the sum of
squares of at most 2048 elements (64 additions a lane and 5 across lanes) is
within 69 * 2^-24, half of that in the root, the root and the gain add 2^-21:
together below 2^-17 of the largest element of the row (times mscale).
Attention: probabilities rounded to bf16 (2^-8 of each term), the logits'
float32 sums, exp2 and the merge (below 2^-9 together at these sizes: 512
products of size q k / sqrt(D) summed with error 2^-23 each, about 15 in all,
give 2^-10): (2^-8 + 2^-9) sum_i p_i |row_i|, then the output's rounding.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import lib_loaded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SLOP = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def csa():
    lib_loaded()
    import long_context_compressed_02_b200 as m
    return m


def half(dt):
    return torch.finfo(dt).eps / 2


def np64(t):
    return t.detach().double().cpu().numpy()


def batch(lens, pos, pad=0):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return (torch.from_numpy(cu).cuda(), torch.tensor(pos, dtype=torch.int64, device="cuda"), int(cu[-1]) + pad,
            O.batch_tokens(cu.tolist(), pos))


BATCHES = {
    "one": ([1], [0]),
    "far": ([1, 1, 1], [1048575, 0, 131072]),
    "ragged": ([5, 0, 17, 1, 0], [3, 9, 4095, 70000, 1]),
    "many": ([1] * 45, list(range(0, 45 * 64, 64))),
}


def close_rows(got, ref, dt, big, what):
    tol = half(dt) * np.abs(ref) + SLOP * big
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.abs(got - ref).max():.3e}"


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("H,D,r,start,il,inv,dt", [
    (64, 512, 64, None, False, True, BF), (8, 128, 128, None, True, False, BF), (3, 96, 32, 8, True, True, F32),
    (1, 16, 16, None, False, False, F32), (5, 2048, 2048, 0, False, False, BF), (2, 1040, 16, 1024, True, False, F32),
    (65, 128, 64, 0, False, False, F32), (1, 512, 64, 0, True, False, BF),
])
def test_rope(csa, name, H, D, r, start, il, inv, dt):
    lens, pos = BATCHES[name]
    cu, qp, n, toks = batch(lens, pos, pad=2)
    g = torch.Generator(device="cuda").manual_seed(H * D + r)
    x = torch.randn(n, H, D, generator=g, device="cuda").to(dt)
    w, ms = csa.csa_rope_freqs(r, factor=4.0, original_len=4096)
    kw = dict(rope_start=start, interleaved=il, inverse=inv, mscale=ms)
    out = torch.full_like(x, 7.0)
    csa.csa_rope(x, cu, qp, w, out=out, **kw)
    same = x.clone()
    assert csa.csa_rope(same, cu, qp, w, out=same, **kw) is same
    csa.check_device_error()
    X, got, w64 = np64(x), np64(out), w.cpu().numpy()
    for i, _, p in toks:
        ref = O.rotate_row(X[i], p, w64, start=start, interleaved=il, inverse=inv, mscale=ms)
        close_rows(got[i], ref, dt, np.abs(X[i]).max(-1, keepdims=True) * ms * 2, (name, i))
        s = D - r if start is None else start
        rest = np.r_[0:s, s + r:D]
        assert np.array_equal(got[i][:, rest], X[i][:, rest])
    assert torch.equal(out[:n - 2], same[:n - 2])
    assert bool((out[n - 2:] == 7.0).all()) and torch.equal(same[n - 2:], x[n - 2:])


def test_rope_views_other_dtype_and_autograd_identity(csa):
    """Strided views in and out, bf16 to float32; the inverse call is the gradient: <g, R x> = <R^T g, x>."""
    cu, qp, n, toks = batch([7, 2], [100, 5])
    big = torch.randn(n, 6, 256, device="cuda").to(BF)
    x = big[:, 1:4, 128:]
    w, _ = csa.csa_rope_freqs(64)
    room = torch.zeros(n, 5, 160, device="cuda")
    y = csa.csa_rope(x, cu, qp, w, interleaved=True, out=room[:, 2:5, 32:])
    for i, _, p in toks:
        ref = O.rotate_row(np64(x[i]), p, w.cpu().numpy(), interleaved=True)
        close_rows(np64(y[i]), ref, F32, 8.0, i)
    assert not room[:, :2].any() and not room[:, 2:, :32].any()
    g = torch.randn(n, 3, 128, device="cuda")
    back = csa.csa_rope(g, cu, qp, w, interleaved=True, inverse=True)
    a, b = float((np64(g) * np64(y)).sum()), float((np64(back) * np64(x)).sum())
    assert abs(a - b) <= SLOP * float(np.abs(np64(g) * np64(y)).sum())


@pytest.mark.parametrize("H", [129, 200, 255, 256])
def test_rope_of_many_narrow_heads(csa, H):
    """A warp's task holds several tokens of more than 128 heads."""
    cu, qp, n, _ = batch([2500, 2500], [7, 100])
    x = torch.randn(n, H, 16, device="cuda").to(BF)
    w, _ = csa.csa_rope_freqs(16)
    out = csa.csa_rope(x, cu, qp, w)
    pos = torch.cat([torch.arange(2500) + 7, torch.arange(2500) + 100]).double().cuda()
    a = (pos[:, None] * w)[:, None]
    X = x.double()
    ref = torch.cat([X[..., :8] * a.cos() - X[..., 8:] * a.sin(), X[..., :8] * a.sin() + X[..., 8:] * a.cos()], -1)
    tol = half(BF) * ref.abs() + SLOP * 2 * X.abs().amax(-1, keepdim=True)
    assert bool(((out.double() - ref).abs() <= tol).all())
    same = x.clone()
    assert torch.equal(csa.csa_rope(same, cu, qp, w, out=same), out)


# ---------------------------------------------------------------- queries and keys

@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("H,Hk,D,r,il,dt,odt,gain,fused", [
    (64, 1, 512, 64, False, BF, BF, True, True), (8, 2, 128, 128, True, BF, F32, False, True),
    (4, 4, 256, 64, True, F32, F32, True, False), (33, 0, 512, 0, False, BF, BF, True, False),
    (1, 1, 48, 16, False, F32, BF, True, True), (2, 1, 2048, 64, False, BF, BF, True, False),
])
def test_qk_norm_rope(csa, name, H, Hk, D, r, il, dt, odt, gain, fused):
    lens, pos = BATCHES[name]
    cu, qp, n, toks = batch(lens, pos, pad=1)
    g = torch.Generator(device="cuda").manual_seed(D + H)
    both = (torch.randn(n, H + Hk, D, generator=g, device="cuda") * 3).to(dt)
    q, k = both[:, :H], both[:, H:] if Hk else None
    if not fused:
        q, k = q.contiguous(), k.contiguous() if Hk else None
    qg = torch.randn(D, generator=g, device="cuda") if gain else None
    kg = torch.rand(D, generator=g, device="cuda") if gain else None
    w = csa.csa_rope_freqs(r)[0] if r else None
    qo = torch.full((n, H, D), 5.0, dtype=odt, device="cuda")
    qo, ko = csa.csa_qk_norm_rope(q, k, cu, qp, w, q_gain=qg, k_gain=kg, interleaved=il, q_out=qo, out_dtype=odt)
    csa.check_device_error()
    w64 = w.cpu().numpy() if r else np.zeros(0)
    for x, y, gg in ((q, qo, qg), (k, ko, kg)):
        if x is None:
            assert y is None
            continue
        X, Y = np64(x), np64(y)
        for i, _, p in toks:
            u = O.norm_row(X[i], None if gg is None else np64(gg))
            close_rows(Y[i], O.rotate_row(u, p, w64, interleaved=il), odt, np.abs(u).max(-1, keepdims=True) * 2, (name, i))
    assert bool((qo[-1] == 5.0).all())
    if odt == dt and Hk:        # in place, on views of one buffer
        csa.csa_qk_norm_rope(q, k, cu, qp, w, q_gain=qg, k_gain=kg, interleaved=il, q_out=q, k_out=k)
        assert torch.equal(q[:-1], qo[:-1]) and torch.equal(k[:-1], ko[:-1])


def test_norm_of_zero_and_huge_rows(csa):
    cu, qp, n, _ = batch([3], [9])
    q = torch.zeros(3, 2, 128, device="cuda", dtype=BF)
    q[1] = 1e18
    q[2] = 1e-20
    y, _ = csa.csa_qk_norm_rope(q, None, cu, qp, None)
    assert not y[0].any() and bool((y[1] == 1.0).all())
    close_rows(np64(y[2]), O.norm_row(np64(q[2])), BF, 1e-14, "tiny")


# ---------------------------------------------------------------- append

def make_pages(rng, n_rows, ps, extra=2):
    """(table [n_seq, max_pages + 1] with -1 where no page is needed, number of pages)."""
    per = [-(-r // ps) for r in n_rows]
    perm = rng.permutation(sum(per) + extra).astype(np.int32)
    tab = np.full((len(per), max(per) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(per):
        tab[b, :k] = perm[at:at + k]
        at += k
    return tab, sum(per) + extra


@pytest.mark.parametrize("lens,pos", [([1], [0]), ([6, 0, 33, 1], [15, 3, 60, 200]), ([1] * 20, list(range(55, 75)))])
@pytest.mark.parametrize("D,ps,kind,dt,il,norm", [
    (512, 64, "bf16", BF, False, True), (512, 16, "e4m3", BF, True, True), (128, 1, "e4m3", F32, False, False),
    (128, 256, "f32", BF, True, True), (80, 32, "bf16", F32, False, True),
])
def test_append(csa, lens, pos, D, ps, kind, dt, il, norm):
    cu, qp, n, toks = batch(lens, pos, pad=1)
    rng = np.random.default_rng(D + ps)
    tab, total = make_pages(rng, [p + k for p, k in zip(pos, lens)], ps)
    rows = torch.randn(n, D + 16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(ps)).to(dt)[:, :D]
    if kind == "e4m3" and not norm:
        rows = rows.clone()
        rows[0] = 0
    gain = torch.rand(D, device="cuda") + 0.5
    w, ms = csa.csa_rope_freqs(64, factor=2.0, original_len=512)
    t = torch.from_numpy(tab).cuda()
    fill = 3
    if kind == "e4m3":
        pages = torch.full((total, ps, D - 64), fill, dtype=torch.uint8, device="cuda")
        pr = torch.full((total, ps, 64), fill, dtype=BF, device="cuda")
        sc = torch.full((total, ps), float(fill), device="cuda")
    else:
        pages, pr, sc = torch.full((total, ps, D), fill, dtype=BF if kind == "bf16" else F32, device="cuda"), None, None
    csa.csa_paged_append(rows, cu, qp, t, pages, w, pages_rope=pr, pages_scale=sc, norm=norm, gain=gain if norm else None,
                         interleaved=il, mscale=ms)
    csa.check_device_error()
    X, w64 = np64(rows), w.cpu().numpy()
    seen = np.zeros((total, ps), bool)
    for i, b, p in toks:
        u = O.norm_row(X[i], np64(gain)) if norm else X[i]
        v = O.rotate_row(u, p, w64, interleaved=il, mscale=ms)
        at = tab[b, p // ps], p % ps
        seen[at] = True
        big = np.abs(u).max() * 2 * ms
        if kind != "e4m3":
            close_rows(np64(pages[at]), v, pages.dtype, big, (i, b, p))
            continue
        s = np.abs(v[:-64]).max() / 448 or 1.0
        assert abs(float(sc[at]) - s) <= s * SLOP
        deq = O.e4m3_decode(pages[at].cpu().numpy()) * float(sc[at])
        # half a step of e4m3: 2^-4 of the value, 2^-10 scales below the normal range
        assert np.all(np.abs(deq - v[:-64]) <= np.maximum(2.0 ** -4 * np.abs(v[:-64]), s * 2.0 ** -10) + SLOP * big)
        close_rows(np64(pr[at]), v[-64:], BF, big, (i, b, p))
    other = ~torch.from_numpy(seen).cuda()
    assert bool((pages[other] == fill).all())
    if kind == "e4m3":
        assert bool((pr[other] == fill).all()) and bool((sc[other] == fill).all())


def test_append_without_a_page_is_recorded_and_skipped(csa):
    cu, qp, n, _ = batch([2, 2, 2], [0, 15, -1])
    pages = torch.zeros(3, 16, 128, dtype=BF, device="cuda")
    tab = torch.tensor([[9], [1], [2]], dtype=torch.int32, device="cuda")    # page 9: none; row 16: behind the table
    rows = torch.ones(n, 128, dtype=BF, device="cuda")
    csa.csa_paged_append(rows, cu, qp, tab, pages, None, norm=False)
    with pytest.raises(csa.CsaError, match="page"):
        csa.check_device_error()
    csa.check_device_error()
    want = torch.zeros_like(pages)
    want[1, 15] = 1
    want[2, 0] = 1                                                           # position -1 is left alone
    assert torch.equal(pages, want)


# ---------------------------------------------------------------- attention

class Case:
    """A batch over caches whose unneeded rows and pages hold NaN."""

    def __init__(self, lens, pos, H, D, *, ps=64, W=128, m=0, kind="bf16", sink=True, seed=0, pad=0, eps=None):
        self.W, self.m, self.D, self.H = W, m, D, H
        rng = np.random.default_rng(seed)
        self.cu, self.qp, self.n, self.toks = batch(lens, pos, pad)
        last = [p + k if k else 0 for p, k in zip(pos, lens)]
        bf = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).to(BF)  # noqa: E731
        self.q = (bf(self.n, H, D) * 1.5).cuda()
        self.sink = torch.from_numpy(rng.standard_normal(H, dtype=np.float32)).cuda() if sink else None
        self.kw = dict(W=W, sink=self.sink)
        if W is not None:
            tab, total = make_pages(rng, last, ps)
            pages = torch.full((total, ps, D), math.nan, dtype=BF)
            for b, (p, k) in enumerate(zip(pos, lens)):
                lo = 0 if W == 0 else max(0, p - W + 1)
                for u in range(lo, p + k):
                    pages[tab[b, u // ps], u % ps] = bf(D)
                tab[b, :lo // ps] = -1                        # pages before the window were given back
            self.tab, self.pages = tab, pages
            self.kw.update(tok_pages=pages.cuda(), tok_table=torch.from_numpy(tab).cuda())
        else:
            self.kw["W"] = 0
        if m:
            tab, total = make_pages(rng, [e // m for e in last], ps)
            if kind == "bf16":
                st = (torch.full((total, ps, D), math.nan, dtype=BF),)
            else:
                st = (torch.full((total, ps, D - 64), 0x7f, dtype=torch.uint8), torch.full((total, ps, 64), math.nan, dtype=BF),
                      torch.full((total, ps), math.nan))
            for b, e in enumerate(last):
                for u in range(e // m):
                    at = tab[b, u // ps], u % ps
                    if kind == "bf16":
                        st[0][at] = bf(D)
                    else:
                        st[0][at] = bf(D - 64).float().mul(64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                        st[1][at] = bf(64)
                        st[2][at] = float(rng.uniform(0.01, 0.02))
            self.ktab, self.store, self.kind = tab, st, kind
            self.kw.update(kv_pages=st[0].cuda(), kv_table=torch.from_numpy(tab).cuda(), m=m)
            if kind == "e4m3":
                self.kw.update(kv_rope=st[1].cuda(), kv_scale=st[2].cuda())

    def rows(self, b, p):
        got = []
        if self.W is not None:
            lo = 0 if self.W == 0 else max(0, p - self.W + 1)
            got.append(O.page_rows(np64(self.pages), self.tab[b], lo, p + 1))
        if self.m:
            ne = (p + 1) // self.m
            if self.kind == "bf16":
                got.append(O.page_rows(np64(self.store[0]), self.ktab[b], 0, ne))
            else:
                got.append(O.e4m3_page_rows(self.store[0].numpy(), np64(self.store[1]), self.store[2].numpy(), self.ktab[b], 0, ne))
        return np.concatenate(got)

    def check(self, out, only=None):
        got, q = np64(out), np64(self.q)
        sink = None if self.sink is None else np64(self.sink)
        for i, b, p in self.toks if only is None else [self.toks[k] for k in only]:
            ref, mag = O.paged_attention_row(q[i], self.rows(b, p), 1 / math.sqrt(self.D), sink)
            tol = (2.0 ** -8 + 2.0 ** -9) * mag + half(out.dtype) * np.abs(ref)
            bad = ~(np.abs(got[i] - ref) <= tol)
            assert not bad.any(), f"token {i} (sequence {b}, position {p}): {int(bad.sum())} off, worst {np.abs(got[i] - ref).max():.3e}"


ATTN = [
    # decode and drafts: few tokens, split rows
    dict(lens=[1], pos=[0], H=64, D=512),
    dict(lens=[1], pos=[1000], H=64, D=512, W=0),
    dict(lens=[1], pos=[5000], H=3, D=128, W=0, ps=16),
    dict(lens=[1, 1, 1, 1], pos=[63, 64, 65, 700], H=8, D=128, W=0),
    dict(lens=[1, 0, 1], pos=[4095, 0, 127], H=64, D=512, m=128, kind="e4m3"),
    dict(lens=[1, 1], pos=[20000, 300], H=16, D=512, m=64, kind="e4m3", ps=16),
    dict(lens=[3, 5, 0, 1], pos=[250, 0, 0, 900], H=64, D=512, m=4, kind="bf16", W=100),
    dict(lens=[9, 2], pos=[10, 400], H=8, D=128, W=0, ps=1, sink=False),
    dict(lens=[2, 2], pos=[126, 511], H=64, D=512, m=128, W=None, sink=False),       # first entry at position 127
    dict(lens=[2, 2], pos=[126, 511], H=5, D=128, m=128, W=None, kind="e4m3", ps=32),
    dict(lens=[1] * 40, pos=[i * 37 for i in range(40)], H=4, D=128, W=1),
    dict(lens=[0] * 600 + [1, 2], pos=[5] * 600 + [700, 90], H=8, D=128, W=0),
    dict(lens=[0] * 250 + [1, 2] + [0] * 100, pos=[5] * 250 + [700, 90] + [9] * 100, H=64, D=512, W=0),
    # chunks: more tokens than ranges
    dict(lens=[70, 1, 0, 33], pos=[0, 500, 0, 131], H=64, D=512),
    dict(lens=[100], pos=[60], H=64, D=512, W=0),
    dict(lens=[50, 61], pos=[0, 190], H=64, D=512, W=0, ps=128, sink=False),
    dict(lens=[40, 77], pos=[1000, 250], H=64, D=512, m=16, W=64, ps=64),
    dict(lens=[40, 77], pos=[1000, 250], H=64, D=512, m=16, W=64, ps=32),
    dict(lens=[90, 10], pos=[600, 7], H=64, D=512, m=4, kind="e4m3", ps=64),
    dict(lens=[130], pos=[300], H=8, D=128, W=0, ps=64),
    dict(lens=[80], pos=[125], H=24, D=512, m=128, W=None),
    dict(lens=[33, 99], pos=[64, 1], H=7, D=512, W=0, ps=256),
]


@pytest.mark.parametrize("k", range(len(ATTN)))
def test_attention(csa, k):
    c = Case(seed=k, pad=k % 3, **ATTN[k])
    out = torch.full_like(c.q, 9.0)
    csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, **c.kw)
    csa.check_device_error()
    c.check(out)
    if k % 3:
        assert bool((out[c.n - k % 3:] == 9.0).all())
    f = csa.csa_paged_attention(c.q, c.cu, c.qp, out_dtype=F32, **c.kw)
    m = c.n - k % 3
    assert torch.equal(f[:m].to(BF), out[:m])            # the same numbers, rounded
    again = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    assert torch.equal(again[:m], out[:m])


LONG = [
    dict(lens=[81, 30], pos=[1500, 700], H=64, D=512, W=0),
    dict(lens=[90], pos=[1900], H=64, D=512, W=0, ps=16),
    dict(lens=[77, 1, 40], pos=[0, 3000, 1023], H=64, D=512, W=0, ps=32, sink=False),
    dict(lens=[100], pos=[2000], H=64, D=512, m=2, W=300, ps=128),
    dict(lens=[128], pos=[960], H=64, D=512, m=1, W=None, ps=64, sink=False),
    dict(lens=[95], pos=[1200], H=16, D=512, W=0),
    dict(lens=[120, 9], pos=[700, 900], H=33, D=512, m=4, W=511, ps=64),
    dict(lens=[200], pos=[500], H=1, D=512, W=0, ps=64),
    dict(lens=[100], pos=[800], H=64, D=128, W=0),
    dict(lens=[99], pos=[4000], H=64, D=512, m=4, W=128, kind="e4m3"),
    dict(lens=[2] * 60, pos=[37 * i for i in range(60)], H=64, D=512, W=0),
]


@pytest.mark.parametrize("k", range(len(LONG)))
def test_attention_of_long_rows(csa, k):
    """Chunks whose rows fill many tiles: first, last and odd tokens of every sequence."""
    c = Case(seed=100 + k, pad=1, **LONG[k])
    out = torch.full_like(c.q, 9.0)
    csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, **c.kw)
    csa.check_device_error()
    ends = {i for i in range(len(c.toks)) if i + 1 == len(c.toks) or c.toks[i][1] != c.toks[i + 1][1] or
            i == 0 or c.toks[i][1] != c.toks[i - 1][1]}
    c.check(out, only=sorted(ends | set(range(0, len(c.toks), 17)))[:24])
    assert bool((out[-1] == 9.0).all()) and not bool(torch.isnan(out).any())
    assert torch.equal(csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)[:-1], out[:-1])


@pytest.mark.parametrize("lens,pos,H,D", [([1, 2], [2000, 700], 64, 512), ([90], [1500], 16, 512), ([3], [900], 8, 128)])
def test_e4m3_rows_as_stored(csa, lens, pos, H, D):
    """Against the stored rows themselves.  The attention rounds their last 64 dims once more, relative to the
    row's scale: by half(bf16) of each element, so a logit moves by at most e = half * scale * sum |q||r| over
    those dims, every weight by a factor within exp(+-2 e), and the result by (half + 2 e) sum p |row|."""
    c = Case(lens=lens, pos=pos, H=H, D=D, m=4, kind="e4m3", W=None, seed=9)
    out = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    csa.check_device_error()
    codes = c.store[0].view(torch.float8_e4m3fn).double().numpy()
    for i, b, p in c.toks[:3] + c.toks[-1:]:
        ne = (p + 1) // 4
        rows = np.concatenate([O.page_rows(codes, c.ktab[b], 0, ne) * O.page_rows(np64(c.store[2]), c.ktab[b], 0, ne)[:, None],
                               O.page_rows(np64(c.store[1]), c.ktab[b], 0, ne)], -1)
        q = np64(c.q[i])
        ref, mag = O.paged_attention_row(q, rows, 1 / math.sqrt(D), np64(c.sink))
        e = half(BF) / math.sqrt(D) * (np.abs(q[:, -64:]) @ np.abs(rows[:, -64:]).T).max(-1, keepdims=True)
        tol = (2.0 ** -8 + 2.0 ** -9 + half(BF) + 2.02 * e) * mag + half(BF) * np.abs(ref)
        assert np.all(np.abs(np64(out[i]) - ref) <= tol), (i, np.abs(np64(out[i]) - ref).max())


@pytest.mark.parametrize("H,D,dims", [(64, 512, (0, 127, 128, 300, 384, 447)), (8, 128, (0, 37, 63))])
def test_nan_codes_reach_the_tokens_that_see_them(csa, H, D, dims):
    """A NaN code in any piece of an e4m3 row, and a NaN or an infinite scale."""
    c = Case(lens=[40], pos=[360], H=H, D=D, m=4, kind="e4m3", W=None)
    clean = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    for row in (91, 95):                                      # complete at positions 367 and 383
        first = 4 * row + 3 - 360
        for d in dims + ("nan", "inf"):
            codes, scale = c.kw["kv_pages"].clone(), c.kw["kv_scale"].clone()
            at = int(c.ktab[0, row // 64]), row % 64
            if isinstance(d, str):
                scale[at] = float(d)
            else:
                codes[at][d] = 0xff if d % 2 else 0x7f
            out = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, kv_pages=codes, kv_scale=scale))
            assert torch.equal(out[:first], clean[:first]), (row, d)
            assert bool(torch.isnan(out[first:]).any(-1).all()), (row, d)
    csa.check_device_error()


def test_tokens_at_negative_positions_are_left_alone(csa):
    for lens, H, D in (([4], 64, 512), ([90], 64, 512), ([90], 8, 128)):
        c = Case(lens=lens, pos=[0], H=H, D=D, W=0)
        out = torch.full_like(c.q, 3.0)
        csa.csa_paged_attention(c.q, c.cu, torch.tensor([-2], device="cuda"), out=out, **c.kw)
        csa.check_device_error()
        assert bool((out[:2] == 3.0).all())
        ref = csa.csa_paged_attention(c.q[2:].contiguous(), torch.tensor([0, lens[0] - 2], dtype=torch.int32, device="cuda"),
                                      torch.tensor([0], device="cuda"), **c.kw)
        tol = 2.0 ** -6 * ref.float().abs().max()               # another split of the rows: other roundings of P
        assert bool(((out[2:].float() - ref.float()).abs() <= tol).all())


@pytest.mark.parametrize("n,H,D,W", [(10, 64, 512, 0), (90, 64, 512, 0), (90, 8, 128, 128)])
def test_batch_that_ends_inside_a_sequence(csa, n, H, D, W):
    """cu_q names more rows than the tensors have: those below n_tok are worked on, none behind them."""
    c = Case(lens=[n // 2, n], pos=[100, 40], H=H, D=D, W=W)
    m = n
    room = torch.full((c.n, H, D), 9.0, dtype=BF, device="cuda")
    csa.csa_paged_attention(c.q[:m], c.cu, c.qp, out=room[:m], **c.kw)
    w, _ = csa.csa_rope_freqs(64)
    turned = torch.full_like(room, 9.0)
    csa.csa_rope(c.q[:m], c.cu, c.qp, w, out=turned[:m])
    csa.check_device_error()
    c.check(room, only=[0, n // 2 - 1, n // 2, m - 1])
    assert torch.equal(turned[:m], csa.csa_rope(c.q, c.cu, c.qp, w)[:m])
    assert bool((room[m:] == 9.0).all()) and bool((turned[m:] == 9.0).all())


def test_rows_out_of_sight_do_not_matter(csa):
    """A later token's NaN row reaches that token and those after it only, in decode-sized and chunk-sized batches."""
    for lens, H, D in (([12], 64, 512), ([110], 64, 512), ([110], 8, 128)):
        c = Case(lens=lens, pos=[90], H=H, D=D, W=0)
        clean = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
        for bad in (math.nan, math.inf):
            p = 95
            pages = c.kw["tok_pages"].clone()
            pages[c.tab[0, p // 64], p % 64] = bad
            out = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, tok_pages=pages))
            assert torch.equal(out[:5], clean[:5])
            assert bool(torch.isnan(out[5:]).any(-1).all())
        csa.check_device_error()


def test_sink_alone_and_nothing(csa):
    """No visible row: zeros, with a sink and without; a sink of -inf takes no part."""
    c = Case(lens=[3], pos=[5], H=8, D=128, m=128, W=None)
    assert not csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw).any()
    assert not csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, sink=None)).any()
    for n in (3, 100):
        c = Case(lens=[n], pos=[700], H=8, D=128, W=50)
        none = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, sink=None))
        off = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, sink=torch.full((8,), -math.inf, device="cuda")))
        assert torch.equal(none, off)
        full = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, sink=torch.full((8,), 3e38, device="cuda")))
        assert not full.any()


def test_large_logits_and_scale(csa):
    """Logits that grow along the rows (the running maximum moves) and reach hundreds."""
    for n in (4, 90):
        c = Case(lens=[n], pos=[900], H=16, D=512, W=0, sink=False)
        ramp = torch.linspace(0.2, 4.0, 1024)
        for u in range(900 + n):
            c.pages[c.tab[0, u // 64], u % 64] *= ramp[u]
        out = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, tok_pages=c.pages.cuda()))
        c.check(out, only=[0, n // 2, n - 1])


def test_missing_page_of_a_visible_row_is_recorded(csa):
    c = Case(lens=[2], pos=[200], H=8, D=128, W=0)
    tab = c.kw["tok_table"].clone()
    tab[0, 1] = c.pages.shape[0]
    csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, tok_table=tab))
    with pytest.raises(csa.CsaError, match="page"):
        csa.check_device_error()


def test_rows_behind_the_table_are_not_visible(csa):
    c = Case(lens=[1], pos=[100], H=8, D=128, W=0)
    short = csa.csa_paged_attention(c.q, c.cu, torch.tensor([1000], device="cuda"), **dict(c.kw, tok_table=c.kw["tok_table"][:, :1].contiguous()))
    ref = csa.csa_paged_attention(c.q, c.cu, torch.tensor([63], device="cuda"), **c.kw)
    csa.check_device_error()
    assert torch.equal(short, ref)


@pytest.mark.parametrize("lens,pos,H,D,W,cut", [([20], [250], 64, 512, 128, 256), ([20], [250], 8, 128, 128, 256),
                                                 ([20, 1], [200, 400], 64, 512, 0, 192), ([100], [1000], 64, 512, 600, 1024),
                                                 ([100], [1000], 64, 512, 800, 1024),
                                                 ([100], [250], 8, 128, 128, 256)])
def test_tokens_behind_the_table(csa, lens, pos, H, D, W, cut):
    """A window that reaches over the table's end shrinks from token to token."""
    c = Case(lens=lens, pos=pos, H=H, D=D, W=W)
    out = csa.csa_paged_attention(c.q, c.cu, c.qp, **dict(c.kw, tok_table=c.kw["tok_table"][:, :cut // 64].contiguous()))
    csa.check_device_error()
    for i, b, p in c.toks[::3]:
        rows = O.page_rows(np64(c.pages), c.tab[b], 0 if W == 0 else max(0, p - W + 1), min(p + 1, cut))
        ref, mag = O.paged_attention_row(np64(c.q[i]), rows, 1 / math.sqrt(D), np64(c.sink))
        assert np.all(np.abs(np64(out[i]) - ref) <= (2.0 ** -8 + 2.0 ** -9) * mag + half(BF) * np.abs(ref)), (i, p)


def test_offsets_beyond_32_bits(csa):
    """Pages behind 2^32 elements of a large cache."""
    ps, D, n_pages = 64, 512, 140000                          # 9.2 GB, 4.6e9 elements
    pages = torch.empty(n_pages, ps, D, dtype=BF, device="cuda")
    cu, qp, n, toks = batch([3], [70])
    tab = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device="cuda")
    rows = torch.randn(73, D, device="cuda").to(BF)
    cu0, qp0, _, _ = batch([73], [0])
    csa.csa_paged_append(rows, cu0, qp0, tab, pages, None, norm=False)
    q = torch.randn(n, 64, D, device="cuda").to(BF)
    out = csa.csa_paged_attention(q, cu, qp, tok_pages=pages, tok_table=tab, W=0)
    big = torch.cat([pages[n_pages - 1], pages[n_pages - 3]])[:73]
    assert torch.equal(big, rows)
    small = torch.stack([pages[n_pages - 1], pages[n_pages - 3]])
    ref = csa.csa_paged_attention(q, cu, qp, tok_pages=small, tok_table=torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), W=0)
    csa.check_device_error()
    assert torch.equal(out, ref)


# ---------------------------------------------------------------- streams, graphs, refusals

def test_another_stream(csa):
    c = Case(lens=[3, 2], pos=[300, 64], H=64, D=512)
    ref = csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = csa.csa_paged_attention(c.q, c.cu, c.qp, stream=s, **c.kw)
    w, _ = csa.csa_rope_freqs(64)
    s.wait_stream(torch.cuda.current_stream())
    turned = csa.csa_rope(out, c.cu, c.qp, w, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(turned, csa.csa_rope(ref, c.cu, c.qp, w))


def test_two_graphs_replayed_with_new_positions(csa):
    """Captured calls keep workspaces of their own and read positions and tables at replay."""
    cases = [Case(lens=[1, 1], pos=[500, 200], H=64, D=512, W=0, seed=s) for s in (1, 2)]
    graphs, outs = [], []
    for c in cases:
        csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw))
        graphs.append(g)
    for shift in (0, -150):
        for c in cases:
            c.qp += shift
        for g in graphs:
            g.replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            assert torch.equal(out, csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw))
    csa.check_device_error()


@pytest.mark.parametrize("kw", [dict(lens=[90, 60], pos=[700, 1500], H=64, D=512, W=0), dict(lens=[1, 2, 1], pos=[900, 40, 2000], H=64, D=512, W=0),
                                dict(lens=[90, 1], pos=[600, 7], H=64, D=512, m=4, kind="e4m3"), dict(lens=[200], pos=[300], H=8, D=128)])
def test_two_calls_at_once(csa, kw):
    """Calls on two streams, back to back and overlapping, and a captured one replayed between them."""
    cs = [Case(seed=s, **kw) for s in (1, 2)]
    ref = [csa.csa_paged_attention(c.q, c.cu, c.qp, **c.kw) for c in cs]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        caught = csa.csa_paged_attention(cs[0].q, cs[0].cu, cs[0].qp, **cs[0].kw)
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(8):
        for i, (c, st) in enumerate(zip(cs, streams)):
            got[i].append(csa.csa_paged_attention(c.q, c.cu, c.qp, stream=st, **c.kw))
        g.replay()
    torch.cuda.synchronize()
    csa.check_device_error()
    assert torch.equal(caught, ref[0])
    assert all(torch.equal(o, ref[i]) for i in (0, 1) for o in got[i])


def test_a_step_captured_as_one_graph(csa):
    """The layer step in a graph, replayed as positions advance, equals the calls one by one."""
    D, H, ps = 512, 64, 64
    w, _ = csa.csa_rope_freqs(64)
    g0 = torch.Generator(device="cuda").manual_seed(3)
    tab = torch.arange(12, dtype=torch.int32, device="cuda").reshape(2, 6)
    start = torch.randn(12, ps, D, generator=g0, device="cuda").to(BF)
    cu, qp, n, _ = batch([1, 1], [100, 250])
    q, rows = torch.empty(n, H, D, dtype=BF, device="cuda"), torch.empty(n, D, dtype=BF, device="cuda")
    inputs = [(torch.randn(n, H, D, generator=g0, device="cuda").to(BF), torch.randn(n, D, generator=g0, device="cuda").to(BF)) for _ in range(4)]
    pages = start.clone()
    want = []
    for k, (a, b) in enumerate(inputs):
        want.append(csa.paged_layer_step(a, b, cu, qp + k, w, pages, tab, W=0))
    held, pos = start.clone(), qp.clone()
    q.copy_(inputs[0][0])
    rows.copy_(inputs[0][1])
    csa.paged_layer_step(q, rows, cu, pos, w, held.clone(), tab, W=0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = csa.paged_layer_step(q, rows, cu, pos, w, held, tab, W=0)
    for k, (a, b) in enumerate(inputs):
        q.copy_(a)
        rows.copy_(b)
        pos.copy_(qp + k)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k]), k
    csa.check_device_error()
    assert torch.equal(held, pages)


def test_binding_refusals(csa):
    c = Case(lens=[2], pos=[10], H=8, D=128)
    x, w = c.q, csa.csa_rope_freqs(64)[0]
    bad = [
        (lambda: csa.csa_rope(x, c.cu.long(), c.qp, w), "int32"), (lambda: csa.csa_rope(x, c.cu, c.qp[:0], w), "cu_q"),
        (lambda: csa.csa_rope(x, c.cu, c.qp, w.float()), "inv_freq"), (lambda: csa.csa_rope(x.half(), c.cu, c.qp, w), "float32 or bfloat16"),
        (lambda: csa.csa_rope(x, c.cu, c.qp, w, out_dtype=torch.float16), "float32 or bfloat16"),
        (lambda: csa.csa_rope(x.transpose(1, 2), c.cu, c.qp, w), "last dimension"), (lambda: csa.csa_rope(x[..., :120], c.cu, c.qp, w), "multiple of 16"),
        (lambda: csa.csa_rope(x[:, 1:], c.cu, c.qp, w, out=x[:, :-1]), "overlap"), (lambda: csa.csa_rope(x, c.cu, c.qp, w, out=x[:1]), "shape"),
        (lambda: csa.csa_rope(x, c.cu, c.qp, w, out=x[:, :1].expand_as(x)), "overlap"),
        (lambda: csa.csa_qk_norm_rope(x, x[..., :64], c.cu, c.qp, w), "one dtype"), (lambda: csa.csa_qk_norm_rope(x, None, c.cu, c.qp, w, q_gain=torch.ones(64, device="cuda")), "q_gain"),
        (lambda: csa.csa_qk_norm_rope(x, x.clone(), c.cu, c.qp, w, q_out=x, k_out=x), "overlap"),
        (lambda: csa.csa_paged_append(x[:, 0], c.cu, c.qp, c.kw["tok_table"], c.kw["tok_pages"][..., :64].contiguous(), w), "pages"),
        (lambda: csa.csa_paged_append(x[:, 0], c.cu, c.qp, c.kw["tok_table"].long(), c.kw["tok_pages"], w), "block_table"),
        (lambda: csa.csa_paged_append(x[:, 0], c.cu, c.qp, c.kw["tok_table"], torch.zeros(4, 48, 128, device="cuda"), w), "power of two"),
        (lambda: csa.csa_paged_attention(x.float(), c.cu, c.qp, **c.kw), "bfloat16"),
        (lambda: csa.csa_paged_attention(x, c.cu, c.qp, **dict(c.kw, sink=c.sink[:3])), "sink"),
        (lambda: csa.csa_paged_attention(x, c.cu, c.qp, **dict(c.kw, tok_table=None)), "tok_table"),
        (lambda: csa.csa_paged_attention(x, c.cu, c.qp, **dict(c.kw, tok_pages=c.kw["tok_pages"].float())), "tok_pages"),
        (lambda: csa.csa_paged_attention(x, c.cu, c.qp, **dict(c.kw, workspace=torch.empty(16, device="cuda"))), "workspace"),
        (lambda: csa.csa_paged_attention(x, c.cu, c.qp, out=x, **c.kw), "overlaps"),
        (lambda: csa.csa_paged_attention(x, c.cu, c.qp), "required"),
    ]
    for call, text in bad:
        with pytest.raises(csa.CsaError, match=text):
            call()
    csa.check_device_error()


def test_empty_batches(csa):
    w = csa.csa_rope_freqs(64)[0]
    cu, qp = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    x = torch.ones(0, 8, 128, dtype=BF, device="cuda")
    assert csa.csa_rope(x, cu, qp, w).shape == x.shape
    c = Case(lens=[0, 0], pos=[10, 0], H=8, D=128, pad=2)
    out = torch.full_like(c.q, 4.0)
    csa.csa_paged_attention(c.q, c.cu, c.qp, out=out, tok_pages=torch.zeros(2, 64, 128, dtype=BF, device="cuda"),
                            tok_table=torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    csa.check_device_error()
    assert bool((out == 4.0).all())


# ---------------------------------------------------------------- a run of them together

@pytest.mark.parametrize("H,D,W,m,il", [(64, 512, 128, 0, False), (8, 128, 0, 0, True), (64, 512, 32, 16, True)])
def test_serving_run(csa, H, D, W, m, il):
    """Prompts in chunks and decode tokens over several steps, against the definition over the sequence's whole rows."""
    rng = np.random.default_rng(H + D)
    steps = [([40, 90, 0], [0, 0, 0]), ([1, 7, 3], [40, 90, 0]), ([1, 1, 1], [41, 97, 3]), ([60, 1, 80], [42, 98, 4])]
    ps, S = 16, 128
    raw = torch.from_numpy(rng.standard_normal((3, S, D), dtype=np.float32)).to(BF)
    w, ms = csa.csa_rope_freqs(64, factor=2.0, original_len=64)
    gain, qg = torch.rand(D) + 0.5, torch.rand(D) + 0.5
    sink = torch.randn(H)
    tab = torch.from_numpy(rng.permutation(3 * S // ps).astype(np.int32).reshape(3, -1)).cuda()
    pages = torch.zeros(3 * S // ps, ps, D, dtype=BF, device="cuda")
    ent = torch.from_numpy(rng.standard_normal((3 * 16, 16, D), dtype=np.float32)).to(BF)
    etab = torch.arange(48, dtype=torch.int32).reshape(3, 16)
    kw = dict(kv_pages=ent.cuda(), kv_table=etab.cuda(), m=m) if m else {}
    w64 = w.cpu().numpy()
    tok_ref = np.zeros((3, S, D))
    for lens, pos in steps:
        cu, qp, n, toks = batch(lens, pos)
        q = torch.from_numpy(rng.standard_normal((n, H, D), dtype=np.float32)).to(BF).cuda()
        rows = torch.stack([raw[b, p] for _, b, p in toks]).cuda()
        out = csa.paged_layer_step(q, rows, cu, qp, w, pages, tab, W=W, sink=sink.cuda(), q_gain=qg.cuda(), gain=gain.cuda(),
                                   interleaved=il, mscale=ms, **kw)
        csa.check_device_error()
        for _, b, p in toks:
            tok_ref[b, p] = np64(pages[tab[b, p // ps], p % ps])          # as stored: checked by the append's own test
            close_rows(tok_ref[b, p], O.rotate_row(O.norm_row(np64(raw[b, p]), np64(gain)), p, w64, interleaved=il, mscale=ms), BF, 12.0, (b, p))
        for i, b, p in toks[::3]:
            qn = O.bf16_round(O.rotate_row(O.norm_row(np64(q[i]), np64(qg)), p, w64, interleaved=il, mscale=ms).astype(np.float32))
            seen = [tok_ref[b, max(0, p - W + 1) if W else 0:p + 1]]
            if m:
                seen.append(O.page_rows(np64(ent), etab[b].numpy(), 0, (p + 1) // m))
            ref, mag = O.paged_attention_row(qn, np.concatenate(seen), 1 / math.sqrt(D), np64(sink))
            ref = O.rotate_row(ref, p, w64, interleaved=il, inverse=True, mscale=1 / ms)
            # the output is rounded before and after it is turned back, and a query may round to the
            # other neighbour: one more step of bf16 on each logit (|q||row| / sqrt(D) below 16 after
            # the gains, of which one element in 2^8 moves by 2^-8: below 2^-10)
            tol = (2.0 ** -8 + 2.0 ** -8) * (mag.max(-1, keepdims=True) * 2) + 2.0 ** -8 * np.abs(ref)
            assert np.all(np.abs(np64(out[i]) - ref) <= tol), (b, p, np.abs(np64(out[i]) - ref).max())
