"""Host side of the paged serving calls, without a GPU: frequencies, refusals
before any launch, workspace arithmetic, and the oracle's own definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
import long_context_compressed_02_b200 as csa


@pytest.fixture(scope="module")
def L():
    from long_context_compressed_02_b200 import build
    build.build()
    return csa.lib()


@pytest.mark.parametrize("r,kw", [(64, {}), (64, dict(factor=4.0)), (128, dict(factor=16.0, original_len=4096)),
                                  (16, dict(factor=1.0, original_len=2048, base=500000.0)),
                                  (64, dict(factor=40.0, original_len=4096, beta_fast=16.0, beta_slow=2.0))])
def test_rope_freqs(L, r, kw):
    w, ms = csa.csa_rope_freqs(r, device="cpu", **kw)
    ref, ref_ms = O.rope_freqs(r, **kw)
    # pow of the two libraries: a few units in the last place of a double
    assert np.allclose(w.numpy(), ref, rtol=1e-14, atol=0) and w.dtype == torch.float64
    assert abs(ms - ref_ms) <= ref_ms * 2 ** -24
    if kw.get("factor", 1.0) == 1.0:
        assert np.allclose(ref, 10000.0 ** (-2.0 * np.arange(r // 2) / r)) or "base" in kw


def test_rope_freqs_by_parts_keeps_fast_and_divides_slow_pairs(L):
    w, _ = csa.csa_rope_freqs(64, factor=8.0, original_len=4096, device="cpu")
    plain, _ = csa.csa_rope_freqs(64, device="cpu")
    ratio = (plain / w).numpy()
    assert ratio[0] == 1.0 and abs(ratio[-1] - 8.0) < 1e-12 and np.all(np.diff(ratio) >= -1e-12)


@pytest.mark.parametrize("kw,text", [(dict(rope_dim=7), "even"), (dict(rope_dim=0), "even"), (dict(factor=0.5), "factor"),
                                     (dict(base=1.0), "base"), (dict(original_len=-1), "original_len"),
                                     (dict(original_len=4096, beta_fast=1.0, beta_slow=1.0), "beta_fast"),
                                     (dict(factor=float("nan")), "factor")])
def test_rope_freqs_refusals(L, kw, text):
    kw = dict(dict(rope_dim=64), **kw)
    with pytest.raises(csa.CsaError, match=text):
        csa.csa_rope_freqs(kw.pop("rope_dim"), device="cpu", **kw)


def test_rotation_definitions_agree():
    """The oracle's half-layout rotation of the last dims is the layer's; the inverse undoes it."""
    rng = np.random.default_rng(0)
    v = rng.standard_normal((3, 128))
    w, _ = O.rope_freqs(64)
    y = O.rotate_row(v, 12345, w)
    assert np.allclose(y, O.rope_partial(v, np.full(3, 12345), 64), atol=1e-9)
    for il in (False, True):
        z = O.rotate_row(v, 77, w, start=8, interleaved=il)
        assert np.allclose(O.rotate_row(z, 77, w, start=8, interleaved=il, inverse=True), v, atol=1e-12)


def test_rotation_gradient_is_its_inverse():
    """d(sum g . rotate(x)) / dx = rotate(g) by the negative angle, against differences."""
    rng = np.random.default_rng(1)
    w, ms = O.rope_freqs(16, factor=4.0, original_len=64)
    x, g = rng.standard_normal(32), rng.standard_normal(32)
    for il in (False, True):
        grad = O.rotate_row(g, 9, w, interleaved=il, inverse=True, mscale=ms)
        for d in range(32):
            e = np.zeros(32)
            e[d] = 1e-6
            f = lambda v: float(g @ O.rotate_row(v, 9, w, interleaved=il, mscale=ms))  # noqa: E731
            assert abs((f(x + e) - f(x - e)) / 2e-6 - grad[d]) < 1e-7


P16 = ctypes.c_void_p(256)


def _rope(L, **kw):
    a = dict(x=P16, dt=1, xt=64 * 512, xh=512, n=4, H=64, D=512, cu=P16, pos=P16, ns=2, w=P16, r=64, r0=448, il=0, inv=0,
             ms=1.0, out=ctypes.c_void_p(1 << 20), odt=1, ot=64 * 512, oh=512)
    a.update(kw)
    return L.csa_rope(*[a[k] for k in ("x", "dt", "xt", "xh", "n", "H", "D", "cu", "pos", "ns", "w", "r", "r0", "il", "inv",
                                       "ms", "out", "odt", "ot", "oh")], None)


@pytest.mark.parametrize("kw,text", [
    (dict(D=100), b"multiple of 16"), (dict(D=4096), b"multiple of 16"), (dict(r=24), b"rope_dim"), (dict(r=1024), b"rope_dim"),
    (dict(r0=452), b"rope_start"), (dict(r0=456), b"rope_start"), (dict(w=None), b"inv_freq"), (dict(dt=2), b"dtypes"),
    (dict(odt=2), b"dtypes"), (dict(x=ctypes.c_void_p(264)), b"aligned"), (dict(out=None), b"non-null"),
    (dict(xh=516), b"strides"), (dict(ot=4), b"strides"), (dict(cu=None), b"cu_q"), (dict(pos=ctypes.c_void_p(4)), b"aligned"),
    (dict(n=-1), b"negative"), (dict(H=-1), b"negative"), (dict(out=P16, ot=512), b"only with"), (dict(out=P16, odt=0), b"only with"),
])
def test_rope_refusals(L, kw, text):
    assert _rope(L, **kw) == 1 and text in L.csa_last_error(), L.csa_last_error()


def test_nothing_to_do_is_no_error(L):
    assert _rope(L, n=0, x=None, out=None, cu=None, pos=None) == 0
    assert _rope(L, H=0) == 0 and _rope(L, ns=0, cu=None, pos=None) == 0
    assert _append(L, n=0) == 0 and _append(L, ns=0) == 0
    assert _attn(L, n=0) == 0 and _attn(L, ns=0) == 0


def _append(L, **kw):
    a = dict(x=P16, dt=1, xt=512, n=4, D=512, cu=P16, pos=P16, ns=2, tab=P16, mp=4, ps=64, np_=16, norm=1, g=None, eps=1e-6,
             w=P16, r=64, il=0, ms=1.0, pages=ctypes.c_void_p(1 << 20), pdt=1, pr=None, sc=None)
    a.update(kw)
    return L.csa_paged_append(*[a[k] for k in ("x", "dt", "xt", "n", "D", "cu", "pos", "ns", "tab", "mp", "ps", "np_", "norm",
                                               "g", "eps", "w", "r", "il", "ms", "pages", "pdt", "pr", "sc")], None)


@pytest.mark.parametrize("kw,text", [
    (dict(ps=48), b"power of two"), (dict(ps=0), b"power of two"), (dict(mp=0), b"positive"), (dict(np_=0), b"positive"),
    (dict(pdt=7), b"page_dtype"), (dict(pdt=2), b"pages_rope"), (dict(pdt=2, r=0, pr=P16, sc=P16), b"rope_dim 64"),
    (dict(pdt=2, D=64, pr=P16, sc=P16), b"rope_dim 64"), (dict(tab=None), b"block_table"), (dict(eps=-1.0), b"eps"),
    (dict(xt=4), b"strides"), (dict(g=ctypes.c_void_p(4)), b"gain"), (dict(pages=ctypes.c_void_p(8)), b"aligned"),
    (dict(pdt=2, pr=ctypes.c_void_p(8), sc=P16), b"aligned"),
])
def test_append_refusals(L, kw, text):
    assert _append(L, **kw) == 1 and text in L.csa_last_error(), L.csa_last_error()


def _attn(L, **kw):
    a = dict(q=P16, n=4, H=64, D=512, cu=P16, pos=P16, ns=2, tp=P16, tt=P16, tmp=4, tn=16, tps=64, W=128, kp=P16, kdt=1, kr=None,
             ks=None, kt=P16, kmp=4, kn=16, kps=64, m=128, sink=None, sc=0.1, ws=P16, wb=1 << 40,
             out=ctypes.c_void_p(1 << 20), odt=1)
    a.update(kw)
    return L.csa_paged_attention(*[a[k] for k in ("q", "n", "H", "D", "cu", "pos", "ns", "tp", "tt", "tmp", "tn", "tps", "W", "kp",
                                                  "kdt", "kr", "ks", "kt", "kmp", "kn", "kps", "m", "sink", "sc", "ws", "wb",
                                                  "out", "odt")], None)


@pytest.mark.parametrize("kw,text", [
    (dict(H=0), b"H must"), (dict(H=65), b"H must"), (dict(D=256), b"D must"), (dict(tp=None, kp=None), b"required"),
    (dict(W=-1), b"W must"), (dict(sc=0.0), b"scale"), (dict(sc=-1.0), b"scale"), (dict(sc=math.nan), b"scale"), (dict(odt=2), b"out_dtype"), (dict(q=ctypes.c_void_p(8)), b"aligned"), (dict(out=None), b"non-null"),
    (dict(cu=None), b"cu_q"), (dict(tt=None), b"table"), (dict(tps=3), b"power of two"), (dict(kps=0), b"power of two"),
    (dict(kt=None), b"table"), (dict(kdt=0), b"kv_dtype"), (dict(kdt=2), b"kv_rope"), (dict(m=0), b"m must"),
    (dict(tmp=0), b"positive"), (dict(kn=0), b"positive"),
])
def test_attention_refusals(L, kw, text):
    assert _attn(L, **kw) == 1 and text in L.csa_last_error(), L.csa_last_error()


def test_attention_refuses_what_its_offsets_cannot_hold(L):
    assert _attn(L, tmp=1 << 25, tps=64) == 2 and b"2^31" in L.csa_last_error()
    assert _attn(L, n=1 << 26) == 2 and b"2^31" in L.csa_last_error()


def test_attention_workspace(L):
    few = L.csa_paged_attention_workspace(4, 2, 64, 512)
    assert few > 0 and few % 256 == 0
    assert L.csa_paged_attention_workspace(100000, 2, 64, 512) == 0
    assert L.csa_paged_attention_workspace(0, 2, 64, 512) == 0
    assert L.csa_paged_attention_workspace(4, 5000, 64, 512) == 0


def test_binding_refuses_host_tensors(L):
    x, cu, pos = torch.zeros(2, 4, 128), torch.tensor([0, 2], dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    w = torch.ones(32, dtype=torch.float64)
    tab = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(csa.CsaError, match="CUDA tensor"):
        csa.csa_rope(x, cu, pos, w)
    with pytest.raises(csa.CsaError, match="CUDA tensor"):
        csa.csa_qk_norm_rope(x, None, cu, pos, w)
    with pytest.raises(csa.CsaError, match="CUDA tensor"):
        csa.csa_paged_append(x[:, 0], cu, pos, tab, torch.zeros(1, 16, 128), w)
    with pytest.raises(csa.CsaError, match="CUDA tensor"):
        csa.csa_paged_attention(x.bfloat16(), cu, pos, tok_pages=torch.zeros(1, 16, 128).bfloat16(), tok_table=tab)


def test_binding_knows_overlapping_rows():
    base = torch.zeros(4, 3, 128)
    assert not csa._shares(base, base) and not csa._shares(base[:, :1], base[:, 1:])
    assert not csa._shares(base[:, 2], base[:, :2]) and not csa._shares(base[:2], base[2:])
    assert csa._shares(base, base[:, 1:]) and csa._shares(base[:, 1:], base) and csa._shares(base[1:], base[:3])
    assert csa._shares(base, base.bfloat16().view(torch.bfloat16)) is False
    assert csa._shares(base, base.view(torch.bfloat16)) and csa._shares(base[..., :64], base[..., 32:96])
    assert not csa._shares(base, torch.zeros(4, 3, 128))
    assert csa._overlap(base, base) and not csa._overlap(base[0], base[1])
    with pytest.raises(csa.CsaError, match="overlap"):
        csa._out_heads("f", "out", torch.zeros(1, 1, 128).expand(4, 3, 128))
    with pytest.raises(csa.CsaError, match="overlap"):
        csa._out_heads("f", "out", torch.zeros(4 * 128).as_strided((3, 128), (64, 1)))
    assert csa._out_heads("f", "out", base.transpose(0, 1)) == (3, 4, 128, 128, 384)


def test_oracle_attention_of_no_rows_is_zero():
    out, mag = O.paged_attention_row(np.ones((2, 8)), np.zeros((0, 8)), 1.0)
    assert not out.any() and not mag.any()
    out, _ = O.paged_attention_row(np.ones((2, 8)), np.ones((1, 8)), 1.0, np.array([8.0, -math.inf]))
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 1.0)


def _pairs(n, n_seq, H, D, W, tok_rows, *, ps=64, kv_rows=0, kv=torch.bfloat16, kv_ps=64):
    m = dict(device="meta")
    q, pos = torch.empty(n, H, D, dtype=torch.bfloat16, **m), torch.empty(n_seq, dtype=torch.int64, **m)
    kw = {}
    if tok_rows:
        kw.update(tok_pages=torch.empty(9, ps, D, dtype=torch.bfloat16, **m), tok_table=torch.empty(n_seq, tok_rows // ps, **m))
    if kv_rows:
        kw.update(kv_pages=torch.empty(9, kv_ps, D, dtype=kv, **m), kv_table=torch.empty(n_seq, kv_rows // kv_ps, **m))
    return csa.csa_paged_attention_pairs(q, pos, W=W, **kw)


def test_which_calls_work_on_pairs(L):
    """Chunks of at least two tokens a sequence on average, and 704 rows a token that window and tables allow,
    fewer with the square of the tokens that a pair holds."""
    assert _pairs(100, 1, 64, 512, 0, 704) and not _pairs(100, 1, 64, 512, 0, 640)
    assert _pairs(100, 50, 64, 512, 0, 704) and not _pairs(100, 51, 64, 512, 0, 704)
    assert not _pairs(74, 1, 64, 512, 0, 4096) and _pairs(75, 1, 64, 512, 0, 4096)       # split over the SMs
    assert not _pairs(100, 1, 64, 128, 0, 4096)
    assert _pairs(100, 1, 64, 512, 704, 1024) and not _pairs(100, 1, 64, 512, 703, 1024)
    assert _pairs(100, 1, 32, 512, 176, 1024) and not _pairs(100, 1, 32, 512, 175, 1024)
    assert _pairs(100, 1, 64, 512, 64, 1024, kv_rows=640) and not _pairs(100, 1, 64, 512, 63, 1024, kv_rows=640)
    assert _pairs(100, 1, 64, 512, 0, 0, kv_rows=704) and not _pairs(100, 1, 64, 512, 0, 704, kv_rows=64, kv=torch.uint8)
    assert not _pairs(100, 1, 64, 512, 0, 4096, ps=8) and not _pairs(100, 1, 64, 512, 0, 4096, kv_rows=64, kv_ps=8)
    assert L.csa_paged_attention_pairs(0, 0, 64, 512, 64, 9, 64, 0, 1, 0, 0, 1) == 0
