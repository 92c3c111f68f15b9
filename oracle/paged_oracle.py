"""Float64 definitions of the paged serving step: a ragged batch of decode
tokens and prompt chunks over caches kept in pages.  Plain loops in numpy."""
from __future__ import annotations

import math

import numpy as np

from .csa_oracle import bf16_round, e4m3_decode

__all__ = ["rope_freqs", "batch_tokens", "rotate_row", "norm_row", "page_rows", "paged_attention_row"]


def rope_freqs(r, base=10000.0, factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """(frequencies [r / 2], magnitude): linear (original_len 0) or by-parts scaling."""
    out = []
    for j in range(r // 2):
        w = base ** (-2.0 * j / r)
        keep = 0.0
        if original_len > 0:
            turns = original_len * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
        out.append(keep * w + (1 - keep) * w / factor)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if original_len > 0 else 1.0)


def batch_tokens(cu_q, q_pos):
    """[(batch row, sequence, position)] of the batch's tokens."""
    return [(i, b, int(q_pos[b]) + i - cu_q[b]) for b in range(len(q_pos)) for i in range(cu_q[b], cu_q[b + 1])]


def rotate_row(v, pos, inv_freq, *, start=None, interleaved=False, inverse=False, mscale=1.0):
    """v [..., D] float64 with the part [start, start + 2 len(inv_freq)) turned by pos * inv_freq."""
    v = np.array(v, np.float64)
    n = len(inv_freq)
    start = v.shape[-1] - 2 * n if start is None else start
    for j in range(n):
        a, b = (start + 2 * j, start + 2 * j + 1) if interleaved else (start + j, start + j + n)
        f = (-pos if inverse else pos) * inv_freq[j]
        x, y = v[..., a].copy(), v[..., b].copy()
        v[..., a] = (x * math.cos(f) - y * math.sin(f)) * mscale
        v[..., b] = (x * math.sin(f) + y * math.cos(f)) * mscale
    return v


def norm_row(v, gain=None, eps=1e-6):
    v = np.asarray(v, np.float64)
    v = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v if gain is None else v * np.asarray(gain, np.float64)


def page_rows(store, table_row, lo, hi):
    """Rows lo .. hi - 1 of a sequence: store [n_pages, page_size, ...]."""
    ps = store.shape[1]
    return np.stack([store[table_row[p // ps], p % ps] for p in range(lo, hi)]) if hi > lo else store[0, :0]


def e4m3_page_rows(codes, rope, scale, table_row, lo, hi):
    """The rows as the attention reads them: codes * scale, and the RoPE part
    divided by the scale, rounded to bf16 and multiplied by it again.  A scale
    below 2^-100 (of a row that was zeroed and never written, say) counts as that."""
    c = e4m3_decode(page_rows(codes, table_row, lo, hi))
    s = page_rows(scale, table_row, lo, hi).astype(np.float32)[:, None]
    s = np.where(np.abs(s) < 2.0 ** -100, np.float32(2.0 ** -100), s)
    r = page_rows(rope, table_row, lo, hi).astype(np.float32)
    turned = bf16_round(r * (np.float32(1) / s))
    return np.concatenate([c, turned], -1) * s.astype(np.float64)


__all__.append("e4m3_page_rows")


def paged_attention_row(q, rows, scale, sink=None):
    """One token: q [H, D], rows [n, D].  Returns (out [H, D], sum_i p_i |row_i| [H, D])."""
    q = np.asarray(q, np.float64)
    rows = np.asarray(rows, np.float64)
    H, D = q.shape
    out, mag = np.zeros((H, D)), np.zeros((H, D))
    for h in range(H):
        z = scale * (rows @ q[h])
        s = -math.inf if sink is None else float(sink[h])
        top = max(z.max(initial=-math.inf), s)
        if top == -math.inf:
            continue
        e = np.exp(z - top)
        den = e.sum() + math.exp(s - top)
        out[h] = e @ rows / den
        mag[h] = e @ np.abs(rows) / den
    return out, mag
