"""The paged key/value cache and its attention (fp64 oracle, test use only).

A cache here is a dict of numpy arrays: table int [B, max_pages], kv_len int [B], page, and k and
v as the values the pages stand for, fp64 [n_pages, Hkv, page, d]. Token j of sequence b lives in
page table[b, j // page], slot j % page. A chunk of n tokens ends the sequence: its token i is at
position kv_len - n + i.

An e4m3 token (one head's d values) is e4m3(fl32(x * r)) * s with r = fl32(448 / amax) and
s = fl32(amax / 448), the decisions taken in fp32 as a kernel takes them; amax < 2^-100 gives
r = s = 1, and a token with a value that is not finite is NaN throughout.
"""
from __future__ import annotations

import numpy as np

from .fp8 import round_e4m3


def quantize_tokens(x):
    """(codes as values fp64, scales fp64) of x [..., d], one scale per leading index."""
    x32 = np.asarray(x, dtype=np.float32)
    fin = np.isfinite(x32).all(-1)
    amax = np.abs(np.where(fin[..., None], x32, np.float32(0))).max(-1)
    small = amax < np.float32(2.0 ** -100)
    safe = np.where(small, np.float32(1), amax).astype(np.float32)
    r = np.where(small, np.float32(1), np.float32(448) / safe).astype(np.float32)
    s = np.where(small, np.float32(1), safe / np.float32(448)).astype(np.float32)
    code = round_e4m3((np.where(fin[..., None], x32, np.float32(0)) * r[..., None]).astype(np.float32))
    return code, np.where(fin, s.astype(np.float64), np.nan)


def slots(cache, b, js):
    """(page index, slot) of positions js of sequence b."""
    js = np.asarray(js, dtype=np.int64)
    return np.asarray(cache["table"])[b, js // cache["page"]], js % cache["page"]


def tokens(cache, name, b, js):
    """[Hkv, len(js), d] fp64: the values of positions js of sequence b."""
    pg, sl = slots(cache, b, js)
    return np.moveaxis(cache[name][pg, :, sl], 0, 1)


def append(cache, k, v, n_new):
    """A copy of the cache with a chunk (k, v fp64 [B, Hkv, N, d]) written at each sequence's end."""
    out = dict(cache, k=cache["k"].copy(), v=cache["v"].copy())
    for b in range(k.shape[0]):
        n, kv = int(n_new[b]), int(cache["kv_len"][b])
        pg, sl = slots(cache, b, np.arange(kv - n, kv))
        for name, x in (("k", k), ("v", v)):
            out[name][pg, :, sl] = np.moveaxis(x[b, :, :n], 1, 0)
    return out


def read(cache, B, N, begin=None):
    """(k, v) fp64 [B, Hkv, N, d]: tokens begin .. begin + N - 1, zero past the end."""
    Hkv, d = cache["k"].shape[1], cache["k"].shape[3]
    out = []
    for name in ("k", "v"):
        x = np.zeros((B, Hkv, N, d))
        for b in range(B):
            b0 = 0 if begin is None else int(begin[b])
            m = min(N, int(cache["kv_len"][b]) - b0)
            if m > 0:
                x[b, :, :m] = tokens(cache, name, b, np.arange(b0, b0 + m))
        out.append(x)
    return tuple(out)


def kept(n, kv, causal, window):
    """bool [n, kv]: the keys each row of a chunk of n tokens keeps."""
    pos = kv - n + np.arange(n)[:, None]
    j = np.arange(kv)[None]
    m = np.ones((n, kv), bool)
    if causal:
        m &= j <= pos
        if window > 0:
            m &= j > pos - window
    return m


def attend(cache, q, n_new, causal, window, scale):
    """fp64 [B, H, N, d]; rows past n_new are NaN (not defined), a row without keys is 0."""
    B, H, N, d = q.shape
    Hkv = cache["k"].shape[1]
    o = np.full(q.shape, np.nan)
    for b in range(B):
        n, kv = int(n_new[b]), int(cache["kv_len"][b])
        K, V = (tokens(cache, name, b, np.arange(kv)) for name in ("k", "v"))
        m = kept(n, kv, causal, window)
        for h in range(H):
            hk = h // (H // Hkv)
            z = np.where(m, (q[b, h, :n] @ K[hk].T) * scale, -np.inf)
            top = z.max(-1, keepdims=True, initial=-np.inf)
            e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
            den = e.sum(-1, keepdims=True)
            o[b, h, :n] = (e @ V[hk]) / np.where(den > 0, den, 1.0)
    return o
