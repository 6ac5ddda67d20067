"""Shared helpers of the paged-cache GPU tests: caches with random page orders, garbage in every
slot no token owns, and the error bound of the attention."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged as OPG
from parity_util import bsa


def build(kind, Hkv, page, d, kv, seed, max_pages=None, garbage=float("nan")):
    """(PagedCache, oracle cache) with tokens drawn for kv[b] positions of each sequence, the pages in
    random order; slots and pages that hold no token hold `garbage` (bf16) or 0xFE codes under a NaN
    scale, and table entries past the last page -7."""
    m = bsa()
    B = len(kv)
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in kv]
    max_pages = max(used + [1]) if max_pages is None else max_pages
    n_pages = sum(used) + 2
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((B, max_pages), -7, dtype=torch.int32)
    vals, own, at = {}, torch.zeros((n_pages, page), dtype=torch.bool), 0
    for b in range(B):
        table[b, :used[b]] = perm[at:at + used[b]].int()
        at += used[b]
        for j in range(kv[b]):
            own[table[b, j // page], j % page] = True
    own = own[:, None, :].expand(n_pages, Hkv, page)
    buf = {}
    for name in ("k", "v"):
        x = torch.randn((n_pages, Hkv, page, d), generator=g).bfloat16()
        if kind == m.CACHE_E4M3:
            code, s = OPG.quantize_tokens(x.float().numpy())
            u8 = torch.from_numpy(code).to(torch.float8_e4m3fn).view(torch.uint8)
            sc = torch.from_numpy(s).float()
            vals[name] = code * s[..., None]
            buf[name] = torch.where(own[..., None], u8, torch.full_like(u8, 0xFE))
            buf[name + "_scale"] = torch.where(own, sc, torch.full_like(sc, float("nan")))
        else:
            vals[name] = x.double().numpy()
            buf[name] = torch.where(own[..., None], x, torch.full_like(x, garbage))
    c = m.PagedCache(**{n: t.cuda() for n, t in buf.items()}, table=table.cuda(),
                     kv_len=torch.tensor(kv, dtype=torch.int32).cuda())
    return c, {"table": table.numpy(), "kv_len": np.array(kv), "page": page, **vals}


def check_attention(o, q, oc, n_new, causal, window, scale, what=""):
    """Every written row within the kernel's bound of the fp64 oracle.

    A weight p is rounded to bf16 (half a step, 2^-8 of it) before the product with V, and o once
    more; a logit carries the fp32 rounding of d products and of the scaling, at most
    (d + 4) 2^-23 scale sum|q_i k_i| (2^-23 rather than 2^-24: the tensor core may truncate), which
    moves p by as much relatively, as the row sum's own fp32 additions do by keys * 2^-23."""
    B, H, N, d = q.shape
    Hkv = oc["k"].shape[1]
    qd, od = q.double().numpy(), o.double().cpu().numpy()
    ref = OPG.attend(oc, qd, n_new, causal, window, scale)
    mag = OPG.attend({**oc, "v": np.abs(oc["v"])}, qd, n_new, causal, window, scale)  # sum_j p_j |v_j|
    for b in range(B):
        n, kv = int(n_new[b]), int(oc["kv_len"][b])
        if n == 0:
            continue
        K = np.abs(OPG.tokens(oc, "k", b, np.arange(kv)))
        for h in range(H):
            zmag = (np.abs(qd[b, h, :n]) @ K[h // (H // Hkv)].T).max(-1, initial=0.0)
            eps = 2.0 ** -8 + (d + 4) * 2.0 ** -23 * scale * zmag * 2 + kv * 2.0 ** -23
            lim = eps[:, None] * mag[b, h, :n] + 2.0 ** -8 * np.abs(ref[b, h, :n]) + 1e-30
            err = np.abs(od[b, h, :n] - ref[b, h, :n])
            worst = float((err / lim).max())
            assert worst <= 1.0, f"{what} b {b} h {h}: {worst:.3f} of the bound"
