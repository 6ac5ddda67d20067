"""The paged-cache oracle against independent forms: torch's own e4m3 conversion, torch's attention
over the gathered tokens, and closed cases."""
import numpy as np
import pytest
import torch

from oracle import paged as OPG


def _cache(B, Hkv, d, page, max_pages, kv, seed):
    rng = np.random.default_rng(seed)
    n_pages = B * max_pages + 2
    table = rng.permutation(n_pages)[:B * max_pages].reshape(B, max_pages)
    k, v = (rng.standard_normal((n_pages, Hkv, page, d)) for _ in range(2))
    return {"table": table, "kv_len": np.asarray(kv), "page": page, "k": k, "v": v}


def test_token_codes_match_torchs_conversion():
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[3] = 0
    x[4] *= 1e-35
    x[5] *= 1e30
    code, s = OPG.quantize_tokens(x.float().numpy())
    amax = x.float().abs().amax(-1)
    r = torch.where(amax >= 2.0 ** -100, 448.0 / amax, torch.ones(()))
    want = (x.float() * r[:, None]).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(code, want)
    assert s[3] == 1.0 and (code[3] == 0).all() and s[4] == 1.0 and (code[4] == 0).all()
    err = np.abs(code * s[:, None] - x.double().numpy())
    # half a step: 2^-4 of the value, 2^-10 scales below the smallest normal code; s and r are
    # rounded to fp32, two roundings of 2^-24 each
    lim = np.maximum(np.abs(x.double().numpy()) * 2.0 ** -4, s[:, None] * 2.0 ** -10) * (1 + 2.0 ** -20)
    keep = [i for i in range(50) if i != 4]
    assert (err[keep] <= lim[keep]).all()


def test_tokens_that_are_not_finite_turn_nan():
    x = np.ones((3, 8), np.float32)
    x[0, 2], x[1, 5] = np.inf, np.nan
    code, s = OPG.quantize_tokens(x)
    assert np.isnan(s[:2]).all() and (code[:2] == 0).all() and s[2] == np.float32(1) / np.float32(448)


def test_append_then_read_gives_the_tokens_back():
    c = _cache(2, 3, 8, 4, 5, [13, 7], 0)
    k = np.random.default_rng(1).standard_normal((2, 3, 6, 8))
    out = OPG.append(c, k, 2 * k, [6, 2])
    rk, rv = OPG.read(out, 2, 6, begin=[7, 5])
    np.testing.assert_array_equal(rk[0], k[0])
    np.testing.assert_array_equal(rk[1, :, :2], k[1, :, :2])
    assert (rk[1, :, 2:] == 0).all()
    np.testing.assert_array_equal(rv, 2 * rk)
    ok, _ = OPG.read(c, 2, 7)
    nk, _ = OPG.read(out, 2, 7)
    np.testing.assert_array_equal(ok[0], nk[0])     # tokens before the chunk are untouched


@pytest.mark.parametrize("causal,window", [(0, 0), (1, 0), (1, 3)])
def test_attention_equals_torchs_on_gathered_tokens(causal, window):
    c = _cache(2, 2, 16, 4, 6, [21, 9], 3)
    q = np.random.default_rng(4).standard_normal((2, 6, 5, 16))
    n_new = [5, 3]
    o = OPG.attend(c, q, n_new, causal, window, 0.3)
    K, V = OPG.read(c, 2, 24)
    for b in range(2):
        n, kv = n_new[b], c["kv_len"][b]
        mask = torch.zeros(n, kv, dtype=torch.bool)
        for i in range(n):
            for j in range(kv):
                p = kv - n + i
                mask[i, j] = bool(not causal or (j <= p and (window == 0 or p - j < window)))
        tq = torch.from_numpy(q[b, :, :n])
        tk, tv = (torch.from_numpy(x[b, :, :kv]).repeat_interleave(3, 0) for x in (K, V))
        want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=mask, scale=0.3)
        np.testing.assert_allclose(o[b, :, :n], want.numpy(), rtol=1e-12, atol=1e-13)
        assert np.isnan(o[b, :, n:]).all()


def test_rows_without_keys_are_zero():
    c = _cache(1, 1, 8, 4, 2, [2], 5)
    o = OPG.attend(c, np.ones((1, 1, 4, 8)), [4], 1, 0, 1.0)   # positions -2 .. 1
    assert (o[0, 0, :2] == 0).all() and (o[0, 0, 2:] != 0).all()
