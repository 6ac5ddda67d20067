"""GPU attention over caches whose values are not alike: tokens of zeros, V over many powers of two,
Q rows with one large channel. Against the fp64 oracle, as tests/test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from oracle import paged as OPG
from paged_util import check_attention
from parity_util import bsa

pytestmark = pytest.mark.gpu

BF16, E4M3 = 1, 2


def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def _cache(kind, k, v, kv, page, seed=1):
    """(PagedCache, oracle cache) of the tokens k, v (bf16 [B, Hkv, L, d]; kv[b] of them), written by
    bsa_paged_append into pages in random order."""
    m = bsa()
    B, Hkv, L, d = k.shape
    mp = -(-L // page)
    c = m.PagedCache.empty(B * mp, Hkv, page, d, B, mp, kind=kind)
    c.table.copy_(torch.randperm(B * mp, generator=torch.Generator().manual_seed(seed)).view(B, mp))
    lens = torch.tensor(kv, dtype=torch.int32).cuda()
    c.kv_len.copy_(lens)
    m.paged_append(m.dims(B, Hkv, L, d, 1, 1, 0), c, k.cuda(), v.cuda(), n_new=lens)
    oc = {"table": c.table.cpu().numpy(), "kv_len": np.array(kv), "page": page,
          "k": np.zeros(c.k.shape), "v": np.zeros(c.k.shape)}
    vals = [x.double().numpy() for x in (k, v)]
    if kind == E4M3:
        vals = [q * s[..., None] for q, s in (OPG.quantize_tokens(x.float().numpy()) for x in (k, v))]
    return c, OPG.append(oc, *vals, kv)


def _forward(c, q, causal, window):
    m = bsa()
    B, H, N, d = q.shape
    dm = m.dims(B, H, N, d, 1, 1, 0)
    ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    o = torch.full((B, H, N, d), -3.0, dtype=torch.bfloat16, device="cuda")
    m.paged_forward(dm, c, q.cuda(), o, ws, causal=causal, window=window)
    assert m.get_device_error() == 0
    return o


def _check(kind, k, v, kv, N, page, causal=True, window=0, G=2):
    c, oc = _cache(kind, k, v, kv, page)
    B, Hkv, _, d = k.shape
    q = _rand((B, G * Hkv, N, d), 77) * 2
    check_attention(_forward(c, q, causal, window), q, oc, [N] * B, causal, window, d ** -0.5)


# one kernel each: few rows, 17 to 128 rows, more
ROWS = [1, 5, 40, 200]


@pytest.mark.parametrize("zeros", ["one", "some", "pages", "negative"])
@pytest.mark.parametrize("down", [0, 20, 40, 60])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", ROWS)
def test_tokens_of_zeros_among_small_values(N, d, down, zeros):
    """Zero V tokens (scale 1 in an e4m3 cache, whatever the others') change nothing for the rest,
    V of 2^-down: a single one, every ninth, whole tiles of them, and negative zeros. The bound is the
    one every case has: it is relative to sum p |v|, which the zeros leave as it is."""
    L = 437 + N
    k, v = _rand((1, 2, L, d), 1), _rand((1, 2, L, d), 2) * 2.0 ** -down
    at = {"one": [11], "some": list(range(3, L, 9)), "pages": list(range(64, 320)),
          "negative": list(range(0, L, 5))}[zeros]
    v[:, :, at] = -0.0 if zeros == "negative" else 0.0
    _check(E4M3, k, v, [L], N, 16)


@pytest.mark.parametrize("N", ROWS)
def test_a_cache_of_zeros_reads_zero(N):
    """Every V token zero: the output is zero, to the bit (and no infinity times zero anywhere)."""
    L = 300 + N
    c, _ = _cache(E4M3, _rand((1, 2, L, 128), 1), torch.zeros((1, 2, L, 128), dtype=torch.bfloat16), [L], 16)
    assert (_forward(c, _rand((1, 4, N, 128), 3), True, 0) == 0).all()


@pytest.mark.parametrize("shape", ["growing", "shrinking", "mixed"])
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", ROWS)
def test_values_over_many_powers_of_two(N, d, kind, shape):
    """V's tokens from 2^-10 to 2^10, along the keys or in any order, with causal rows, windows and
    sequences of two lengths, over enough keys that runs start and end inside a sequence."""
    L = 2500 + N
    k, v = _rand((2, 1, L, d), 5), _rand((2, 1, L, d), 6)
    e = torch.linspace(-10, 10, L)
    if shape == "shrinking":
        e = e.flip(0)
    elif shape == "mixed":
        e = e[torch.randperm(L, generator=torch.Generator().manual_seed(7))]
    v = (v.float() * torch.exp2(e.round())[:, None]).bfloat16()
    for causal, window in ((True, 0), (True, 150), (False, 0)):
        _check(kind, k, v, [L, L - 1111], N, 64, causal, window)


@pytest.mark.parametrize("shape", ["growing", "shrinking"])
@pytest.mark.parametrize("N", ROWS)
def test_small_values_with_zeros_next_to_large_ones(N, shape):
    """Zero tokens everywhere and V from 2^-30 to 2^-10: sigma moves through its whole range below the
    zeros' scale."""
    L = 1500 + N
    k, v = _rand((1, 1, L, 128), 8), _rand((1, 1, L, 128), 9)
    e = torch.linspace(-30, -10, L)
    v = (v.float() * torch.exp2((e if shape == "growing" else e.flip(0)).round())[:, None]).bfloat16()
    v[:, :, ::7] = 0
    _check(E4M3, k, v, [L], N, 32)


@pytest.mark.parametrize("up", [10, 20])
@pytest.mark.parametrize("at", ["last", "outside"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [5, 40, 200])
def test_a_large_token_that_most_rows_do_not_keep(N, d, at, up):
    """e4m3: V of 2^up at the chunk's last position (one row keeps it), or before every row's window:
    the other rows' results keep their bits, as the header says down to 2^-20 of the largest scale."""
    L = 700 + N
    k, v = _rand((1, 2, L, d), 15), _rand((1, 2, L, d), 16)
    j = L - 1 if at == "last" else L - N - 131
    v[:, :, j] *= 2.0 ** up
    _check(E4M3, k, v, [L], N, 16, window=0 if at == "last" else 130)


@pytest.mark.parametrize("big", [4, 8, 11])
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("N", ROWS)
def test_queries_with_one_large_channel(N, kind, big):
    """One channel of Q 2^big times the others, on keys that are small there: bf16 caches take Q as it is,
    and few rows nearly so (2^-25 of the largest value); e4m3 chunks add an error of 2^-17 of the row's
    largest value a channel, which the header states (the row's largest value is brought to 2^7 .. 2^8, the
    second e4m3 part ends at 2^-9, so half a step is 2^-10): it moves a logit by at most
    scale 2^-17 max|q| sum|k|, and the weights by that."""
    L, d = 500 + N, 128
    k, v = _rand((1, 1, L, d), 21), _rand((1, 1, L, d), 22)
    k[..., 17] *= 2.0 ** -big
    q = _rand((1, 2, N, d), 23)
    q[..., 17] = 2.0 ** big
    c, oc = _cache(kind, k, v, [L], 64)
    o = _forward(c, q, True, 0)
    if kind == BF16 or 2 * N <= 16:
        check_attention(o, q, oc, [N], True, 0, d ** -0.5)
        return
    qd, od = q.double().numpy(), o.double().cpu().numpy()
    ref = OPG.attend(oc, qd, [N], True, 0, d ** -0.5)
    mag = OPG.attend({**oc, "v": np.abs(oc["v"])}, qd, [N], True, 0, d ** -0.5)
    K = np.abs(OPG.tokens(oc, "k", 0, np.arange(L)))
    zmag = (np.abs(qd[0]) @ K[0].T).max(-1)
    split = 2.0 ** -17 * np.abs(qd[0]).max(-1) * K[0].sum(-1).max()
    # as check_attention, with the split's error on a logit: twice, for the weight and for the row's sum
    eps = 2.0 ** -8 + d ** -0.5 * 2 * (split + (d + 4) * 2.0 ** -23 * zmag) + L * 2.0 ** -23
    lim = eps[..., None] * mag[0] + 2.0 ** -8 * np.abs(ref[0])
    assert (np.abs(od[0] - ref[0]) <= lim).all(), float((np.abs(od[0] - ref[0]) / lim).max())
