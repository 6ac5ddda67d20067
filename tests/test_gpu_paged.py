"""GPU paged cache (bsa_paged_append, bsa_paged_read, bsa_paged_forward) against the fp64 oracle.

Slots that hold no token hold NaN in every case here, and table entries past a sequence's pages
are out of range, so a result that reads either shows it."""
import numpy as np
import pytest
import torch

from oracle import paged as OPG
from paged_util import build, check_attention
from parity_util import bsa

pytestmark = pytest.mark.gpu

BF16, E4M3 = 1, 2


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


# ---------------------------------------------------------------------------- append and read

SHAPES = [  # B, Hkv, N, d, page, kv_len, n_new
    (1, 1, 1, 64, 16, [1], [1]),
    (3, 2, 1, 128, 16, [16, 17, 33], [1, 0, 1]),
    (2, 3, 37, 128, 32, [37, 100], [37, 5]),
    (4, 1, 50, 64, 64, [50, 64, 65, 1], [50, 0, 50, 1]),
    (2, 5, 130, 128, 1024, [1030, 131], [129, 130]),
]


@pytest.mark.parametrize("B,Hkv,N,d,page,kv,n_new", SHAPES)
@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_append_writes_the_chunk_and_nothing_else(kind, B, Hkv, N, d, page, kv, n_new):
    m = bsa()
    c, _ = build(kind, Hkv, page, d, kv, 5)
    before = {n: getattr(c, n).clone() for n in ("k", "v", "k_scale", "v_scale") if getattr(c, n) is not None}
    k, v = _rand((B, Hkv, N, d), 1), _rand((B, Hkv, N, d), 2) * 37
    k[0, 0, 0] = 0                       # an all-zero token: scale 1
    m.paged_append(m.dims(B, Hkv, N, d, 1, 1, 0), c, k.cuda(), v.cuda(), n_new=_i32(n_new))
    assert m.get_device_error() == 0
    table = c.table.cpu().numpy()
    for name, x in (("k", k), ("v", v)):
        want = {n: t.cpu().clone() for n, t in before.items() if n.startswith(name)}
        for b in range(B):
            for i in range(n_new[b]):
                j = kv[b] - n_new[b] + i
                pg, sl = int(table[b, j // page]), j % page
                if kind == BF16:
                    want[name][pg, :, sl] = x[b, :, i]
                else:
                    code, s = OPG.quantize_tokens(x[b, :, i].float().numpy())
                    want[name][pg, :, sl] = torch.from_numpy(code).to(torch.float8_e4m3fn).view(torch.uint8)
                    want[name + "_scale"][pg, :, sl] = torch.from_numpy(s).float()
        for n, t in want.items():
            got = getattr(c, n).cpu()
            # bit for bit (the garbage holds NaN; a zero's sign is the input's)
            as_int = {torch.bfloat16: torch.int16, torch.float32: torch.int32, torch.uint8: torch.uint8}[t.dtype]
            assert torch.equal(got.view(as_int), t.view(as_int)), n


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_extreme_tokens(d):
    """Tokens near the ends of bf16, subnormal ones, and ones that are not finite; the read-back of
    the last is NaN in every channel, of the others the oracle's value to the bit."""
    m = bsa()
    k = _rand((1, 1, 8, d), 3)
    k[0, 0, 0] *= 2.0 ** 120
    k[0, 0, 1] *= 2.0 ** -90
    k[0, 0, 2] *= 2.0 ** -110            # below the smallest scale: reads as zero
    k[0, 0, 3] *= 2.0 ** -128
    k[0, 0, 4, 5] = float("inf")
    k[0, 0, 5, 7] = float("nan")
    k[0, 0, 6, 9] = float("-inf")
    k[0, 0, 7, :] = torch.finfo(torch.bfloat16).max
    c, _ = build(E4M3, 1, 16, d, [8], 1)
    dm = m.dims(1, 1, 8, d, 1, 1, 0)
    m.paged_append(dm, c, k.cuda(), (k.flip(2)).cuda())
    rk, rv = torch.empty(1, 1, 8, d, dtype=torch.bfloat16).cuda(), torch.empty(1, 1, 8, d, dtype=torch.bfloat16).cuda()
    m.paged_read(dm, c, rk, rv)
    assert m.get_device_error() == 0
    for got, x in ((rk, k), (rv, k.flip(2))):
        code, s = OPG.quantize_tokens(x.float().numpy())
        want = torch.from_numpy((code.astype(np.float32) * s.astype(np.float32)[..., None])).bfloat16()
        assert torch.equal(got.cpu().isnan(), want.isnan())
        assert torch.equal(got.cpu().nan_to_num(), want.nan_to_num())


def test_every_code_reads_back_exactly():
    """All 254 codes that stand for a number, under scales 1 and 2^-3: exact in bf16."""
    m = bsa()
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F] + [0, 0], dtype=torch.uint8)
    c, _ = build(E4M3, 1, 16, 128, [2], 1)
    pg = int(c.table[0, 0])
    for t in (c.k, c.v):
        t[pg, 0, :2] = codes.view(2, 128).cuda()
    c.k_scale[pg, 0, :2], c.v_scale[pg, 0, :2] = 1.0, 0.125
    k, v = (torch.empty((1, 1, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.paged_read(m.dims(1, 1, 2, 128, 1, 1, 0), c, k, v)
    want = codes.view(torch.float8_e4m3fn).float().view(2, 128)
    assert torch.equal(k[0, 0].float().cpu(), want) and torch.equal(v[0, 0].float().cpu(), want / 8)


@pytest.mark.parametrize("B,Hkv,N,d,page,kv,begin", [
    (1, 1, 1, 64, 16, [1], None), (2, 3, 50, 128, 16, [77, 50], [20, 13]), (3, 2, 33, 64, 128, [0, 40, 33], [0, 33, 40]),
    (2, 1, 200, 128, 64, [129, 200], None)])
@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_read_gathers_and_zeroes(kind, B, Hkv, N, d, page, kv, begin):
    m = bsa()
    c, oc = build(kind, Hkv, page, d, kv, 9)
    k, v = (torch.full((B, Hkv, N, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.paged_read(m.dims(B, Hkv, N, d, 1, 1, 0), c, k, v, begin=None if begin is None else _i32(begin))
    assert m.get_device_error() == 0
    for got, want in zip((k, v), OPG.read(oc, B, N, begin)):
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).bfloat16())


# ---------------------------------------------------------------------------- attention

def _forward(c, q, n_new, causal, window, scale=None, stream=None):
    m = bsa()
    B, H, N, d = q.shape
    dm = m.dims(B, H, N, d, 1, 1, 0)
    ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                                              # NaN scratch
    o = torch.full((B, H, N, d), -3.0, dtype=torch.bfloat16, device="cuda")
    m.paged_forward(dm, c, q.cuda(), o, ws, n_new=None if n_new is None else _i32(n_new), causal=causal, window=window,
                    scale=scale, stream=stream)
    return o


def _check(kind, H, Hkv, N, d, page, kv, n_new, causal, window, seed=11, q=None):
    m = bsa()
    B = len(kv)
    c, oc = build(kind, Hkv, page, d, kv, seed)
    q = _rand((B, H, N, d), seed + 1) * 2 if q is None else q
    o = _forward(c, q, n_new, causal, window)
    assert m.get_device_error() == 0
    n = [N] * B if n_new is None else n_new
    check_attention(o, q, oc, n, causal, window, d ** -0.5)
    for b in range(B):
        assert (o[b, :, n[b]:] == -3.0).all()                   # rows behind the chunk, left as they were
    return o


CASES = [  # H, Hkv, N, page, kv_len, n_new, causal, window
    # single tokens: one key, page and tile borders, many heads a key head, a long row next to short ones
    (1, 1, 1, 16, [1], None, True, 0),
    (4, 2, 1, 16, [15, 16, 17, 63, 64, 65], None, True, 0),
    (16, 1, 1, 32, [128, 1], None, True, 0),
    (5, 1, 1, 64, [700, 3, 1029], None, True, 100),
    (8, 8, 1, 128, [2500], None, False, 0),
    (6, 2, 1, 1024, [2047, 1025], [1, 0], True, 0),
    # a few tokens: packed query heads, fewer than, exactly and more than 16 rows a key head
    (4, 2, 3, 16, [50, 3], [3, 3], True, 0),
    (8, 2, 4, 64, [129, 70], [4, 2], False, 0),
    (2, 2, 16, 32, [257, 16], None, True, 5),
    (4, 2, 9, 16, [300, 9, 41], [9, 9, 1], True, 0),
    (1, 1, 17, 64, [17], None, True, 0),
    # blocks and chunks: row tiles that end inside a chunk, chunks shorter than their padding
    (2, 1, 32, 64, [333, 1200], None, False, 0),
    (3, 3, 64, 16, [64, 200], [64, 61], True, 0),
    (4, 2, 65, 32, [300, 65], [65, 30], True, 0),
    (2, 2, 128, 128, [128, 513], None, True, 64),
    (2, 1, 129, 256, [1000], None, True, 0),
    (3, 1, 200, 16, [777, 201, 200], [200, 1, 150], True, 0),
    (2, 2, 300, 64, [300, 1111], [300, 257], True, 130),
    (1, 1, 513, 64, [2000], None, False, 0),
    (5, 1, 107, 16, [900, 107], [107, 50], True, 300),
    # one head over many tiles: an item split over most of the GPU
    (2, 1, 1, 64, [20000], None, True, 0),
    (1, 1, 33, 128, [20001], None, False, 0),
    (1, 1, 260, 32, [9000], None, True, 0),
]


@pytest.mark.parametrize("H,Hkv,N,page,kv,n_new,causal,window", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_forward_matches_the_oracle(kind, d, H, Hkv, N, page, kv, n_new, causal, window):
    _check(kind, H, Hkv, N, d, page, kv, n_new, causal, window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("H,N", [(2, 1), (2, 20), (2, 150)])
def test_more_items_than_the_gpu_has_ctas(kind, H, N, wide):
    """200 sequences of 1 to 500 tokens (empty chunks among them): CTAs run through several items,
    whole (a narrow table) or cut anywhere (a wide one)."""
    m = bsa()
    kv = [1 + (i * 37) % 500 for i in range(200)]
    n_new = [min(N, k, 1 + i % (N + 1)) if i % 7 else 0 for i, k in enumerate(kv)]
    c, oc = build(kind, 2, 16, 64, kv, 30, max_pages=200 if wide else 32)
    q = _rand((200, H, N, 64), 31)
    o = _forward(c, q, n_new, True, 0)
    assert m.get_device_error() == 0
    check_attention(o, q, oc, n_new, True, 0, 64 ** -0.5)
    for b in range(200):
        assert (o[b, :, n_new[b]:] == -3.0).all()


def test_offsets_past_32_bits():
    """Caches of more than 2^31 values (and bytes): the sequence's pages lie at the very end."""
    m = bsa()
    n_pages, Hkv, page, d = 2100, 8, 1024, 128                  # 2.2e9 codes each
    g = torch.Generator(device="cuda").manual_seed(1)
    code = lambda: torch.empty((n_pages, Hkv, page, d), dtype=torch.uint8, device="cuda")
    c = m.PagedCache(code(), code(), _i32([[n_pages - 1, n_pages - 2]]), _i32([1500]),
                     *(torch.ones((n_pages, Hkv, page), device="cuda") for _ in range(2)))
    k, v = (torch.randn((1, Hkv, 1500, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    m.paged_append(m.dims(1, Hkv, 1500, d, 1, 1, 0), c, k, v)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    m.paged_read(m.dims(1, Hkv, 1500, d, 1, 1, 0), c, rk, rv)
    oc = {"table": np.array([[0, 1]]), "kv_len": np.array([1500]), "page": page, "k": np.zeros((2, Hkv, page, d)),
          "v": np.zeros((2, Hkv, page, d))}
    vals = []
    for x, r in ((k, rk), (v, rv)):
        code_, s = OPG.quantize_tokens(x.float().cpu().numpy())
        vals.append(code_ * s[..., None])
        assert torch.equal(r.cpu(), torch.from_numpy((code_.astype(np.float32) * s.astype(np.float32)[..., None])).bfloat16())
    oc = OPG.append(oc, *vals, [1500])
    for N in (1, 40, 200):
        q = _rand((1, Hkv, N, d), N)
        check_attention(_forward(c, q, None, True, 0), q, oc, [N], True, 0, d ** -0.5)
    assert m.get_device_error() == 0


@pytest.mark.parametrize("N", [1, 40, 200])
def test_a_token_that_is_not_finite_reaches_only_its_own_sequence(N):
    """e4m3: a token with an infinity in K and V, appended mid-sequence: every row of that sequence
    that keeps it is NaN, the other sequence's rows are as before."""
    m = bsa()
    kv = [300 + N, 400 + N]
    c, _ = build(E4M3, 2, 16, 128, kv, 12)
    q = _rand((2, 4, N, 128), 13)
    good = _forward(c, q, None, True, 0)
    pg = int(c.table[0, 100 // 16])
    c.k_scale[pg, :, 100 % 16] = float("nan")
    c.v_scale[pg, :, 100 % 16] = float("nan")
    o = _forward(c, q, None, True, 0)
    assert o[0].isnan().all() and torch.equal(o[1], good[1])
    assert torch.equal(_forward(c, q, None, True, 64)[0].isnan(), torch.zeros_like(o[0], dtype=torch.bool))
    assert m.get_device_error() == 0


def test_sequences_may_share_pages():
    """Two sequences with the same prompt pages and a page of their own each."""
    m = bsa()
    c, oc = build(BF16, 2, 16, 64, [64, 80], 14)
    c.table[1, :3] = c.table[0, :3]
    oc["table"][1, :3] = oc["table"][0, :3]
    q = _rand((2, 4, 10, 64), 15)
    check_attention(_forward(c, q, None, True, 0), q, oc, [10, 10], True, 0, 64 ** -0.5)
    assert m.get_device_error() == 0


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("H,Hkv,N,kv", [(4, 1, 1, 4000), (2, 1, 40, 6000), (1, 1, 300, 9000)])
def test_a_wait_that_runs_out_is_reported_and_the_context_survives(kind, H, Hkv, N, kv):
    """The producer withholds a CTA's second key tile and waits are bounded by 2 ms: the call ends
    with BSA_DEVERR_TIMEOUT, and the next one is right."""
    m = bsa()
    c, oc = build(kind, Hkv, 64, 128, [kv, kv - 100], 16)
    q = _rand((2, H, N, 128), 17)
    good = _forward(c, q, None, True, 0)
    assert m.get_device_error() == 0
    m.set_wait_limit_ns(2_000_000)
    m.set_withheld_tile(1)
    try:
        _forward(c, q, None, True, 0)
        assert m.get_device_error() == m.DEVERR_TIMEOUT
    finally:
        m.set_withheld_tile(-1)
        m.set_wait_limit_ns(0)
    assert torch.equal(_forward(c, q, None, True, 0), good)
    assert m.get_device_error() == 0


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("N,n_new,kv", [(1, [1, 0, 0], [0, 0, 5]), (40, [40, 30, 0], [12, 0, 9]), (300, [300, 290], [20, 0])])
def test_rows_that_keep_no_key_are_zero(kind, N, n_new, kv):
    """A chunk longer than its cache (rows at negative positions), empty caches, empty chunks."""
    o = _check(kind, 4, 2, N, 128, 16, kv, n_new, True, 0)
    for b in range(len(kv)):
        empty = max(0, n_new[b] - kv[b])
        assert (o[b, :, :empty] == 0).all()
    if N > 1:
        _check(kind, 4, 2, N, 128, 16, kv, n_new, False, 0)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("N", [1, 40, 150])
def test_peaked_rows_and_large_logits(kind, N):
    """Logits in the hundreds: the running maximum moves far, late keys take everything."""
    _check(kind, 4, 2, N, 128, 32, [N + 700], None, True, 0, q=_rand((1, 4, N, 128), 3) * 60)


@pytest.mark.parametrize("N", [1, 24, 140])
def test_keys_at_the_ends_of_the_type_are_masked(N):
    """K of the type's lowest value, infinite and NaN, and V of the type's largest values, at
    positions past the window and the chunk's end: not a bit of the result may change."""
    m = bsa()
    kv = 500 + N
    c, _ = build(BF16, 2, 16, 128, [kv], 4, max_pages=(kv + 15) // 16 + 4)
    q = _rand((1, 4, N, 128), 5)
    o = _forward(c, q, None, True, 90)
    low = torch.finfo(torch.bfloat16).min
    for x in (low, float("inf"), float("nan")):
        for j in range(kv - N - 90 + 1):
            pg = int(c.table[0, j // 16])
            c.k[pg, :, j % 16] = x
            c.v[pg, :, j % 16] = low
        assert torch.equal(_forward(c, q, None, True, 90), o)
    assert m.get_device_error() == 0


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("H,Hkv,N", [(8, 2, 1), (2, 2, 70), (2, 1, 200)])
def test_results_repeat_to_the_bit(kind, H, Hkv, N):
    c, _ = build(kind, Hkv, 64, 128, [5000, 40 + N, 900], 6)
    q = _rand((3, H, N, 128), 7)
    o = _forward(c, q, None, True, 0)
    for _ in range(3):
        assert torch.equal(_forward(c, q, None, True, 0), o)


def test_equal_tokens_give_v_back():
    """Every key alike: the result is the mean of V over the kept keys, whatever the tile split."""
    m = bsa()
    kv = 1300
    c, oc = build(BF16, 1, 64, 64, [kv], 8)
    c.k.fill_(1.0)
    q = _rand((1, 1, 1, 64), 9)
    o = _forward(c, q, None, True, 0)
    mean = OPG.tokens(oc, "v", 0, np.arange(kv)).mean(1)
    # the weights are equal and exact in bf16 (1): only the output's rounding and fp32 sums remain
    lim = 2.0 ** -8 * np.abs(mean) + kv * 2.0 ** -23 * np.abs(OPG.tokens(oc, "v", 0, np.arange(kv))).mean(1)
    assert (np.abs(o[0, 0].double().cpu().numpy() - mean) <= lim).all()
    assert m.get_device_error() == 0


# ---------------------------------------------------------------------------- used together

@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_a_prompt_in_chunks_then_single_tokens(kind):
    """A prompt appended in two ragged chunks, then tokens one by one, attention after each, as a
    causal model runs; every step against the oracle's cache of the same tokens, and at the end the
    read-back equals what was appended (rounded to codes)."""
    m = bsa()
    B, H, Hkv, d, page, max_pages = 2, 4, 2, 128, 16, 20
    c = m.PagedCache.empty(B * max_pages, Hkv, page, d, B, max_pages, kind=kind)
    c.table.copy_(torch.randperm(B * max_pages, generator=torch.Generator().manual_seed(1)).view(B, max_pages))
    oc = {"table": c.table.cpu().numpy(), "kv_len": np.zeros(B, int), "page": page,
          "k": np.zeros(c.k.shape), "v": np.zeros(c.k.shape)}
    for step, (N, n_new) in enumerate([(150, [150, 90]), (40, [11, 40]), (1, [1, 1]), (1, [0, 1]), (1, [1, 1])]):
        k, v, q = (_rand((B, h, N, d), 100 * step + i) for i, h in enumerate((Hkv, Hkv, H)))
        kd, vd = k.double().numpy(), v.double().numpy()
        if kind == E4M3:
            kd, vd = (c_ * s[..., None] for c_, s in (OPG.quantize_tokens(x.float().numpy()) for x in (k, v)))
        n = _i32(n_new)
        c.kv_len += n
        oc["kv_len"] = oc["kv_len"] + np.array(n_new)
        oc = OPG.append(oc, kd, vd, n_new)
        m.paged_append(m.dims(B, H, N, d, 1, 1, 0), c, k.cuda(), v.cuda(), n_new=n)
        o = _forward(c, q, n_new, True, 0)
        assert m.get_device_error() == 0
        check_attention(o, q, oc, n_new, True, 0, d ** -0.5, f"step {step}")
    L = int(oc["kv_len"].max())
    k, v = (torch.empty((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.paged_read(m.dims(B, H, L, d, 1, 1, 0), c, k, v)
    for got, want in zip((k, v), OPG.read(oc, B, L)):
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).bfloat16())


def test_read_back_feeds_the_selection_and_the_sparse_forward():
    """The cached tokens read back into the contiguous layout: bsa_forward over them equals
    bsa_paged_forward without a mask (both within the attention bar), and bsa_select_topk of the
    read-back keys equals the selection on the keys that were appended."""
    m = bsa()
    B, H, N, d, bs = 1, 2, 640, 128, 128
    q, k, v = (_rand((B, H, N, d), 40 + i).cuda() for i in range(3))
    c = m.PagedCache.empty(40, H, 16, d, B, 40)
    c.table.copy_(torch.arange(39, -1, -1))
    c.kv_len.fill_(N)
    dm = m.dims(B, H, N, d, bs, bs, 0)
    m.paged_append(dm, c, k, v)
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    m.paged_read(dm, c, rk, rv)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    spec = m.select_spec(m.SELECT_POOLED_QK, [(0, 5, 2)], False)
    ws = torch.empty(m.select_workspace_size(dm, spec), dtype=torch.uint8, device="cuda")
    a, b = (m.BlockList.empty(B, H, 5, 5) for _ in range(2))
    m.select_topk(dm, q, k, spec, a, ws)
    m.select_topk(dm, q, rk, spec, b, ws)
    assert torch.equal(a.idx, b.idx) and torch.equal(a.cnt, b.cnt)
    o1 = torch.empty_like(q)
    m.forward(dm, q, rk, rv, o1, torch.zeros(H, dtype=torch.int32, device="cuda"))
    o2 = _forward(c, q.cpu(), None, False, 0)
    # both round the weights and the output to bf16: two half steps each of the largest |v|
    assert (o1.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max()
    assert m.get_device_error() == 0


# ---------------------------------------------------------------------------- streams, graphs, faults

def test_two_graphs_and_a_side_stream():
    """A decode step (append, forward) captured into two graphs with a workspace each, replayed in
    turn and again after the lengths moved; a third call on a side stream. All equal the eager call."""
    m = bsa()
    B, H, Hkv, d = 2, 8, 2, 128
    dm = m.dims(B, H, 1, d, 1, 1, 0)
    sets = []
    for s in range(2):
        c, _ = build(BF16, Hkv, 64, d, [900 + 64 * s, 130], 20 + s, garbage=0.5)
        k, v = _rand((B, Hkv, 1, d), s).cuda(), _rand((B, Hkv, 1, d), 5 + s).cuda()
        q = _rand((B, H, 1, d), 9 + s).cuda()
        o = torch.zeros_like(q)
        ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")

        def step(c=c, k=k, v=v, q=q, o=o, ws=ws):
            m.paged_append(dm, c, k, v)
            m.paged_forward(dm, c, q, o, ws)
        step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        sets.append((c, o, gr, step))
    for move in (0, -70, 33):
        for c, o, gr, step in sets:
            c.kv_len += move
        want = []
        for c, o, gr, step in sets:
            step()
            want.append(o.clone())
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(2):
            for c, o, gr, step in sets:
                gr.replay()
        torch.cuda.synchronize()
        for (c, o, gr, step), w in zip(sets, want):
            assert torch.equal(o, w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for c, o, gr, step in sets:
                o.zero_()
                step()
        side.synchronize()
        for (c, o, gr, step), w in zip(sets, want):
            assert torch.equal(o, w)
    assert m.get_device_error() == 0


@pytest.mark.parametrize("H,N", [(8, 1), (4, 40), (4, 200)])
def test_a_call_captured_behind_copies_and_a_fork(H, N):
    """The queries arrive by a copy node, the cache by a kernel on a forked stream: the captured call
    waits for both, replay after replay, with new queries and new keys each time."""
    m = bsa()
    kv = 1500
    c, oc = build(BF16, 2, 64, 128, [kv], 50, max_pages=64)
    dm = m.dims(1, H, N, 128, 1, 1, 0)
    ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")
    src, q = (torch.zeros((1, H, N, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros((1, 2, N, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    o = torch.zeros_like(q)
    m.paged_forward(dm, c, q, o, ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            m.paged_append(dm, c, k, v)
        q.copy_(src)
        main.wait_stream(side)
        m.paged_forward(dm, c, q, o, ws)
        q.copy_(src)
        m.paged_forward(dm, c, q, o, ws)
    for seed in range(3):
        hk, hv, hq = _rand((1, 2, N, 128), seed), _rand((1, 2, N, 128), 10 + seed), _rand((1, H, N, 128), 20 + seed)
        k.copy_(hk)
        v.copy_(hv)
        src.copy_(hq)
        oc = OPG.append(oc, hk.double().numpy(), hv.double().numpy(), [N])
        gr.replay()
        torch.cuda.synchronize()
        check_attention(o, hq, oc, [N], True, 0, 128 ** -0.5, f"replay {seed}")
    assert m.get_device_error() == 0


def test_two_streams_at_once():
    """Calls of both kernels on two streams, a workspace each, launched without waiting: as alone."""
    m = bsa()
    work = []
    for i, (H, N) in enumerate([(8, 1), (4, 300)]):
        c, _ = build(E4M3 if i else BF16, 2, 16, 128, [3000 + N, 40 + N], 60 + i, garbage=0.5)
        q = _rand((2, H, N, 128), 70 + i).cuda()
        dm = m.dims(2, H, N, 128, 1, 1, 0)
        ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")
        o = torch.zeros_like(q)
        m.paged_forward(dm, c, q, o, ws)
        work.append((dm, c, q, o, ws, o.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for dm, c, q, o, ws, want, st in work:
            m.paged_forward(dm, c, q, o, ws, stream=st)
    torch.cuda.synchronize()
    for dm, c, q, o, ws, want, st in work:
        assert torch.equal(o, want)
    assert m.get_device_error() == 0


@pytest.mark.parametrize("N", [1, 30, 140])
@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_faults_are_reported_and_the_next_call_is_right(kind, N):
    """Page indices outside the cache (read as page 0), lengths outside the table and the chunk:
    BSA_DEVERR_BAD_INDEX, and a sound call afterwards gives the sound result."""
    m = bsa()
    kv = [200 + N]
    c, oc = build(kind, 2, 16, 64, kv, 3, garbage=0.25)
    if kind == E4M3:
        c.k_scale.nan_to_num_(1.0)
        c.v_scale.nan_to_num_(1.0)
    q = _rand((1, 2, N, 64), 4)
    k = _rand((1, 2, N, 64), 5).cuda()
    dm = m.dims(1, 2, N, 64, 1, 1, 0)
    good = _forward(c, q, None, True, 0)
    kept = {n: getattr(c, n).clone() for n in ("table", "kv_len", "k", "v", "k_scale", "v_scale") if getattr(c, n) is not None}
    assert m.get_device_error() == 0

    def restore():
        for n, t in kept.items():
            getattr(c, n).copy_(t)
    for bad in (-1, c.k.shape[0], 1 << 30, -(1 << 31)):
        c.table[0, 3] = bad
        o = _forward(c, q, None, True, 0)
        assert m.get_device_error() == m.DEVERR_BAD_INDEX
        c.table[0, 3] = 0                                       # page 0 in its place
        assert torch.equal(_forward(c, q, None, True, 0), o)
        assert m.get_device_error() == 0
        restore()
    c.table[0, 1] = 1 << 20
    rk, rv = (torch.full((1, 2, 40, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.paged_read(m.dims(1, 2, 40, 64, 1, 1, 0), c, rk, rv)
    assert m.get_device_error() == m.DEVERR_BAD_INDEX
    assert (rk[:, :, 16:32] == 0).all() and (rk[:, :, :16] != 9).all() and (rv[:, :, 32:] != 0).any()
    restore()
    before = c.k.clone()
    c.table.fill_(-2)
    m.paged_append(dm, c, k, k)
    assert m.get_device_error() == m.DEVERR_BAD_INDEX
    assert torch.equal(c.k.view(torch.uint8), before.view(torch.uint8))
    restore()
    for n_kv, n_n in ((1 << 20, N), (-5, N), (kv[0], N + 1), (kv[0], -1)):
        c.kv_len.fill_(n_kv)
        _forward(c, q, [n_n], True, 0)
        code = m.get_device_error()
        assert code == m.DEVERR_BAD_INDEX, (n_kv, n_n)
        m.paged_read(m.dims(1, 2, 40, 64, 1, 1, 0), c, rk, rv)
        assert m.get_device_error() == (0 if n_kv == kv[0] else m.DEVERR_BAD_INDEX)
    restore()
    m.paged_read(m.dims(1, 2, 40, 64, 1, 1, 0), c, rk, rv, begin=_i32([-3]))
    assert m.get_device_error() == m.DEVERR_BAD_INDEX
    c.kv_len.fill_(N - 1)                                       # the chunk's first token has no position
    m.paged_append(dm, c, k, k)
    assert m.get_device_error() == m.DEVERR_BAD_INDEX
    restore()
    assert torch.equal(_forward(c, q, None, True, 0), good)
    assert m.get_device_error() == 0


def test_misuse_is_refused_before_a_launch():
    m = bsa()
    c, _ = build(BF16, 2, 16, 64, [20], 3)
    q = _rand((1, 2, 1, 64), 4).cuda()
    dm = m.dims(1, 2, 1, 64, 1, 1, 0)
    ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        m.paged_forward(dm, c, _rand((1, 2, 1, 128), 1).cuda()[..., ::2], q, ws)
    with pytest.raises(ValueError, match="CUDA device"):
        m.paged_forward(dm, c, q.cpu(), q, ws)
    with pytest.raises(m.BsaError, match="workspace"):
        m.paged_forward(dm, c, q, q, ws[:-256])
    with pytest.raises(m.BsaError, match="invalid"):
        m.paged_forward(dm, c, q, q, ws, causal=False, window=3)
    with pytest.raises(m.BsaError, match="invalid"):
        m.paged_forward(m.dims(1, 3, 1, 64, 1, 1, 0), c, _rand((1, 3, 1, 64), 1).cuda(), _rand((1, 3, 1, 64), 1).cuda(), ws)
    assert m.get_device_error() == 0
