"""GPU: calls that the header allows and that are easily broken: the output over the queries, padding
that holds anything, pages of 1,024 in tiles, one page twice in a table, thousands of sequences, calls
from two threads, and a first call that is captured."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import paged as OPG
from paged_util import build, check_attention
from parity_util import bsa

pytestmark = pytest.mark.gpu

BF16, E4M3 = 1, 2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _workspace(m, dm, c):
    return torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("H,N", [(8, 1), (4, 40), (4, 200), (2, 700)])
def test_the_output_may_lie_over_the_queries(kind, H, N):
    m = bsa()
    c, _ = build(kind, 2, 64, 128, [3000 + N, 100 + N], 31)
    q = _rand((2, H, N, 128), 32).cuda()
    dm = m.dims(2, H, N, 128, 1, 1, 0)
    ws, o = _workspace(m, dm, c), torch.empty_like(q)
    m.paged_forward(dm, c, q, o, ws)
    m.paged_forward(dm, c, q, q, ws)
    assert torch.equal(q, o) and m.get_device_error() == 0


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("H,N,n_new", [(4, 4, [1, 3]), (2, 60, [60, 7]), (4, 300, [5, 299])])
def test_padding_may_hold_anything(kind, H, N, n_new):
    """NaN, infinities and the type's largest values in the rows behind each sequence's tokens, in Q and
    in the chunk's K and V: the cache and the results are as with zeros there."""
    m = bsa()
    kv = [n + x for n, x in zip(n_new, (500, 33))]
    q, k, v = _rand((2, H, N, 128), 1), _rand((2, 2, N, 128), 2), _rand((2, 2, N, 128), 3)
    outs = []
    for fill in (0.0, float("nan"), float("inf"), -torch.finfo(torch.bfloat16).max):
        c, oc = build(kind, 2, 16, 128, kv, 5, garbage=0.5)
        for t in (q, k, v):
            for b in range(2):
                t[b, :, n_new[b]:] = fill
        dm, n = m.dims(2, H, N, 128, 1, 1, 0), _i32(n_new)
        o = torch.full((2, H, N, 128), -3.0, dtype=torch.bfloat16, device="cuda")
        m.paged_append(dm, c, k.cuda(), v.cuda(), n_new=n)
        m.paged_forward(dm, c, q.cuda(), o, _workspace(m, dm, c), n_new=n)
        assert m.get_device_error() == 0
        outs.append((o, c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()))
    for x in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, outs[0]))
    assert all((outs[0][0][b, :, n_new[b]:] == -3.0).all() for b in range(2))


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [40, 256, 257])
def test_large_pages_in_tiles(kind, d, N):
    m = bsa()
    kv = [2100, 1024 + N]
    c, oc = build(kind, 1, 1024, d, kv, 8)
    q = _rand((2, 2, N, d), 9)
    dm = m.dims(2, 2, N, d, 1, 1, 0)
    o = torch.zeros((2, 2, N, d), dtype=torch.bfloat16, device="cuda")
    m.paged_forward(dm, c, q.cuda(), o, _workspace(m, dm, c))
    assert m.get_device_error() == 0
    check_attention(o, q, oc, [N, N], True, 0, d ** -0.5)


@pytest.mark.parametrize("N", [1, 50, 200])
def test_one_page_may_stand_twice_in_a_table(N):
    m = bsa()
    c, oc = build(BF16, 2, 16, 64, [320], 10)
    c.table[0, 5:9] = c.table[0, 2]
    oc["table"][0, 5:9] = oc["table"][0, 2]
    q = _rand((1, 2, N, 64), 11)
    dm = m.dims(1, 2, N, 64, 1, 1, 0)
    o = torch.zeros((1, 2, N, 64), dtype=torch.bfloat16, device="cuda")
    m.paged_forward(dm, c, q.cuda(), o, _workspace(m, dm, c))
    check_attention(o, q, oc, [N], True, 0, 64 ** -0.5)
    k, v = (torch.empty((1, 2, 320, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.paged_read(m.dims(1, 2, 320, 64, 1, 1, 0), c, k, v)
    for got, want in zip((k, v), OPG.read(oc, 1, 320)):
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).bfloat16())
    assert m.get_device_error() == 0


@pytest.mark.parametrize("N", [1, 20])
def test_thousands_of_sequences(N):
    """5,000 sequences of one page that they share, of 1 to 16 tokens (some of no new token)."""
    m = bsa()
    B = 5000
    k, v = _rand((4, 1, 16, 64), 1), _rand((4, 1, 16, 64), 2)
    table = torch.arange(B).remainder(4).int()[:, None].contiguous()
    kv = [1 + i % 16 for i in range(B)]
    n_new = [min(N, x) if i % 11 else 0 for i, x in enumerate(kv)]
    c = m.PagedCache(k.cuda(), v.cuda(), table.cuda(), _i32(kv))
    oc = {"table": table.numpy(), "kv_len": np.array(kv), "page": 16, "k": k.double().numpy(), "v": v.double().numpy()}
    q = _rand((B, 1, N, 64), 3)
    dm = m.dims(B, 1, N, 64, 1, 1, 0)
    o = torch.full((B, 1, N, 64), -3.0, dtype=torch.bfloat16, device="cuda")
    m.paged_forward(dm, c, q.cuda(), o, _workspace(m, dm, c), n_new=_i32(n_new))
    assert m.get_device_error() == 0
    check_attention(o, q, oc, n_new, True, 0, 64 ** -0.5)
    assert all((o[b, :, n:] == -3.0).all() for b, n in list(enumerate(n_new))[::97])


def test_calls_from_two_threads():
    """Two threads, a stream, a cache and a workspace each, appending and attending at once."""
    m = bsa()
    jobs, errors = [], []
    for i, (kind, H, N) in enumerate([(BF16, 8, 1), (E4M3, 4, 130)]):
        c, _ = build(kind, 2, 16, 128, [2000 + N, N + 5], 80 + i, garbage=0.5)
        k, v, q = (_rand((2, h, N, 128), 90 + i).cuda() for h in (2, 2, H))
        dm = m.dims(2, H, N, 128, 1, 1, 0)
        ws, o = _workspace(m, dm, c), torch.zeros_like(q)
        m.paged_append(dm, c, k, v)
        m.paged_forward(dm, c, q, o, ws)
        jobs.append((dm, c, k, v, q, o, ws, o.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(dm, c, k, v, q, o, ws, want, st):
        try:
            for _ in range(100):
                m.paged_append(dm, c, k, v, stream=st)
                m.paged_forward(dm, c, q, o, ws, stream=st)
            st.synchronize()
            assert torch.equal(o, want)
        except BaseException as e:  # noqa: BLE001 (reported by the test's own thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors and m.get_device_error() == 0


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import block_sparse_attention_37_b200 as m
torch.manual_seed(0)
for kind in (m.CACHE_BF16, m.CACHE_E4M3):
    for N in (1, 40, 200):
        c = m.PagedCache.empty(200, 2, 16, 128, 1, 200, kind=kind)
        c.table.copy_(torch.randperm(200).view(1, 200))
        c.kv_len.fill_(3000)
        k, v, q = (torch.randn((1, h, n, 128), device="cuda").bfloat16() for h, n in ((2, 3000), (2, 3000), (4, N)))
        o, big, dm = torch.zeros_like(q), m.dims(1, 2, 3000, 128, 1, 1, 0), m.dims(1, 4, N, 128, 1, 1, 0)
        rk, rv = torch.zeros_like(k), torch.zeros_like(v)
        ws = torch.empty(m.paged_workspace_size(dm, c), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.paged_append(big, c, k, v)
            m.paged_forward(dm, c, q, o, ws)
            m.paged_read(big, c, rk, rv)
        g.replay()
        torch.cuda.synchronize()
        got = o.clone(), rk.clone(), rv.clone()
        o.zero_()
        m.paged_forward(dm, c, q, o, ws)
        m.paged_read(big, c, rk, rv)
        torch.cuda.synchronize()
        assert o.abs().sum() > 0 and all(torch.equal(a, b) for a, b in zip(got, (o, rk, rv)))
assert m.get_device_error() == 0
print("same")
"""


def test_a_first_call_may_be_captured():
    out = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip().endswith("same"), out.stderr[-2000:]
