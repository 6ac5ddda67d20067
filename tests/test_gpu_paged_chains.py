"""GPU: chains of paged calls that rewrite what the call before them reads, launched without waiting
and captured: a block denoised in place, step after step."""
import pytest
import torch

from parity_util import bsa

pytestmark = pytest.mark.gpu

BF16, E4M3 = 1, 2


def _setup(kind, B, Hkv, N, d, page, kv):
    m = bsa()
    mp = -(-kv // page)
    c = m.PagedCache.empty(B * mp, Hkv, page, d, B, mp, kind=kind)
    c.table.copy_(torch.randperm(B * mp, generator=torch.Generator().manual_seed(3)).view(B, mp))
    c.kv_len.fill_(kv)
    g = torch.Generator(device="cuda").manual_seed(4)
    new = lambda h, n: torch.randn((B, h, n, d), generator=g, device="cuda").bfloat16()
    m.paged_append(m.dims(B, Hkv, kv, d, 1, 1, 0), c, new(Hkv, kv), new(Hkv, kv))
    return m, c, new, m.dims(B, Hkv, N, d, 1, 1, 0)


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("B,Hkv,N,d", [(1, 2, 32, 128), (4, 8, 1, 64), (2, 8, 700, 128)])
def test_read_append_read_of_the_same_positions(kind, B, Hkv, N, d):
    """Each step reads the block, writes new values over it and reads again, kv_len unchanged; every
    read equals the values written just before, bit for bit (bf16), or the eager read-back with a
    wait between the calls (e4m3)."""
    kv, steps = 900 + N, 12
    m, c, new, dm = _setup(kind, B, Hkv, N, d, 16, kv)
    begin = torch.full((B,), kv - N, dtype=torch.int32, device="cuda")
    ks, vs = [new(Hkv, N) for _ in range(steps)], [new(Hkv, N) for _ in range(steps)]
    want = []
    for k, v in zip(ks, vs):
        m.paged_append(dm, c, k, v)
        torch.cuda.synchronize()
        r = torch.empty_like(k), torch.empty_like(v)
        m.paged_read(dm, c, *r, begin=begin)
        torch.cuda.synchronize()
        want.append(r)
        if kind == BF16:
            assert torch.equal(r[0], k) and torch.equal(r[1], v)
    out = [[torch.empty_like(ks[0]) for _ in range(4)] for _ in range(steps)]

    def chain():
        for k, v, o in zip(ks, vs, out):
            m.paged_read(dm, c, o[0], o[1], begin=begin)
            m.paged_append(dm, c, k, v)
            m.paged_read(dm, c, o[2], o[3], begin=begin)

    def check():
        torch.cuda.synchronize()
        for s in range(steps):
            for i in range(2):
                assert torch.equal(out[s][i], want[s - 1][i])        # (the first finds the last step's)
                assert torch.equal(out[s][2 + i], want[s][i])
                out[s][i].zero_()
                out[s][2 + i].zero_()
    for _ in range(3):
        chain()
        check()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        chain()
    for _ in range(3):
        gr.replay()
        check()
    assert m.get_device_error() == 0


@pytest.mark.parametrize("kind", [BF16, E4M3])
@pytest.mark.parametrize("G,N", [(2, 1), (2, 32), (4, 200)])
def test_append_and_attention_over_the_same_positions(kind, G, N):
    """The same with the attention as the reader, its workspace shared by the calls of one stream, and
    queries and inputs that a kernel just before the call wrote."""
    m, c, new, dm = _setup(kind, 2, 2, N, 128, 64, 1500 + N)
    fm = m.dims(2, 2 * G, N, 128, 1, 1, 0)
    ws = torch.empty(m.paged_workspace_size(fm, c), dtype=torch.uint8, device="cuda")
    steps = 8
    ks, vs, qs = ([new(h, N) for _ in range(steps)] for h in (2, 2, 2 * G))
    k, v, q = torch.empty_like(ks[0]), torch.empty_like(vs[0]), torch.empty_like(qs[0])
    out = [torch.empty_like(qs[0]) for _ in range(steps)]

    def chain(wait=lambda: None):
        for s in range(steps):
            for dst, src in ((k, ks[s]), (v, vs[s]), (q, qs[s])):
                torch.add(src, 0, out=dst)
            wait()
            m.paged_append(dm, c, k, v)
            wait()
            m.paged_forward(fm, c, q, out[s], ws)
            wait()
    chain(torch.cuda.synchronize)
    want = [o.clone() for o in out]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        chain()
    for go in (chain, gr.replay) * 3:
        for o in out:
            o.zero_()
        go()
        torch.cuda.synchronize()
        for o, w in zip(out, want):
            assert torch.equal(o, w)
    assert m.get_device_error() == 0
