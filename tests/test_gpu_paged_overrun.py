"""GPU: an append whose kv_len runs past the table. Tokens past its end are dropped and reported; the
tokens that were in the cache keep their places and their bytes."""
import pytest
import torch

from parity_util import bsa

pytestmark = pytest.mark.gpu

BF16, E4M3 = 1, 2


@pytest.mark.parametrize("kv,fits", [(51, 2), (53, 0), (54, 0), (1 << 30, 0), (2**31 - 1, 0)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_an_append_past_the_table_overwrites_nothing(kind, d, kv, fits):
    """Three pages of 16 hold a full sequence; five tokens end at kv. Of them `fits` have a position in
    the table. A second sequence of the batch is appended to as always."""
    m = bsa()
    B, Hkv, page, N = 2, 2, 16, 5
    full = m.PagedCache.empty(B * 3, Hkv, page, d, B, 3, kind=kind)
    full.table.copy_(torch.arange(B * 3).view(B, 3))
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda n: torch.randn((B, Hkv, n, d), generator=g, device="cuda").bfloat16()
    full.kv_len.copy_(torch.tensor([48, 40]))
    m.paged_append(m.dims(B, Hkv, 48, d, 1, 1, 0), full, new(48), new(48),
                   n_new=torch.tensor([48, 40], dtype=torch.int32).cuda())
    assert m.get_device_error() == 0
    names = ["k", "v"] + (["k_scale", "v_scale"] if kind == E4M3 else [])
    want = {n: getattr(full, n).clone() for n in names}
    k, v = new(N), new(N)
    # what a sound append writes: the same tokens into a cache with room for them
    wide = m.PagedCache.empty(B * 5, Hkv, page, d, B, 5, kind=kind)
    wide.table.copy_(torch.arange(B * 5).view(B, 5))
    wide.kv_len.copy_(torch.tensor([min(kv, 60), 45]))
    dm = m.dims(B, Hkv, N, d, 1, 1, 0)
    m.paged_append(dm, wide, k, v)
    assert m.get_device_error() == 0
    for n in names:
        w, x = want[n], getattr(wide, n)
        for i in range(fits):
            j = kv - N + i
            w[j // page, :, j % page] = x[j // page, :, j % page]
        for j in range(40, 45):
            w[3 + j // page, :, j % page] = x[5 + j // page, :, j % page]
    full.kv_len.copy_(torch.tensor([kv, 45]))
    m.paged_append(dm, full, k, v)
    assert m.get_device_error() == m.DEVERR_BAD_INDEX
    for n in names:
        assert torch.equal(getattr(full, n).view(torch.uint8), want[n].view(torch.uint8)), n
