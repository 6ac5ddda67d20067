"""PagedCache hands the library the addresses of its tensors once: a tensor that is replaced, moved or
resized behind its back is refused (CPU tensors: nothing runs)."""
import pytest
import torch

from test_paged_host import _m, _tensors, recorded  # noqa: F401 (fixture)


def _make(m, e4m3):
    return m.PagedCache(**_tensors(m, m.CACHE_E4M3 if e4m3 else m.CACHE_BF16))


def _names(e4m3):
    return ["k", "v", "table", "kv_len"] + (["k_scale", "v_scale"] if e4m3 else [])


@pytest.mark.parametrize("e4m3", [False, True])
def test_tensors_are_not_replaced(recorded, e4m3):  # noqa: F811
    m, _ = recorded
    c = _make(m, e4m3)
    for name in _names(e4m3):
        held = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, held + 1)
        with pytest.raises(AttributeError):
            setattr(c, name, held.clone())
        with pytest.raises(AttributeError):
            setattr(c, name, None)
        with pytest.raises(AttributeError):
            delattr(c, name)
        assert getattr(c, name) is held
    with pytest.raises(AttributeError):
        c.kv_len = c.kv_len + 1
    if not e4m3:
        with pytest.raises(AttributeError):
            c.k_scale = torch.zeros(6, 2, 16)


def test_writing_in_place_is_what_a_program_does(recorded):  # noqa: F811
    m, rec = recorded
    c = _make(m, False)
    at = c.kv_len.data_ptr()
    c.kv_len += 5
    c.kv_len[1] = 3
    c.table.copy_(torch.ones_like(c.table))
    assert c.kv_len.tolist() == [5, 3] and c.kv_len.data_ptr() == at and c._c.kv_len == at


@pytest.mark.parametrize("how", ["set", "storage", "resize"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_moved_tensors_are_refused_by_every_call(recorded, e4m3, how):  # noqa: F811
    m, rec = recorded
    dm = m.dims(2, 4, 5, 64, 1, 1, 0)
    kv = torch.zeros((2, 2, 5, 64), dtype=torch.bfloat16)
    q, ws = torch.zeros((2, 4, 5, 64), dtype=torch.bfloat16), torch.zeros(4096, dtype=torch.uint8)
    for name in _names(e4m3):
        c = _make(m, e4m3)
        t = getattr(c, name)
        if how == "set":
            t.set_(torch.zeros_like(t))
        elif how == "storage":
            t.untyped_storage().resize_(0)
        else:
            t.resize_(t.numel() * 1000)
        rec.calls.clear()
        for call in (lambda: m.paged_append(dm, c, kv, kv, stream=0), lambda: m.paged_read(dm, c, kv, kv, stream=0),
                     lambda: m.paged_forward(dm, c, q, q, ws, stream=0)):
            with pytest.raises(ValueError, match="moved or resized"):
                call()
        assert not rec.calls, name


def test_a_torch_without_its_short_ways_to_device_and_stream_will_do():
    """The binding falls back to torch's public functions (a process of its own: the module is imported
    after the private names are gone)."""
    import os
    import subprocess
    import sys
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda i=None: type("S", (), {"cuda_stream": 1000 + i})
import block_sparse_attention_37_b200 as m
assert m._current_device() == 3 and m._raw_stream(2) == 1002
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
