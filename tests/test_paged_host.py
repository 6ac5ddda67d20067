"""The paged cache's calls on the host: every refusal of the C ABI before any CUDA call, the
binding's refusals, and the order in which it passes its buffers (CPU tensors: nothing runs)."""
import ctypes

import pytest
import torch


def _m():
    from block_sparse_attention_37_b200 import build
    build.build()
    import block_sparse_attention_37_b200 as m
    return m


P, BAD = 4096, 4097   # addresses never dereferenced: aligned, and not


def _cache_c(m, **kw):
    f = dict(kind=m.CACHE_BF16, n_pages=8, Hkv=2, page=16, d=64, max_pages=4, k=P, v=P, k_scale=None, v_scale=None,
             table=P, kv_len=P)
    f.update(kw)
    return m.PagedCacheC(**f)


def _dims(m, B=2, H=4, N=3, d=64):
    return m.dims(B, H, N, d, 1, 1, 0)


BAD_CACHES = [
    ("kind", dict(kind=3), "ERR_INVALID_ARG"), ("pages", dict(n_pages=0), "ERR_INVALID_ARG"),
    ("heads", dict(Hkv=0), "ERR_INVALID_ARG"), ("table width", dict(max_pages=0), "ERR_INVALID_ARG"),
    ("d of the dims", dict(d=128), "ERR_INVALID_ARG"), ("null k", dict(k=None), "ERR_INVALID_ARG"),
    ("null v", dict(v=None), "ERR_INVALID_ARG"), ("null table", dict(table=None), "ERR_INVALID_ARG"),
    ("null kv_len", dict(kv_len=None), "ERR_INVALID_ARG"), ("misaligned k", dict(k=BAD), "ERR_INVALID_ARG"),
    ("misaligned v", dict(v=BAD), "ERR_INVALID_ARG"), ("e4m3 without scales", dict(kind=2), "ERR_INVALID_ARG"),
    ("e4m3, one scale", dict(kind=2, k_scale=P), "ERR_INVALID_ARG"),
    ("e4m3, misaligned scale", dict(kind=2, k_scale=P, v_scale=BAD), "ERR_INVALID_ARG"),
    ("small page", dict(page=8), "ERR_UNSUPPORTED"), ("large page", dict(page=2048), "ERR_UNSUPPORTED"),
    ("odd page", dict(page=48), "ERR_UNSUPPORTED"), ("long row", dict(max_pages=1 << 27), "ERR_UNSUPPORTED"),
]


def _calls(m, lib, dm, c):
    d, cc = ctypes.byref(dm), ctypes.byref(c) if c is not None else None
    return {
        "append": lambda k=P, v=P: lib.bsa_paged_append(d, k, v, None, cc, None),
        "read": lambda k=P, v=P: lib.bsa_paged_read(d, cc, None, k, v, None),
        "forward": lambda q=P, o=P, causal=1, window=0, scale=0.5, ws=P, wb=1 << 40: lib.bsa_paged_forward(
            d, q, None, cc, causal, window, scale, ws, wb, o, None),
    }


@pytest.mark.parametrize("what,kw,status", BAD_CACHES, ids=[c[0] for c in BAD_CACHES])
def test_bad_caches_are_refused_by_every_call(what, kw, status):
    m = _m()
    dm, c = _dims(m), _cache_c(m, **kw)
    for call in _calls(m, m.library(), dm, c).values():
        assert call() == getattr(m, status)
    assert m.library().bsa_paged_workspace_size(ctypes.byref(dm), ctypes.byref(c)) == 0


def test_bad_arguments_are_refused():
    m = _m()
    lib = m.library()
    good = _calls(m, lib, _dims(m), _cache_c(m))
    for name in ("append", "read"):
        for kw in (dict(k=None), dict(v=None), dict(k=BAD), dict(v=BAD)):
            assert good[name](**kw) == m.ERR_INVALID_ARG
    inf, nan = float("inf"), float("nan")
    for kw in (dict(q=None), dict(o=None), dict(q=BAD), dict(o=BAD), dict(causal=2), dict(causal=-1), dict(window=-1),
               dict(causal=0, window=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan)):
        assert good["forward"](**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(wb=0), dict(ws=P + 128)):
        assert good["forward"](**kw) == m.ERR_WORKSPACE, kw
    need = m.paged_workspace_size(_dims(m), type("C", (), {"_ref": ctypes.byref(_cache_c(m))}))
    assert need > 0 and good["forward"](wb=need - 1) == m.ERR_WORKSPACE
    for bad in (_dims(m, B=0), _dims(m, N=0), _dims(m, H=0)):
        for call in _calls(m, lib, bad, _cache_c(m)).values():
            assert call() == m.ERR_INVALID_ARG
    assert lib.bsa_paged_append(None, P, P, None, ctypes.byref(_cache_c(m)), None) == m.ERR_INVALID_ARG
    for call in _calls(m, lib, _dims(m), None).values():
        assert call() == m.ERR_INVALID_ARG
    # query heads not a multiple of the cache's: the forward alone minds
    assert _calls(m, lib, _dims(m, H=3), _cache_c(m))["forward"]() == m.ERR_INVALID_ARG
    # head dimension outside the kernels, and more rows than an index holds
    for call in _calls(m, lib, _dims(m, d=96), _cache_c(m, d=96)).values():
        assert call() == m.ERR_UNSUPPORTED
    assert _calls(m, lib, _dims(m, B=1 << 10, N=1 << 21), _cache_c(m))["forward"]() == m.ERR_UNSUPPORTED


def test_workspace_does_not_grow_with_the_cache():
    m = _m()
    dm, lib = _dims(m, B=4, H=8, N=300, d=128), m.library()
    a, b = (lib.bsa_paged_workspace_size(ctypes.byref(dm), ctypes.byref(_cache_c(m, d=128, n_pages=n, max_pages=w)))
            for n, w in ((8, 4), (1 << 20, 1 << 20)))
    assert a == b > 0


def _tensors(m, kind, n_pages=6, Hkv=2, page=16, d=64, B=2, max_pages=3):
    dt = torch.uint8 if kind == m.CACHE_E4M3 else torch.bfloat16
    t = {"k": torch.zeros((n_pages, Hkv, page, d), dtype=dt), "v": torch.zeros((n_pages, Hkv, page, d), dtype=dt),
         "table": torch.zeros((B, max_pages), dtype=torch.int32), "kv_len": torch.zeros(B, dtype=torch.int32)}
    if kind == m.CACHE_E4M3:
        t |= {s: torch.zeros((n_pages, Hkv, page)) for s in ("k_scale", "v_scale")}
    return t


def test_cache_construction_refuses_what_does_not_fit():
    m = _m()
    for kind in (m.CACHE_BF16, m.CACHE_E4M3):
        t = _tensors(m, kind)
        with pytest.raises(ValueError, match="CUDA device"):
            m.PagedCache(**t)
        for name, x in t.items():
            with pytest.raises((TypeError, ValueError)):
                m.PagedCache(**{**t, name: x.double()})
            with pytest.raises((TypeError, ValueError)):
                m.PagedCache(**{**t, name: None})
            with pytest.raises(ValueError):
                m.PagedCache(**{**t, name: x[..., :-1].contiguous() if name in ("v", "k_scale", "v_scale")
                                else x[:1] if name == "kv_len" else x.reshape(-1)})
    with pytest.raises(TypeError, match="belongs to an e4m3"):
        m.PagedCache(**_tensors(m, m.CACHE_BF16), k_scale=torch.zeros(6, 2, 16), v_scale=torch.zeros(6, 2, 16))
    with pytest.raises(ValueError, match="kind"):
        m.PagedCache.empty(4, 1, 16, 64, 1, 2, kind=7, device="cpu")


class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, {}

    def __getattr__(self, name):
        if name in ("bsa_error_string", "bsa_paged_workspace_size"):
            return getattr(self.real, name)

        def call(*args):
            self.calls[name] = args
            return 0
        return call


@pytest.fixture
def recorded(monkeypatch):
    m = _m()
    rec = _Recorder(m.library())
    monkeypatch.setattr(m, "_lib", lambda: rec)

    def host_ptr(t, dtype=None, name="tensor", numel=None):
        if t is None:
            return None
        m._check_buffer(t, dtype, name, numel)
        return t.data_ptr()
    monkeypatch.setattr(m, "_ptr", host_ptr)
    return m, rec


@pytest.mark.parametrize("e4m3", [False, True])
def test_buffers_are_passed_in_abi_order(recorded, e4m3):
    m, rec = recorded
    t = _tensors(m, m.CACHE_E4M3 if e4m3 else m.CACHE_BF16)
    c = m.PagedCache(**t)
    B, H, N, d = 2, 4, 5, 64
    dm = m.dims(B, H, N, d, 1, 1, 0)
    k, v = (torch.zeros((B, 2, N, d), dtype=torch.bfloat16) for _ in range(2))
    q, o = (torch.zeros((B, H, N, d), dtype=torch.bfloat16) for _ in range(2))
    n_new, ws = torch.ones(B, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)

    def holds(ref):
        s = ref._obj
        assert (s.n_pages, s.Hkv, s.page, s.d, s.max_pages) == (6, 2, 16, 64, 3)
        assert s.kind == (m.CACHE_E4M3 if e4m3 else m.CACHE_BF16)
        for name in ("k", "v", "table", "kv_len", "k_scale", "v_scale"):
            assert getattr(s, name) == (t[name].data_ptr() if name in t else None)

    m.paged_append(dm, c, k, v, n_new=n_new, stream=0)
    a = rec.calls["bsa_paged_append"]
    assert a[0]._obj is dm and a[1:4] == (k.data_ptr(), v.data_ptr(), n_new.data_ptr())
    holds(a[4])
    m.paged_read(dm, c, k, v, begin=n_new, stream=0)
    a = rec.calls["bsa_paged_read"]
    holds(a[1])
    assert a[2:5] == (n_new.data_ptr(), k.data_ptr(), v.data_ptr())
    m.paged_forward(dm, c, q, o, ws, n_new=n_new, causal=True, window=7, stream=0)
    a = rec.calls["bsa_paged_forward"]
    assert a[1:3] == (q.data_ptr(), n_new.data_ptr())
    holds(a[3])
    assert a[4:6] == (1, 7) and a[6] == pytest.approx(d ** -0.5)
    assert a[7:10] == (ws.data_ptr(), 4096, o.data_ptr())
    m.paged_forward(dm, c, q, o, ws, causal=False, scale=0.25, stream=0)
    a = rec.calls["bsa_paged_forward"]
    assert a[2] is None and a[4:7] == (0, 0, 0.25)


def test_calls_refuse_short_buffers_and_other_batches(recorded):
    m, _ = recorded
    c = m.PagedCache(**_tensors(m, m.CACHE_BF16))
    dm = m.dims(2, 4, 5, 64, 1, 1, 0)
    kv = torch.zeros((2, 2, 5, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 5, 64), dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    one = torch.ones(1, dtype=torch.int32)
    for f in (m.paged_append, m.paged_read):
        for args in ((kv[:1], kv), (kv, kv[:1]), (kv.float(), kv), (None, kv)):
            with pytest.raises((TypeError, ValueError, AttributeError)):
                f(dm, c, *args)
        with pytest.raises(ValueError, match="sequences"):
            f(m.dims(3, 4, 5, 64, 1, 1, 0), c, kv, kv)
    with pytest.raises(ValueError, match="n_new holds"):
        m.paged_append(dm, c, kv, kv, n_new=one)
    with pytest.raises(ValueError, match="begin holds"):
        m.paged_read(dm, c, kv, kv, begin=one)
    for args in ((q[:1], q, ws), (q, q[:1], ws), (q.float(), q, ws), (q, q, None)):
        with pytest.raises((TypeError, ValueError)):
            m.paged_forward(dm, c, *args)
    with pytest.raises(ValueError, match="n_new holds"):
        m.paged_forward(dm, c, q, q, ws, n_new=one)
