"""Argument checks of the attention calls (CPU only): every call below fails validation, so
nothing is launched and no pointer is followed."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from quantized_grouped_gemm_router_gb300 import build as B  # noqa: E402

A = 1 << 20  # a fake, aligned pointer


@pytest.fixture(scope="module")
def m():
    B.build()
    import quantized_grouped_gemm_router_gb300 as mod
    return mod


@pytest.fixture(scope="module")
def fn(m):
    from quantized_grouped_gemm_router_gb300 import attention
    return attention._fn


def test_workspace_and_dims(m):
    assert m.attn_workspace_bytes(m.AttnDims(16, 2, 128)) >= 256
    for bad in ((16, 2, 96), (16, 3, 128), (0, 0, 128), (2, 4, 64), (65, 1, 64), (2048, 2048, 64), (16, -2, 128)):
        assert m.attn_workspace_bytes(m.AttnDims(*bad)) == 0, bad
    with pytest.raises(m.MoeError):
        m.attn_workspace(m.AttnDims(16, 2, 100), device="cpu")
    assert m.status_string(9) != "unknown status"


def test_prefill_refusals(m, fn):
    from quantized_grouped_gemm_router_gb300.attention import HeadsView
    dims = m.AttnDims(16, 2, 128)
    need = m.attn_workspace_bytes(dims)
    q, kv = HeadsView(A, 2048, 128), HeadsView(A, 256, 128)

    def call(dims=dims, q=q, k=kv, v=kv, cu_q=A, cu_k=A, n=1, tq=5, tk=5, scale=0.1, o=A, lse=None, ws=A, size=need):
        return fn("moe_attn_prefill")(ctypes.byref(dims), q, k, v, cu_q, cu_k, n, tq, tk, scale, 1, o, lse, ws, size,
                                      None)

    assert call(dims=m.AttnDims(16, 2, 80)) == 2
    assert call(n=0) == 1 and call(n=4097) == 2
    assert call(cu_q=None) == 1 and call(cu_k=None) == 1 and call(cu_q=A + 2) == 3
    assert call(tq=-1) == 1 and call(tk=-1) == 1 and call(tq=(1 << 30) + 1) == 2
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == 1, s
    assert call(o=None) == 1 and call(o=A + 8) == 3 and call(lse=A + 2) == 3
    assert call(ws=None) == 1 and call(ws=A + 64) == 3 and call(size=need - 1) == 4
    assert call(q=HeadsView(None, 2048, 128)) == 1 and call(q=HeadsView(A + 8, 2048, 128)) == 3
    assert call(k=HeadsView(A, 250, 128)) == 1                    # a stride that is not a multiple of 8
    assert call(v=HeadsView(A, 64, 128)) == 1                     # rows that overlap
    assert call(v=HeadsView(A, 256, 0)) == 1 and call(v=HeadsView(A, 1 << 38, 128)) == 1
    assert call(tq=0, q=HeadsView(None, 0, 0), o=None) == 0       # nothing to do


def test_cache_refusals(m, fn):
    from quantized_grouped_gemm_router_gb300.attention import HeadsView, KvCacheC
    dims = m.AttnDims(16, 2, 128)
    need = m.attn_workspace_bytes(dims)
    q, kv = HeadsView(A, 2048, 128), HeadsView(A, 256, 128)

    def cache(**kw):
        c = dict(dims=dims, format=0, page_size=16, n_pages=10, k=A, v=A, k_scale=None, v_scale=None)
        c.update(kw)
        return KvCacheC(*c.values())

    def append(c=None, k=kv, v=kv, cu=A, start=A, table=A, width=4, n=1, total=5, ws=A, size=need):
        return fn("moe_kv_append")(ctypes.byref(c or cache()), k, v, cu, start, table, width, n, total, ws, size, None)

    def decode(c=None, q=q, lens=A, table=A, width=4, n=1, scale=0.1, o=A, lse=None, ws=A, size=need):
        return fn("moe_attn_decode")(ctypes.byref(c or cache()), q, lens, table, width, n, scale, o, lse, ws, size, None)

    for call in (append, decode):
        assert call(cache(format=2)) == 1 and call(cache(format=1)) == 1          # e4m3 without scales
        assert call(cache(format=1, k_scale=A + 1, v_scale=A)) == 3
        assert call(cache(k=None)) == 1 and call(cache(v=A + 8)) == 3
        assert call(cache(page_size=0)) == 1 and call(cache(n_pages=0)) == 1
        assert call(cache(page_size=65537)) == 2
        assert call(cache(page_size=65536, n_pages=1 << 14)) == 2                 # 2^31 cache rows
        assert call(cache(dims=m.AttnDims(15, 2, 128))) == 2
        assert call(n=0) == 1 and call(n=4097) == 2 and call(width=0) == 1
        assert call(table=None) == 1 and call(table=A + 2) == 3
        assert call(ws=None) == 1 and call(ws=A + 16) == 3 and call(size=need - 1) == 4
    assert append(cu=None) == 1 and append(start=None) == 1 and append(start=A + 1) == 3
    assert append(total=-1) == 1 and append(total=0) == 0 and append(k=HeadsView(A, 256, 4)) == 1
    assert append(v=HeadsView(A + 2, 256, 128)) == 3
    assert decode(lens=None) == 1 and decode(lens=A + 2) == 3 and decode(o=None) == 1 and decode(o=A + 4) == 3
    assert decode(lse=A + 3) == 3 and decode(q=HeadsView(None, 2048, 128)) == 1
    for s in (0.0, -0.5, math.inf, math.nan):
        assert decode(scale=s) == 1, s


def test_binding_refuses_host_tensors(m):
    dims = m.AttnDims(4, 2, 64)
    q, kv = torch.zeros(3, 4, 64, dtype=torch.int16), torch.zeros(3, 2, 64, dtype=torch.int16)
    cu, ws = torch.tensor([0, 3], dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.attn_prefill(dims, q, kv, kv, cu, cu, ws)
    with pytest.raises(ValueError):
        m.KvCache(dims, torch.zeros(3, 2, 16, 64, dtype=torch.int16), torch.zeros(3, 2, 16, 64, dtype=torch.int16))
    with pytest.raises(ValueError):
        m.KvCache(dims, torch.zeros(3, 2, 16, 64), torch.zeros(3, 2, 16, 64))


class Placed(torch.Tensor):
    """A host tensor that says it lies on CUDA device `place`."""
    place = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.place


def place(t, dev):
    t = t.as_subclass(Placed)
    t.place = dev
    return t


def test_binding_refuses_other_devices(m, monkeypatch):
    """Every tensor of a call lies on the current device; else nothing reaches the library."""
    from quantized_grouped_gemm_router_gb300 import attention
    reached = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(attention, "_fn", lambda name: lambda *a: reached.append(name) or 0)
    dims, i16, i32 = m.AttnDims(4, 2, 64), torch.int16, torch.int32

    def rows(h):
        return torch.zeros(3, h, 64, dtype=i16)

    def cells():
        return torch.zeros(3, 2, 16, 64, dtype=torch.uint8)

    def calls():
        """name -> (call, its tensors)"""
        ws, lse = torch.zeros(256, dtype=torch.uint8), torch.zeros(3, 4)
        cu, table = torch.tensor([0, 3], dtype=i32), torch.zeros(1, 2, dtype=i32)
        kv = dict(k=cells(), v=cells(), k_scale=torch.ones(2), v_scale=torch.ones(2))
        return {
            "moe_attn_prefill": (lambda t: m.attn_prefill(dims, t["q"], t["k"], t["v"], t["cu_q"], t["cu_k"], t["ws"],
                                                          o=t["o"], lse=t["lse"]),
                                 dict(q=rows(4), k=rows(2), v=rows(2), cu_q=cu, cu_k=cu, ws=ws, o=rows(4), lse=lse)),
            "moe_kv_append": (lambda t: m.kv_append(m.KvCache(dims, *(t["c_" + n] for n in kv)), t["k"], t["v"], t["cu"],
                                                    t["start"], t["table"], t["ws"]),
                              dict({"c_" + n: x for n, x in kv.items()}, k=rows(2), v=rows(2), cu=cu,
                                   start=torch.zeros(1, dtype=i32), table=table, ws=ws)),
            "moe_attn_decode": (lambda t: m.attn_decode(m.KvCache(dims, *(t["c_" + n] for n in kv)), t["q"], t["lens"],
                                                        t["table"], t["ws"], o=t["o"], lse=t["lse"]),
                                dict({"c_" + n: x for n, x in kv.items()}, q=rows(4), lens=torch.ones(3, dtype=i32),
                                     table=torch.zeros(3, 2, dtype=i32), ws=ws, o=rows(4), lse=lse)),
        }

    for name, (call, tensors) in calls().items():
        for current in (0, 1):
            call({n: place(t, current) for n, t in tensors.items()})
            assert reached.pop() == name
            with pytest.raises(ValueError):
                call({n: place(t, 1 - current) for n, t in tensors.items()})
            for odd in tensors:
                with pytest.raises(ValueError):
                    call({n: place(t, 1 - current if n == odd else current) for n, t in tensors.items()})
                assert not reached, (name, odd)
