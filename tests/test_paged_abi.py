"""CPU tests of the paged calls' argument checks: through the C ABI with
addresses that are never dereferenced, and through the binding with stand-in
tensors.  Every refused call returns before it touches a device."""

from __future__ import annotations

import contextlib
import gc
import math
import weakref

import pytest
import torch

import causal_self_attention_flash_b200 as cattn
from causal_self_attention_flash_b200 import _binding
from test_binding_host import FakeDev, FakeLib

A = 0x10000          # 256-byte aligned, never dereferenced
L = _binding.Layout
INVALID, UNSUPPORTED = cattn.ERR_INVALID_ARG, cattn.ERR_UNSUPPORTED


def decode(sparse=False, **kw):
    a = dict(q=A, lq=L(512, 64, 64), k=A, lk=L(2048, 64, 128), v=A, lv=L(2048, 64, 128), scale=0.1,
             B=2, H=4, Hkv=2, Tq=1, D=64, n_pages=9, P=16, table=A, stride=5, width=5, lengths=A)
    if sparse:
        a.update(pages=A, K=3)
    a.update(o=A, lo=L(512, 64, 64), lse=A, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return getattr(cattn.LIB, "attn_decode_sparse" if sparse else "attn_decode_paged")(*a.values())


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(H=-4), dict(Hkv=0), dict(Hkv=3), dict(Tq=0), dict(n_pages=0), dict(P=0),
    dict(width=0), dict(width=6), dict(stride=4), dict(width=1 << 20, stride=1 << 20, P=1 << 11),
    dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(q=None), dict(k=None),
    dict(v=None), dict(table=None), dict(lengths=None), dict(o=None), dict(lse=None),
    dict(ws=None), dict(ws=A + 128), dict(ws_bytes=1000), dict(q=A + 8), dict(k=A + 2),
    dict(table=A + 2), dict(lengths=A + 1), dict(lse=A + 2), dict(lk=L(2048, 63, 128)),
    dict(lk=L(0, 64, 128)), dict(lo=L(512, 32, 64))])
def test_decode_refusals(sparse, bad):
    assert decode(sparse, **bad) == INVALID


def test_decode_refuses_more_chunks_than_it_counts():
    assert decode(B=1 << 20, width=1 << 20, stride=1 << 20) == INVALID
    assert decode(B=1 << 10, H=1 << 18, Hkv=1 << 18, width=1 << 17, stride=1 << 17) == INVALID
    assert decode(B=1, H=1 << 21, Hkv=1) == INVALID


def test_decode_counts_what_a_request_costs_beside_its_chunks():
    """the places of a request on the flat axis are its chunks and 4 (2 at D =
    128) more: their sum has to fit 32 bits, and 2^38 for all heads"""
    if torch.cuda.is_available():
        pytest.skip("the calls that are not refused would run")
    wide = dict(P=32, n_pages=9)                # D = 64: a page is a chunk

    def refused(B, width, **kw):
        return decode(B=B, width=width, stride=width, **{**wide, **kw}) == INVALID
    assert refused(64, (1 << 25) - 1) and refused(64, (1 << 25) - 4)
    assert not refused(64, (1 << 25) - 5)
    big = dict(D=128, P=16, lq=L(512, 128, 128), lo=L(512, 128, 128), lk=L(4096, 128, 256),
               lv=L(4096, 128, 256))
    assert refused(64, (1 << 25) - 2, **big) and not refused(64, (1 << 25) - 3, **big)
    heads = dict(H=1 << 12, Hkv=1 << 12, lq=L(1 << 18, 64, 64), lo=L(1 << 18, 64, 64),
                 lk=L(1 << 23, 64, 1 << 18), lv=L(1 << 23, 64, 1 << 18))
    assert refused(2, (1 << 25) - 3, **heads) and not refused(2, (1 << 25) - 4, **heads)


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_unsupported_and_empty(sparse):
    assert decode(sparse, D=48) == UNSUPPORTED
    assert decode(sparse, Tq=9) == UNSUPPORTED
    assert decode(sparse, B=0) == cattn.OK and decode(sparse, H=0) == cattn.OK


def test_sparse_refusals():
    assert decode(True, pages=None) == INVALID
    assert decode(True, K=0) == INVALID
    assert decode(True, pages=A + 2) == INVALID
    assert decode(True, K=1 << 30) == INVALID


def test_workspace_bytes():
    f = cattn.attn_decode_paged_workspace_bytes
    assert f(2, 4, 2, 1, 64) > 0 and f(2, 4, 2, 8, 64) > f(2, 4, 2, 1, 64)
    assert f(1, 4, 2, 1, 64) == f(500, 4, 2, 1, 64)        # the batch does not matter
    for bad in [(2, 4, 3, 1, 64), (2, 4, 2, 9, 64), (2, 4, 2, 0, 64), (2, 4, 2, 1, 48),
                (0, 4, 2, 1, 64), (-1, 4, 2, 1, 64), (2, 4, 0, 1, 64)]:
        assert f(*bad) == 0, bad
    g = cattn.attn_page_select_workspace_bytes
    assert g(2, 3, 100) >= 2 * 3 * 100 * 12 and g(0, 3, 100) == g(2, 0, 100) == g(2, 3, 0) == 0


def plan(**kw):
    a = dict(new=A, lengths=A, table=A, stride=5, ring=A, state=A, B=3, width=5, n_pages=9, P=16,
             n_slots=7, lengths_out=A, state_out=A, cu=A, slots=A, positions=A, status=A,
             stream=None)
    a.update(kw)
    return cattn.LIB.attn_paged_plan(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(width=0), dict(stride=4), dict(n_pages=0), dict(P=0), dict(n_slots=-1),
    dict(n_slots=1 << 31), dict(width=1 << 20, stride=1 << 20, P=1 << 11), dict(new=None),
    dict(lengths=None), dict(table=None), dict(ring=None), dict(state=None),
    dict(lengths_out=None), dict(state_out=None), dict(cu=None), dict(slots=None),
    dict(positions=None), dict(status=None), dict(state=A + 4), dict(slots=A + 4),
    dict(status=A + 2)])
def test_plan_refusals(bad):
    assert plan(**bad) == INVALID


def test_plan_request_limit():
    assert plan(B=8193) == UNSUPPORTED


def append(**kw):
    a = dict(kn=A, lkn=L(0, 64, 512), vn=A, lvn=L(0, 64, 512), n=4, Hkv=2, D=64, n_pages=9, P=16,
             slots=A, k=A, lk=L(2048, 64, 128), v=A, lv=L(2048, 64, 128), bounds=A, stream=None)
    a.update(kw)
    return cattn.LIB.attn_cache_append(*a.values())


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(Hkv=0), dict(n_pages=0), dict(P=0), dict(kn=None), dict(vn=None),
    dict(slots=None), dict(k=None), dict(v=None), dict(kn=A + 8), dict(slots=A + 4),
    dict(bounds=A + 8), dict(lkn=L(0, 64, 12)), dict(lvn=L(0, 0, 512)), dict(lk=L(2048, 64, 64)),
    dict(lv=L(8, 64, 128)), dict(n_pages=1 << 30)])
def test_append_refusals(bad):
    assert append(**bad) == INVALID


def test_append_unsupported_and_empty():
    assert append(D=40) == UNSUPPORTED
    assert append(n=0, kn=None, vn=None, slots=None) == cattn.OK


def select(**kw):
    a = dict(q=A, lq=L(512, 64, 64), bounds=A, B=2, H=4, Hkv=2, Tq=1, D=64, n_pages=9, P=16,
             table=A, stride=50, width=50, lengths=A, K=8, n_first=1, n_last=1, pages=A, ws=A,
             ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return cattn.LIB.attn_page_select(*a.values())


@pytest.mark.parametrize("bad", [
    dict(K=0), dict(n_first=-1), dict(n_last=-1), dict(n_first=8), dict(n_first=5, n_last=4),
    dict(Tq=0), dict(Hkv=3), dict(q=None), dict(bounds=None), dict(table=None),
    dict(lengths=None), dict(pages=None), dict(ws=None), dict(ws_bytes=100), dict(ws=A + 16),
    dict(bounds=A + 8), dict(pages=A + 2), dict(stride=49), dict(lq=L(512, 60, 64))])
def test_select_refusals(bad):
    assert select(**bad) == INVALID


def test_select_unsupported_and_empty():
    assert select(D=24) == UNSUPPORTED and select(Tq=9) == UNSUPPORTED
    assert select(B=0) == cattn.OK


def test_calls_by_words():
    """attn_paged_call: unknown calls, wrong counts, words that do not fit"""
    f = cattn.LIB.attn_paged_call
    assert f(-1, b"\0" * 400, 18) == INVALID and f(5, b"\0" * 400, 18) == INVALID
    for call, pack in enumerate(_binding.CALL_WORDS):
        n = pack.size // 8
        assert f(call, b"\0" * 400, n - 1) == INVALID and f(call, None, n) == INVALID
    pack = _binding.CALL_WORDS[cattn.CALL_CACHE_APPEND].pack
    ok = [A, 0, 64, 512, A, 0, 64, 512, 0, 2, 64, 9, 16, A, A, 2048, 64, 128, A, 2048, 64, 128, 0, 0]
    assert f(cattn.CALL_CACHE_APPEND, pack(*ok), 24) == cattn.OK          # no rows
    for i in (9, 10, 11, 12):
        big = list(ok)
        big[i] += 1 << 32
        assert f(cattn.CALL_CACHE_APPEND, pack(*big), 24) == INVALID


# ---------------------------------------------------------------- binding

@pytest.fixture
def fake(monkeypatch):
    lib = FakeLib(cattn.LIB)
    monkeypatch.setattr(cattn, "LIB", lib)
    monkeypatch.setattr(cattn.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(cattn, "_stream", lambda s: 77)
    return lib


def dev(*shape, dtype=torch.bfloat16, strides=None):
    return FakeDev(shape, dtype, strides)


def test_binding_hands_over_sizes_and_strides(fake):
    B, H, Hkv, Tq, D, P, n_pages, width = 2, 8, 2, 3, 64, 16, 30, 7
    q = dev(B, H, Tq, D, strides=(Tq * H * D, D, H * D, 1))
    k, v = (dev(n_pages, Hkv, P, D, strides=(P * Hkv * D, D, Hkv * D, 1)) for _ in range(2))
    table, lengths = dev(B, width, dtype=torch.int32, strides=(9, 1)), dev(B, dtype=torch.int32)
    o, lse = dev(B, H, Tq, D), dev(B, H, Tq, dtype=torch.float32)
    ws = dev(1 << 20, dtype=torch.uint8)
    pages = dev(B, Hkv, 5, dtype=torch.int32)
    cattn.attn_decode_paged(q, k, v, table, lengths, 0.25, o, lse, ws)
    cattn.attn_decode_sparse(q, k, v, table, lengths, pages, None, o, lse, ws)
    (name, (which, words, n)), (_, (which2, words2, n2)) = fake.calls
    assert name == "attn_paged_call" and (which, n, which2, n2) == (2, 32, 4, 34)
    w = _binding.CALL_WORDS[2].unpack(words)
    assert w[:4] == (q.data_ptr(), Tq * H * D, D, H * D)
    assert w[12:20] == (0.25, B, H, Hkv, Tq, D, n_pages, P)
    assert w[20:24] == (table.data_ptr(), 9, width, lengths.data_ptr())
    assert w[24:28] == (o.data_ptr(), H * Tq * D, Tq * D, D)
    assert w[28:] == (lse.data_ptr(), ws.data_ptr(), 1 << 20, 77)
    w2 = _binding.CALL_WORDS[4].unpack(words2)
    assert w2[12] == 0.125 and w2[24:26] == (pages.data_ptr(), 5)


def test_binding_refuses_before_the_call(fake):
    q, k = dev(2, 4, 1, 64), dev(9, 2, 16, 64)
    t, n = dev(2, 5, dtype=torch.int32), dev(2, dtype=torch.int32)
    o, lse, ws = dev(2, 4, 1, 64), dev(2, 4, 1, dtype=torch.float32), dev(99, dtype=torch.uint8)
    with pytest.raises(ValueError, match="v_cache: expected shape"):
        cattn.attn_decode_paged(q, k, dev(8, 2, 16, 64), t, n, 1.0, o, lse, ws)
    with pytest.raises(ValueError, match="unit last stride"):
        cattn.attn_decode_paged(dev(2, 4, 1, 64, strides=(256, 64, 64, 2)), k, k, t, n, 1.0, o, lse, ws)
    with pytest.raises(ValueError, match="block_table"):
        cattn.attn_decode_paged(q, k, k, dev(3, 5, dtype=torch.int32), n, 1.0, o, lse, ws)
    with pytest.raises(ValueError, match="lengths"):
        cattn.attn_decode_paged(q, k, k, t, dev(2, dtype=torch.int64), 1.0, o, lse, ws)
    with pytest.raises(ValueError, match="pages"):
        cattn.attn_decode_sparse(q, k, k, t, n, dev(2, 4, 3, dtype=torch.int32), 1.0, o, lse, ws)
    with pytest.raises(ValueError, match="k_new"):
        cattn.attn_cache_append(dev(3, 4, 64), dev(3, 2, 64), k, k, dev(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="slots"):
        cattn.attn_cache_append(dev(3, 2, 64), dev(3, 2, 64), k, k, dev(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="bounds"):
        cattn.attn_page_select(q, dev(9, 2, 3, 64), t, n, 16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        cattn.attn_decode_paged(torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16), k, k, t, n)
    assert fake.calls == []


def test_sparse_needs_its_lists(fake, monkeypatch):
    """attn_decode_sparse without lists is refused; the marshalling never sees
    it (there, no lists means the dense call)"""
    class Dense:
        def decode(self, *args):
            return 0
    monkeypatch.setattr(cattn, "TORCH_CALLS", Dense())
    q, k = dev(2, 4, 1, 64), dev(9, 2, 16, 64)
    t, n = dev(2, 5, dtype=torch.int32), dev(2, dtype=torch.int32)
    o, lse, ws = dev(2, 4, 1, 64), dev(2, 4, 1, dtype=torch.float32), dev(99, dtype=torch.uint8)
    with pytest.raises(ValueError, match="pages"):
        cattn.attn_decode_sparse(q, k, k, t, n, None, 1.0, o, lse, ws)
    with pytest.raises(ValueError, match="pages"):
        cattn.attn_decode_sparse(q, k, k, t, n, dev(2, 6, dtype=torch.int32))
    assert fake.calls == []


def test_binding_needs_the_current_device(fake, monkeypatch):
    monkeypatch.setattr(cattn.torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        cattn.attn_cache_append(dev(3, 2, 64), dev(3, 2, 64), dev(9, 2, 16, 64), dev(9, 2, 16, 64),
                                dev(3, dtype=torch.int64))
    assert fake.calls == []


def test_torch_calls_leave_foreign_tensors_to_the_long_way():
    t = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    assert cattn.TORCH_CALLS.decode(t, t, t, t, t, None, 1.0, t, t, t) == -1
    assert cattn.TORCH_CALLS.decode(*[None] * 10) == -1
    assert cattn.TORCH_CALLS.append(1, 2) == -1
    assert cattn.TORCH_CALLS.plan(*["x"] * 13) == -1
    assert cattn.TORCH_CALLS.select(*[t] * 10) == -1


def paged_calls(stream):
    """every paged call with nothing given that it can allocate itself"""
    i32, i64 = torch.int32, torch.int64
    q, k = dev(2, 4, 1, 64), dev(9, 2, 16, 64)
    t, n = dev(2, 5, dtype=i32), dev(2, dtype=i32)
    yield 6, lambda: cattn.attn_paged_plan(n, n, t, dev(9, dtype=i32), dev(2, dtype=i64), 16, 3,
                                           stream=stream)
    yield 3, lambda: cattn.attn_decode_paged(q, k, k, t, n, stream=stream)
    yield 3, lambda: cattn.attn_decode_sparse(q, k, k, t, n, dev(2, 2, 3, dtype=i32), stream=stream)
    yield 2, lambda: cattn.attn_page_select(q, dev(9, 2, 2, 64), t, n, 16, 3, stream=stream)


@pytest.mark.parametrize("stream", ["none", "object", "handle"])
def test_allocations_live_until_the_call_and_belong_to_its_stream(fake, monkeypatch, stream):
    """what a paged call allocates (outputs, workspace) is held when the library
    is called, and was allocated under the stream that the call is made on"""
    new, current, seen = [], [None], []

    class Stream:                               # stands in for torch.cuda.Stream
        def __init__(self, handle=99, device=None):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def under(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def empty(shape, dtype, device):
        t = dev(*shape, dtype=dtype)
        new.append((weakref.ref(t), current[-1]))
        return t

    def call(*args):
        gc.collect()
        seen.append([(ref() is not None, s) for ref, s in new])
        return 0
    monkeypatch.setattr(cattn, "_stream", lambda s: getattr(s, "cuda_stream", s) or 0)
    monkeypatch.setattr(cattn.torch, "empty", empty)
    monkeypatch.setattr(cattn.torch.cuda, "stream", under)
    monkeypatch.setattr(cattn.torch.cuda, "Stream", Stream)
    monkeypatch.setattr(cattn.torch.cuda, "ExternalStream", Stream)
    fake.attn_paged_call = call
    given, on = {"none": (None, None), "object": (Stream(55), 55), "handle": (66, 66)}[stream]
    for count, make in paged_calls(given):
        new.clear()
        make()
        assert seen[-1] == [(True, on)] * count
