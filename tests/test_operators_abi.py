"""Refusals of the operators' C ABI, and of the binding's own checks: every call
fails before the device is touched, so no GPU is needed."""
import ctypes

import pytest

from collective_communication_gb300 import binding as B

S = B.Status
MIB = 1 << 20
BASE = 1 << 40  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from collective_communication_gb300 import build
    build.build()
    return B.load_library()


def at(i):
    return BASE + i * 256 * MIB


def ranks(first, n=2, step=64 * MIB):
    return (ctypes.c_void_p * n)(*[at(first) + r * step for r in range(n)])


def tables(lib, **kw):
    a = dict(lens=at(1), new=at(2), n=4, free=at(3), num_free=10, count=at(4), page=16, pages=64, table=at(5), stride=8,
             blocks=8, lens_out=at(6), starts=at(7), positions=at(8), slots=at(9), tokens=32, count_out=at(10), ws=at(11),
             bytes=MIB)
    a.update(kw)
    return lib.rar_page_tables(*a.values(), None)


def test_page_tables_refusals(lib):
    for bad in (dict(n=-1), dict(num_free=-1), dict(tokens=-1), dict(blocks=0), dict(page=0), dict(page=24),
                dict(page=2048), dict(pages=0), dict(pages=1 << 28), dict(stride=7), dict(blocks=1 << 28, stride=1 << 28),
                dict(lens=0), dict(new=0), dict(free=0), dict(count=0), dict(table=0), dict(lens_out=0), dict(starts=0),
                dict(positions=0), dict(slots=0), dict(count_out=0), dict(lens_out=at(1)), dict(count_out=at(4)),
                dict(slots=at(8) + 4), dict(table=at(3)), dict(ws=at(5))):
        assert tables(lib, **bad) == S.ERR_ARG, bad
    assert tables(lib, lens=at(1) + 2) == S.ERR_ALIGN
    assert tables(lib, ws=0) == S.ERR_WORKSPACE
    assert tables(lib, ws=at(11) + 16) == S.ERR_ALIGN
    assert tables(lib, bytes=1000) == S.ERR_WORKSPACE


def rope(lib, form="plain", **kw):
    a = dict(qkv=ranks(1), n=2, tokens=10, stride=640, wq=at(2), wk=at(3), cs=at(4), max_pos=100, rot=64, inter=0,
             pos=at(5))
    if form == "cached":
        a["slots"] = at(6)
    a.update(q=8, kv=1, d=64, dtype=1, eps=1e-6)
    if form == "backward":
        a.update(dq=ranks(7), dqs=512, dk=ranks(8), dks=64, dv=ranks(9), dvs=64, dx=ranks(10), dxs=640,
                 dwq=ranks(11), dwk=ranks(12))
    else:
        a.update(out=ranks(7), outs=512)
        a.update(dict(k=ranks(8), v=ranks(9), pages=4, page=16) if form == "cached" else dict(k=ranks(8), ks=64))
    a.update(ws=at(13), bytes=16 * MIB)
    assert set(kw) <= set(a), kw
    a.update(kw)
    name = {"plain": "rar_qk_norm_rope", "cached": "rar_qk_norm_rope_cached", "backward": "rar_qk_norm_rope_backward"}
    return getattr(lib, name[form])(*a.values(), None)


@pytest.mark.parametrize("form", ["plain", "cached", "backward"])
def test_norm_rope_refusals(lib, form):
    bad = [dict(n=0), dict(n=33), dict(dtype=2), dict(tokens=-1), dict(tokens=1 << 31), dict(d=60), dict(d=264),
           dict(d=0), dict(q=0), dict(kv=0), dict(q=1025), dict(rot=0), dict(rot=4), dict(rot=20), dict(rot=72),
           dict(max_pos=0), dict(wq=0), dict(wk=0), dict(cs=0), dict(pos=0), dict(qkv=None), dict(stride=632)]
    if form == "backward":
        bad += [dict(dq=None), dict(dx=ranks(1)), dict(dx=ranks(7)), dict(dwq=ranks(12)), dict(dvs=56), dict(dxs=632)]
        assert rope(lib, form, bytes=B.OP_WORKSPACE_MIN_BYTES) == S.ERR_WORKSPACE
        assert rope(lib, form, dxs=644) == S.ERR_ALIGN
    else:
        bad += [dict(out=None), dict(outs=504), dict(out=ranks(1)), dict(k=ranks(1)), dict(k=ranks(7)),
                dict(out=ranks(1), outs=648)]
        assert rope(lib, form, outs=516) == S.ERR_ALIGN
    if form == "cached":
        bad += [dict(slots=0), dict(page=12), dict(pages=0), dict(v=None), dict(v=ranks(8)), dict(pages=1 << 28)]
    for b in bad:
        assert rope(lib, form, **b) == S.ERR_ARG, b
    for b in (dict(wq=at(2) + 4), dict(cs=at(4) + 4), dict(pos=at(5) + 2), dict(stride=644),
              dict(qkv=(ctypes.c_void_p * 2)(at(1) + 2, at(1) + MIB)), dict(ws=at(13) + 128)):
        assert rope(lib, form, **b) == S.ERR_ALIGN, b
    assert rope(lib, form, ws=0) == S.ERR_WORKSPACE


def attention(lib, **kw):
    a = dict(q=ranks(1), qs=512, k=ranks(2), v=ranks(3), n=2, batch=4, heads=8, kv=2, d=64, dtype=1, pages=16, page=16,
             table=at(4), ts=8, blocks=8, lens=at(5), scale=0.1, out=ranks(6), outs=512, lse=ranks(7), ws=at(8),
             bytes=128 * MIB)
    a.update(kw)
    return lib.rar_decode_attention(*a.values(), None)


def test_attention_refusals(lib):
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(n=0), dict(n=33), dict(batch=-1),
                dict(heads=7), dict(heads=0), dict(kv=0), dict(d=4), dict(d=260), dict(dtype=9), dict(page=3),
                dict(pages=0), dict(pages=1 << 28), dict(blocks=0), dict(ts=7), dict(table=0), dict(lens=0), dict(qs=504),
                dict(outs=504), dict(out=ranks(1)), dict(out=ranks(2)), dict(lse=ranks(6)), dict(ws=at(3))):
        assert attention(lib, **bad) == S.ERR_ARG, bad
    for bad in (dict(qs=516), dict(table=at(4) + 1), dict(lens=at(5) + 2), dict(ws=at(8) + 64),
                dict(k=(ctypes.c_void_p * 2)(at(2) + 8, at(2) + MIB))):
        assert attention(lib, **bad) == S.ERR_ALIGN, bad
    assert attention(lib, bytes=4096) == S.ERR_WORKSPACE
    assert attention(lib, ws=0) == S.ERR_WORKSPACE
    assert lib.rar_decode_attention_workspace_bytes(2, 4, 7, 2, 64) == 0
    assert lib.rar_decode_attention_workspace_bytes(0, 4, 8, 2, 64) == 0
    assert lib.rar_decode_attention_workspace_bytes(2, 4, 8, 2, 64) >= B.OP_WORKSPACE_MIN_BYTES


def i64s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def logprobs(lib, **kw):
    a = dict(x=ranks(1), vocab=i64s(100, 101), strides=i64s(100, 110), n=2, rows=3, dtype=0, tokens=at(2), lp=at(3),
             entropy=at(4), lse=at(5), top=5, values=at(6), ids=at(7), ws=at(8), bytes=64 * MIB)
    a.update(kw)
    return lib.rar_token_logprobs(*a.values(), None)


def logprobs_backward(lib, **kw):
    a = dict(x=ranks(1), vocab=i64s(100, 101), strides=i64s(100, 110), n=2, rows=3, dtype=0, tokens=at(2), lse=at(3),
             entropy=at(4), gl=at(5), gh=at(6), dx=ranks(7), dstrides=i64s(100, 110), ws=at(8), bytes=MIB)
    a.update(kw)
    return lib.rar_token_logprobs_backward(*a.values(), None)


def test_logprobs_refusals(lib):
    for call in (logprobs, logprobs_backward):
        for bad in (dict(x=None), dict(vocab=None), dict(strides=None), dict(n=0), dict(n=33), dict(rows=-1),
                    dict(dtype=5), dict(tokens=0), dict(lse=0), dict(entropy=0), dict(vocab=i64s(0, 5)),
                    dict(vocab=i64s(1 << 30, 1 << 30), strides=i64s(1 << 30, 1 << 30), rows=1),
                    dict(strides=i64s(99, 110))):
            assert call(lib, **bad) == S.ERR_ARG, (call, bad)
        for bad in (dict(tokens=at(2) + 1), dict(ws=at(8) + 1), dict(x=(ctypes.c_void_p * 2)(at(1) + 2, at(1) + MIB))):
            assert call(lib, **bad) == S.ERR_ALIGN, (call, bad)
        assert call(lib, bytes=100) == S.ERR_WORKSPACE
        assert call(lib, ws=0) == S.ERR_WORKSPACE
    for bad in (dict(top=-1), dict(top=33), dict(values=0), dict(ids=0), dict(lp=0), dict(lp=at(1)), dict(lse=at(4)),
                dict(ids=at(6) + 4), dict(vocab=i64s(2, 1), strides=i64s(2, 1))):
        assert logprobs(lib, **bad) == S.ERR_ARG, bad
    for bad in (dict(gl=0), dict(dx=None), dict(dstrides=i64s(99, 110)), dict(dx=ranks(1), dstrides=i64s(104, 110)),
                dict(dx=ranks(2))):
        assert logprobs_backward(lib, **bad) == S.ERR_ARG, bad
    assert lib.rar_token_logprobs_workspace_bytes(3, 33) == 0
    assert lib.rar_token_logprobs_workspace_bytes(-1, 3) == 0


def test_binding_refuses_host_tensors_and_shapes(lib):
    torch = pytest.importorskip("torch")

    class Ws:
        ptr, nbytes = at(0), MIB

    x = torch.zeros(2, 3, 8, 64)
    cache = torch.zeros(2, 4, 2, 16, 64)
    table, lens = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(B.RarError) as e:
        B.decode_attention(x, cache, cache, table, lens, x, None, Ws)
    assert e.value.status == S.ERR_ARG
    with pytest.raises(B.RarError):
        B.token_logprobs([torch.zeros(3, 5)], lens, lens, lens, lens, None, None, Ws)
    with pytest.raises(B.RarError):
        B.page_tables(lens, lens, lens, lens[:1], table, 16, 64, lens, lens, lens, lens, lens[:1], Ws)
    with pytest.raises(B.RarError):
        B.qk_norm_rope(torch.zeros(2, 3, 640), x[0, 0, 0], x[0, 0, 0], torch.zeros(4, 64), lens, x, x[:, :, :1], Ws)


class OnDevice:
    """A host tensor that says it is in device memory: for calls that must be refused before any launch."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


class Ws:
    ptr, nbytes = at(0), MIB


def attention_call(torch, **kw):
    d = lambda *s, dtype=torch.float32: OnDevice(torch.zeros(*s, dtype=dtype))
    i32 = torch.int32
    a = dict(q=d(2, 3, 8, 64), k=d(2, 4, 2, 16, 64), v=d(2, 4, 2, 16, 64), table=d(3, 4, dtype=i32), lens=d(3, dtype=i32),
             out=d(2, 3, 8, 64), lse=d(2, 3, 8))
    a.update({k: v(d) if callable(v) else v for k, v in kw.items()})
    B.decode_attention(*a.values(), Ws, stream=0)


@pytest.mark.parametrize("bad", [
    dict(q=lambda d: d(2, 3, 8, 32)), dict(q=lambda d: d(3, 8, 64)), dict(q=lambda d: d(2, 2, 8, 64)),
    dict(q=lambda d: d(33, 3, 8, 64)), dict(q=lambda d: [d(3, 8, 64)]), dict(q=lambda d: [d(3, 8, 64), d(3, 8, 63)]),
    dict(q=[]), dict(q=lambda d: [d(3, 8, 64)] * 33), dict(q=lambda d: d(1, 1, 1, 1, 2, 3, 8, 64)),
    dict(q=lambda d: OnDevice(d(2, 3, 64, 8).t.transpose(2, 3))),
    dict(k=lambda d: d(2, 4, 2, 16, 32)), dict(v=lambda d: d(2, 5, 2, 16, 64)),
    dict(k=lambda d: OnDevice(d(2, 8, 2, 16, 64).t[:, ::2]), v=lambda d: OnDevice(d(2, 8, 2, 16, 64).t[:, ::2])),
    dict(table=lambda d: d(3, 4)), dict(table=lambda d: OnDevice(d(4, 3).t.int().t())), dict(lens=lambda d: d(3)),
    dict(out=lambda d: d(2, 3, 8, 32)), dict(lse=lambda d: d(2, 3, 4)), dict(lse=lambda d: OnDevice(d(2, 3, 16).t[..., ::2])),
], ids=str)
def test_binding_refuses_what_does_not_fit(lib, bad):
    torch = pytest.importorskip("torch")
    with pytest.raises(B.RarError) as e:
        attention_call(torch, **bad)
    assert e.value.status == S.ERR_ARG


def test_binding_refuses_dtypes(lib):
    torch = pytest.importorskip("torch")
    for dtype in (torch.float16, torch.int32, torch.float64):
        with pytest.raises(TypeError):
            attention_call(torch, q=lambda d: d(2, 3, 8, 64, dtype=dtype))
        with pytest.raises(B.RarError):
            attention_call(torch, k=lambda d: d(2, 4, 2, 16, 64, dtype=dtype))
    with pytest.raises(AttributeError):
        attention_call(torch, q=5)


def test_binding_reads_a_list_that_shrinks(lib):
    """Reading a tensor-like may run Python; the list it is in may change meanwhile."""
    torch = pytest.importorskip("torch")
    queries = []

    class Shrinks(OnDevice):
        def data_ptr(self):
            del queries[1:]
            return 0

    queries += [Shrinks(torch.zeros(3, 8, 64)) for _ in range(4)]
    with pytest.raises(IndexError):
        attention_call(torch, q=queries)


def test_binding_refuses_numbers_past_the_abi(lib):
    torch = pytest.importorskip("torch")
    i32 = lambda *s: OnDevice(torch.zeros(*s, dtype=torch.int32))
    for page_size, pages in ((2**32 + 16, 64), (16, 2**32 + 64), (-16, 64), (16, -1), (12, 64)):
        with pytest.raises(B.RarError) as e:
            B.page_tables(i32(3), i32(3), i32(9), i32(1), i32(3, 4), page_size, pages, i32(3), i32(4), i32(5), i32(5), i32(1),
                          Ws, stream=0)
        assert e.value.status == S.ERR_ARG
