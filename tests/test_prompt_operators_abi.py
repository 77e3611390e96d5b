"""Refusals of the prompt and training operators' C ABI, and of the binding's own
checks: every call fails before the device is touched, so no GPU is needed."""
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


def i64s(*v):
    return (ctypes.c_int64 * len(v))(*v)


WS = 128 * MIB


def prompt(lib, form="plain", **kw):
    cached = form == "cached"
    a = dict(q=ranks(1), qs=512, k=ranks(2))
    if not cached:
        a.update(ks=128)
    a.update(v=ranks(3))
    if not cached:
        a.update(vs=128)
    a.update(n=2, tokens=10, heads=8, kv=2, d=64, dtype=1)
    if cached:
        a.update(pages=16, page=16, table=at(4), ts=8, blocks=8)
    a.update(starts=at(5))
    if cached:
        a.update(lens=at(6))
    a.update(sequences=3, scale=0.1, out=ranks(7), outs=512, lse=ranks(8))
    if form == "backward":
        a.update(dout=ranks(9), douts=512, dq=ranks(10), dqs=512, dk=ranks(11), dks=128, dv=ranks(12), dvs=128)
    a.update(ws=at(13), bytes=WS)
    assert set(kw) <= set(a), kw
    a.update(kw)
    name = {"plain": "", "cached": "_cached", "backward": "_backward"}[form]
    return getattr(lib, "rar_prompt_attention" + name)(*a.values(), None)


@pytest.mark.parametrize("form", ["plain", "cached", "backward"])
def test_prompt_refusals(lib, form):
    bad = [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(n=0), dict(n=33), dict(tokens=-1),
           dict(tokens=1 << 28), dict(heads=7), dict(heads=0), dict(kv=0), dict(heads=1025, kv=1025), dict(d=4), dict(d=260),
           dict(d=264), dict(dtype=2), dict(sequences=-1), dict(sequences=1 << 28), dict(starts=0), dict(qs=504),
           dict(outs=504), dict(ws=at(1))]
    if form == "backward":
        bad += [dict(lse=None), dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(douts=504), dict(dks=120),
                dict(dq=ranks(1)), dict(dk=ranks(2)), dict(dv=ranks(11)), dict(dq=ranks(7)), dict(dv=ranks(9)),
                dict(dk=ranks(8))]
    else:
        bad += [dict(out=ranks(1)), dict(out=ranks(2)), dict(lse=ranks(7)), dict(lse=ranks(3))]
    if form == "cached":
        bad += [dict(page=0), dict(page=24), dict(page=2048), dict(pages=0), dict(pages=1 << 28), dict(blocks=0), dict(ts=7),
                dict(table=0), dict(lens=0), dict(blocks=1 << 28, ts=1 << 28)]
    else:
        bad += [dict(ks=120), dict(vs=120)]
    for b in bad:
        assert prompt(lib, form, **b) == S.ERR_ARG, b
    for b in (dict(starts=at(5) + 2), dict(qs=516), dict(ws=at(13) + 64), dict(k=(ctypes.c_void_p * 2)(at(2) + 8, at(2) + MIB))):
        assert prompt(lib, form, **b) == S.ERR_ALIGN, b
    assert prompt(lib, form, bytes=4096) == S.ERR_WORKSPACE
    assert prompt(lib, form, ws=0) == S.ERR_WORKSPACE
    # the size that the query says fits, one byte less does not
    need = lib.rar_prompt_attention_workspace_bytes(2, 10, 8, 2, 64)
    assert prompt(lib, form, bytes=need - 1) == S.ERR_WORKSPACE
    # nothing to do: no tensors either
    assert prompt(lib, form, tokens=0) == S.OK
    assert prompt(lib, form, sequences=0) == S.OK


def test_prompt_workspace_bytes(lib):
    f = lib.rar_prompt_attention_workspace_bytes
    for bad in ((0, 10, 8, 2, 64), (33, 10, 8, 2, 64), (2, -1, 8, 2, 64), (2, 10, 7, 2, 64), (2, 10, 8, 2, 60),
                (2, 1 << 29, 8, 2, 64), (2, 10, 2048, 2, 64)):
        assert f(*bad) == 0, bad
    assert f(1, 0, 8, 2, 64) >= B.OP_WORKSPACE_MIN_BYTES
    # delta of the gradient, a float a row
    assert f(4, 100000, 32, 8, 128) >= B.OP_WORKSPACE_MIN_BYTES + 4 * 100000 * 32 * 4


def test_workspaces_serve_fewer_tokens(lib):
    """A workspace for the largest call is one for every smaller one, though only small calls are split."""
    counts = sorted({n + d for k in range(17) for n in (1 << k, 5 << k, 19 * k * k) for d in (-1, 0, 1) if n + d >= 0})
    for n, heads, kv, dim in ((1, 8, 1, 128), (2, 16, 4, 64), (8, 64, 8, 128), (1, 4, 4, 256), (1, 130, 1, 80), (1, 1, 1, 8), (32, 32, 32, 64)):
        need = [lib.rar_prompt_attention_workspace_bytes(n, t, heads, kv, dim) for t in counts]
        assert need == sorted(need) and need[0] >= B.OP_WORKSPACE_MIN_BYTES, (n, heads, kv, dim)
    for hidden in (8, 64, 512, 4096, 1 << 20):
        need = [lib.rar_embed_tokens_workspace_bytes(t, hidden) for t in counts]
        assert need == sorted(need) and need[0] >= B.OP_WORKSPACE_MIN_BYTES, hidden


def test_prompt_gradients_side_by_side(lib):
    """dq, dk and dv in one buffer (qkv's gradient) are apart; shifted into one another they are not."""
    parts = dict(dq=ranks(10), dk=(ctypes.c_void_p * 2)(*[at(10) + r * 64 * MIB + 1024 for r in range(2)]),
                 dv=(ctypes.c_void_p * 2)(*[at(10) + r * 64 * MIB + 1280 for r in range(2)]), dqs=768, dks=768, dvs=768)
    assert prompt(lib, "backward", bytes=4096, **parts) == S.ERR_WORKSPACE  # past the check of what meets what
    parts["dv"] = parts["dk"]
    assert prompt(lib, "backward", bytes=4096, **parts) == S.ERR_ARG


def embed(lib, **kw):
    a = dict(tokens=at(1), count=10, tables=ranks(2), vocab=i64s(100, 50), strides=i64s(64, 72), n=2, hidden=64, dtype=1,
             scale=1.0, out=at(3), outs=64, ws=at(4), bytes=MIB)
    a.update(kw)
    return lib.rar_embed_tokens(*a.values(), None)


def embed_backward(lib, **kw):
    a = dict(tokens=at(1), count=10, dout=at(3), outs=64, dtype=1, scale=1.0, tables=ranks(2), vocab=i64s(100, 50),
             strides=i64s(64, 72), n=2, hidden=64, accumulate=0, ws=at(4), bytes=MIB)
    a.update(kw)
    return lib.rar_embed_tokens_backward(*a.values(), None)


def test_embed_refusals(lib):
    for call in (embed, embed_backward):
        for bad in (dict(tables=None), dict(vocab=None), dict(strides=None), dict(n=0), dict(n=33), dict(count=-1),
                    dict(dtype=3), dict(tokens=0), dict(hidden=0), dict(hidden=60), dict(hidden=1 << 21), dict(outs=56),
                    dict(strides=i64s(56, 64)), dict(vocab=i64s(0, 5)), dict(vocab=i64s(1 << 30, 1 << 30)),
                    dict(count=1 << 31), dict(ws=at(2)), dict(tables=(ctypes.c_void_p * 2)(at(2), None))):
            assert call(lib, **bad) == S.ERR_ARG, (call, bad)
        for bad in (dict(tokens=at(1) + 2), dict(outs=68), dict(strides=i64s(66, 72)), dict(ws=at(4) + 8),
                    dict(tables=(ctypes.c_void_p * 2)(at(2) + 8, at(2) + MIB))):
            assert call(lib, **bad) == S.ERR_ALIGN, (call, bad)
        assert call(lib, bytes=100) == S.ERR_WORKSPACE
        assert call(lib, ws=0) == S.ERR_WORKSPACE
    for bad in (dict(out=0), dict(out=at(2)), dict(out=at(1))):
        assert embed(lib, **bad) == S.ERR_ARG, bad
    for bad in (dict(dout=0), dict(tables=ranks(3)), dict(tables=(ctypes.c_void_p * 2)(at(2), at(2) + 64))):
        assert embed_backward(lib, **bad) == S.ERR_ARG, bad
    assert lib.rar_embed_tokens_workspace_bytes(-1, 64) == 0
    assert lib.rar_embed_tokens_workspace_bytes(10, 12) == 0
    assert lib.rar_embed_tokens_workspace_bytes(1 << 31, 64) == 0
    need = lib.rar_embed_tokens_workspace_bytes(10, 64)
    assert embed_backward(lib, bytes=need - 1) == S.ERR_WORKSPACE
    assert embed(lib, count=0) == S.OK


class OnDevice:
    """A host tensor that says it is in device memory: for calls that must be refused before any launch."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


class Ws:
    ptr, nbytes = at(0), MIB


def tensors(torch):
    return lambda *s, dtype=torch.float32: OnDevice(torch.zeros(*s, dtype=dtype))


@pytest.mark.parametrize("bad", [
    dict(q=lambda d: d(2, 9, 8, 32)), dict(q=lambda d: d(9, 8, 64)), dict(q=lambda d: d(33, 9, 8, 64)), dict(q=[]),
    dict(k=lambda d: d(2, 9, 2, 32)), dict(k=lambda d: d(2, 8, 2, 64)), dict(k=lambda d: d(2, 9, 4, 64)),
    dict(v=lambda d: d(1, 9, 2, 64)), dict(v=lambda d: OnDevice(d(2, 9, 64, 2).t.transpose(2, 3))),
    dict(out=lambda d: d(2, 9, 4, 64)), dict(lse=lambda d: d(2, 9, 4)), dict(lse=lambda d: OnDevice(d(2, 9, 16).t[..., ::2])),
    dict(starts=lambda d: d(0)),
], ids=str)
def test_binding_refuses_what_does_not_fit(lib, bad):
    torch = pytest.importorskip("torch")
    d = tensors(torch)
    i32 = lambda *s: d(*s, dtype=torch.int32)  # noqa: E731
    a = dict(q=d(2, 9, 8, 64), k=d(2, 9, 2, 64), v=d(2, 9, 2, 64), starts=i32(3), out=d(2, 9, 8, 64), lse=d(2, 9, 8))
    a.update({k: v(d) if callable(v) else v for k, v in bad.items()})
    if "starts" in bad:
        a["starts"] = i32(0)
    with pytest.raises(B.RarError) as e:
        B.prompt_attention(*a.values(), Ws, stream=0)
    assert e.value.status == S.ERR_ARG
    b = dict(a, dout=d(2, 9, 8, 64), dq=d(2, 9, 8, 64), dk=d(2, 9, 2, 64), dv=d(2, 9, 2, 64))
    with pytest.raises(B.RarError) as e:
        B.prompt_attention_backward(*b.values(), Ws, stream=0)
    assert e.value.status == S.ERR_ARG


def test_binding_refuses_other_operands(lib):
    torch = pytest.importorskip("torch")
    d = tensors(torch)
    i32 = lambda *s: d(*s, dtype=torch.int32)  # noqa: E731
    q, cache = d(2, 9, 8, 64), d(2, 4, 2, 16, 64)
    ok = dict(q=q, k=cache, v=cache, table=i32(3, 4), starts=i32(4), lens=i32(3), out=d(2, 9, 8, 64), lse=None)
    for bad in (dict(k=d(2, 4, 2, 16, 32)), dict(v=d(2, 5, 2, 16, 64)), dict(table=i32(2, 4)), dict(lens=i32(4)),
                dict(starts=i32(3)), dict(table=d(3, 4)), dict(out=d(2, 8, 8, 64))):
        with pytest.raises(B.RarError) as e:
            B.prompt_attention_cached(*{**ok, **bad}.values(), Ws, stream=0)
        assert e.value.status == S.ERR_ARG
    for tables, out in ((d(2, 50, 64), d(9, 32)), (d(2, 50, 64), d(8, 64)), ([d(50, 64), d(20, 32)], d(9, 64)),
                        (d(2, 50, 64), d(9, 64, dtype=torch.bfloat16)), (d(50, 64), d(9, 64)),
                        (d(2, 50, 64), OnDevice(d(64, 9).t.t()))):
        with pytest.raises(B.RarError) as e:
            B.embed_tokens(i32(9), tables, out, Ws, stream=0)
        assert e.value.status == S.ERR_ARG
    with pytest.raises(B.RarError):  # gradients of the tables are float32
        B.embed_tokens_backward(i32(9), d(9, 64), d(2, 50, 64, dtype=torch.bfloat16), Ws, stream=0)
    with pytest.raises(B.RarError):  # host tensors
        B.embed_tokens(torch.zeros(9, dtype=torch.int32), d(2, 50, 64), d(9, 64), Ws, stream=0)
    for dtype in (torch.float16, torch.float64):
        with pytest.raises(TypeError):
            B.embed_tokens(i32(9), d(2, 50, 64, dtype=dtype), d(9, 64, dtype=dtype), Ws, stream=0)
        with pytest.raises(TypeError):
            B.prompt_attention(d(2, 9, 8, 64, dtype=dtype), q, q, i32(3), q, None, Ws, stream=0)
