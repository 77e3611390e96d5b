"""Layouts that the prompt operators take and refuse, without a GPU: a call that gets as far as its workspace, which is
too small, has passed every check of its tensors."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from collective_communication_gb300 import binding as B
from test_prompt_operators_abi import BASE, MIB, OnDevice

S = B.Status
N, T, HEADS, KV, D = 2, 9, 8, 2, 64


@pytest.fixture(scope="module", autouse=True)
def lib():
    from collective_communication_gb300 import build
    build.build()
    return B.load_library()


class Ws:
    ptr, nbytes = BASE, 4096


def status(name, a):
    with pytest.raises(B.RarError) as e:
        getattr(B, name)(*[OnDevice(x) if isinstance(x, torch.Tensor) else x for x in a], Ws, stream=0)
    return e.value.status


def by_head(*shape):
    """[ranks, tokens, heads, d] whose heads are d * tokens apart."""
    n, t, h, d = shape
    return torch.zeros(n, h, t, d).transpose(1, 2)


def by_token(*shape):
    return torch.zeros(*shape)


def interleaved(t):
    """Queries, keys and values of as many heads, a head's three side by side."""
    return torch.zeros(N, t, KV, 3, D).unbind(3)


def gradient(t=T, make=by_head):
    q, k = make(N, t, HEADS, D), make(N, t, KV, D)
    like = lambda x: make(*x.shape)  # noqa: E731
    starts = torch.tensor([0, t], dtype=torch.int32)
    return dict(q=q, k=k, v=like(k), starts=starts, out=like(q), lse=torch.zeros(N, t, HEADS), dout=like(q), dq=like(q), dk=like(k),
                dv=like(k))


@pytest.mark.parametrize("t", [1, 2, T])
@pytest.mark.parametrize("name", ["q", "k", "v", "out", "dout", "dq", "dk", "dv", "all"])
def test_tensors_laid_out_by_head(name, t):
    a = gradient(t, by_head if name == "all" else by_token)
    if name != "all":
        a[name] = gradient(t)[name]
    assert status("prompt_attention_backward", a.values()) == S.ERR_WORKSPACE
    assert status("prompt_attention", list(a.values())[:6]) == S.ERR_WORKSPACE
    cache = torch.zeros(N, 4, KV, 16, D)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    assert status("prompt_attention_cached", (a["q"], cache, cache, table, a["starts"], lens, a["out"], a["lse"])) == S.ERR_WORKSPACE


@pytest.mark.parametrize("t", [1, 2, T])
def test_gradients_interleaved_by_head(t):
    a = gradient(t, by_token)
    a.update(zip(("q", "k", "v"), interleaved(t)), lse=torch.zeros(N, t, KV), out=by_head(N, t, KV, D), dout=by_head(N, t, KV, D))
    a.update(zip(("dq", "dk", "dv"), interleaved(t)))
    assert status("prompt_attention_backward", a.values()) == S.ERR_WORKSPACE
    for x, y in (("dq", "dk"), ("dk", "dv"), ("dv", "q"), ("dq", "v")):
        assert status("prompt_attention_backward", dict(a, **{x: a[y]}).values()) == S.ERR_ARG, (x, y)
    # the ranks side by side in one row
    buffer = torch.zeros(t, N, KV, 3, D)
    a.update((x, [OnDevice(buffer[:, r, :, i]) for r in range(N)]) for i, x in enumerate(("dq", "dk", "dv")))
    assert status("prompt_attention_backward", a.values()) == S.ERR_WORKSPACE
    a["dk"] = a["dk"][::-1]
    assert status("prompt_attention_backward", a.values()) == S.ERR_WORKSPACE
    a["dk"] = a["dq"][::-1]
    assert status("prompt_attention_backward", a.values()) == S.ERR_ARG


@pytest.mark.parametrize("bad,want", [
    (lambda x: x[:, :, :1].expand(N, T, HEADS, D), S.ERR_ARG),                                    # one head for all
    (lambda x: x[:, :1].expand(N, T, HEADS, D), S.ERR_ARG),                                       # one token for all
    (lambda x: torch.zeros(N, T, D, HEADS).transpose(2, 3), S.ERR_ARG),                           # heads that are not dense
    (lambda x: torch.zeros(99999).as_strided((N, T, HEADS, D), (9000, D // 2, T * D, 1)), S.ERR_ARG),  # rows into one another
    (lambda x: torch.zeros(99999).as_strided((N, T, HEADS, D), (9000, D, (T - 1) * D, 1)), S.ERR_ARG),
    (lambda x: torch.zeros(99999).as_strided((N, T, HEADS, D), (9000, (HEADS - 1) * D, D, 1)), S.ERR_ARG),
    (lambda x: torch.zeros(99999).as_strided((N, T, HEADS, D), (9000, D, T * D + 2, 1)), S.ERR_ALIGN),
    (lambda x: torch.zeros(99999).as_strided((N, T, HEADS, D), (9000, HEADS * D + 16, D + 2, 1)), S.ERR_ALIGN),
], ids=range(8))
def test_rows_that_meet_or_do_not_fit(bad, want):
    for name in ("q", "out", "dout", "dq"):
        a = gradient(make=by_token)
        a[name] = bad(a[name])
        assert status("prompt_attention_backward", a.values()) == want, name


def test_distances_of_the_c_abi(lib):
    """Null and huge distances, and the calls without them as the ones with head_dim."""
    at = lambda i: (ctypes.c_void_p * 2)(BASE + i * 256 * MIB, BASE + (i * 256 + 64) * MIB)  # noqa: E731

    def call(stride=HEADS * D, head=D, tokens=T, kv_head=D):
        return lib.rar_prompt_attention_ex(at(1), stride, head, at(2), KV * D, kv_head, at(3), KV * D, D, 2, tokens, HEADS, KV, D, 1,
                                           BASE, 1, 0.1, at(4), HEADS * D, D, None, BASE + 13 * 256 * MIB, 4096, None)

    assert call() == S.ERR_WORKSPACE
    assert call(stride=D, head=T * D) == S.ERR_WORKSPACE
    assert call(stride=0, tokens=1) == S.ERR_WORKSPACE
    for bad in (dict(head=0), dict(head=-D), dict(stride=-D), dict(head=1 << 62), dict(stride=1 << 62), dict(head=D - 8), dict(kv_head=0),
                dict(stride=D, head=T * D - 8), dict(stride=HEADS * D - 8)):
        assert call(**bad) == S.ERR_ARG, bad
    assert call(head=D + 4, stride=HEADS * (D + 8)) == S.ERR_ALIGN
