"""GPU tests of what the prompt operators do at their edges: tensors laid out in other ways, waits that run out of
time, single keys that are no numbers, what the roundings of weights leave, weights and gradients of few keys."""
import pytest

torch = pytest.importorskip("torch")

from collective_communication_gb300 import binding as B
from test_gpu_prompt_operators import (DT, MARK, attend, backward, cached_forward, close, forward, gen, i32, normal, paged,
                                       prompt_inputs, scores, starts_of, U, workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()
    yield


# ---------------------------------------------------------------- layouts
def by_head(x):
    """A copy whose heads are apart by all tokens and 16 elements more, with marks between them."""
    n, t, h, d = x.shape
    buffer = torch.full((n, h, t * d + 16), MARK, dtype=x.dtype, device="cuda")
    view = buffer[:, :, :t * d].unflatten(2, (t, d)).transpose(1, 2)
    view.copy_(x)
    return view, buffer[:, :, t * d:]


def apart(x):
    """A copy with 8 elements more behind each head, and 24 behind each token."""
    n, t, h, d = x.shape
    buffer = torch.full((n, t, h * (d + 8) + 24), MARK, dtype=x.dtype, device="cuda")
    view = buffer[:, :, :h * (d + 8)].unflatten(2, (h, d + 8))
    view[..., :d].copy_(x)
    return view[..., :d], torch.cat([view[..., d:].flatten(), buffer[:, :, h * (d + 8):].flatten()])


LAYOUTS = [
    ([97], 8, 1, 128, "bf16"), ([300, 0, 41], 6, 2, 64, "bf16"), ([1], 4, 2, 64, "bf16"), ([1], 4, 2, 64, "f32"), ([1100, 30], 16, 2, 128, "bf16"),
    ([140, 5], 6, 3, 80, "bf16"), ([60], 4, 2, 192, "bf16"), ([140, 5], 6, 3, 80, "f32"), ([600], 16, 2, 64, "f32"), ([33, 2], 5, 5, 40, "bf16"),
]


@pytest.mark.parametrize("layout", [by_head, apart])
@pytest.mark.parametrize("lens,heads,kv,dim,dtype", LAYOUTS, ids=str)
def test_layouts_change_nothing(lens, heads, kv, dim, dtype, layout):
    """Heads of any distance give the same bits as dense ones, and what lies between rows is left as it was."""
    q, k, v, starts = prompt_inputs(2, lens, heads, kv, dim, dtype, behind=2)
    out, lse = forward(q, k, v, starts)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    want = [out, *backward(q, k, v, starts, out, lse, dout)]
    q, k, v, dout = (layout(x)[0] for x in (q, k, v, dout))
    (out, g0), (dq, g1), (dk, g2), (dv, g3) = (layout(torch.full_like(x, MARK)) for x in want)
    ws = workspace(q, kv)
    again = torch.full_like(lse, MARK)
    B.prompt_attention(q, k, v, starts, out, again, ws)
    B.prompt_attention_backward(q, k, v, starts, out, lse, dout, dq, dk, dv, ws)
    assert B.get_status(ws) == B.Status.OK and torch.equal(again, lse)
    for got, w in zip((out, dq, dk, dv), want):
        assert torch.equal(got, w)
    assert all(bool((g == MARK).all()) for g in (g0, g1, g2, g3))


@pytest.mark.parametrize("layout", [by_head, apart])
@pytest.mark.parametrize("new,lens,heads,kv,dim,page,dtype", [
    ([5], [3000], 16, 2, 128, 64, "bf16"), ([40, 130], [300, 400], 6, 2, 80, 16, "bf16"), ([3, 9], [60, 500], 4, 2, 64, 2, "bf16"),
    ([4], [900], 4, 2, 64, 16, "f32"), ([1], [500], 4, 1, 192, 32, "bf16")], ids=str)
def test_cached_layouts_change_nothing(new, lens, heads, kv, dim, page, dtype, layout):
    g = gen(3)
    k, v, table, _, _ = paged(g, 2, lens, kv, dim, page, DT[dtype])
    q = normal(g, 2, sum(new) + 1, heads, dim, dtype=DT[dtype])
    starts, lens = starts_of(new), i32(*lens)
    want, want_lse = cached_forward(q, k, v, table, starts, lens)
    q = layout(q)[0]
    out, gaps = layout(torch.full_like(want, MARK))
    lse, ws = torch.full_like(want_lse, MARK), workspace(q, kv)
    B.prompt_attention_cached(q, k, v, table, starts, lens, out, lse, ws)
    assert B.get_status(ws) == B.Status.OK
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and bool((gaps == MARK).all())


def test_forward_result_of_torch():
    """The gradient takes out as a product of heads leaves it, turned back to tokens, and tensors of different layouts."""
    q, k, v, starts = prompt_inputs(2, [150], 4, 2, 64, "bf16")
    out, lse = forward(q, k, v, starts)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    want = backward(q, k, v, starts, out, lse, dout)
    turned = out.transpose(1, 2).contiguous().transpose(1, 2)
    assert not turned.is_contiguous()
    for a, b in zip(want, backward(q, by_head(k)[0], v, starts, turned, lse, apart(dout)[0])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("requests", [3, 40])
@pytest.mark.parametrize("dim,page,dtype", [(64, 16, "bf16"), (128, 2, "bf16"), (64, 16, "f32")], ids=str)
def test_cached_requests_without_tokens(dim, page, dtype, requests):
    """Whatever the length and pages of a request are that has no tokens in the call: nothing is looked at or reported."""
    new, lens = [4, 0, 7] + [0] * (requests - 3), [30, 9, 20] + [5] * (requests - 3)
    k, v, table, _, _ = paged(gen(3), 1, lens, 2, dim, page, DT[dtype])
    q = normal(gen(4), 1, sum(new), 4, dim, dtype=DT[dtype])
    starts = starts_of(new)
    want = cached_forward(q, k, v, table, starts, i32(*lens))
    for bad in (-1, 2 ** 30):
        lens[1] = bad
        table[1] = -5
        assert all(torch.equal(a, b) for a, b in zip(cached_forward(q, k, v, table, starts, i32(*lens)), want))


@pytest.mark.parametrize("new,lens", [([5], [2000]), ([40, 130, 0, 3], [300, 130, 17, 129])], ids=str)
@pytest.mark.parametrize("dim", [40, 64, 72, 128])
def test_cached_in_pages_of_any_size(dim, new, lens):
    """Pages on both sides of the sizes at which they are copied in another way: the same bits."""
    g = gen(5)
    q = normal(g, 2, sum(new), 4, dim, dtype=torch.bfloat16)
    starts, first = starts_of(new), None
    for page in (4, 8, 16, 32):
        k, v, table, keys, values = paged(gen(6), 2, lens, 2, dim, page, torch.bfloat16, extra_columns=0)
        table = torch.cat([table, table.new_full((len(lens), 2048 // page - table.shape[1]), -7)], 1)  # as wide in tokens
        found = cached_forward(q, k, v, table, starts, i32(*lens))
        first = first or found
        assert all(torch.equal(x, y) for x, y in zip(first, found))


# ---------------------------------------------------------------- waits that run out
@pytest.fixture
def short_limit():
    """Waits of 20 ms, and a warp of each block that works out weights leaves at its first item: nothing that the others
    wait for comes, so they leave as well."""
    B.set_spin_timeout_ns(20_000_000)
    B.debug_set_fault(4)
    yield
    B.debug_set_fault(0)
    B.set_spin_timeout_ns(0)


def run_out(call, ws, outs):
    """The call ends with its status, and writes no rows of tokens in no sequence (the last two)."""
    call()
    assert B.get_status(ws) == B.Status.ERR_TIMEOUT
    assert all(bool((x[:, -2:] == MARK).all()) for x in outs)


@pytest.mark.parametrize("lens,heads,kv,dim", [([700], 8, 1, 128), ([97], 8, 1, 128), ([4000], 4, 1, 64), ([60, 200], 6, 2, 80)], ids=str)
def test_forward_runs_out_of_time(short_limit, lens, heads, kv, dim):
    q, k, v, starts = prompt_inputs(2, lens, heads, kv, dim, "bf16", behind=2)
    ws, out, lse = workspace(q, kv), torch.full_like(q, MARK), torch.full(q.shape[:3], MARK, device="cuda")
    run_out(lambda: B.prompt_attention(q, k, v, starts, out, lse, ws), ws, (out, lse))
    B.debug_set_fault(0)
    want, want_lse = forward(q, k, v, starts)
    out, lse = forward(q, k, v, starts, ws=ws)  # the same workspace
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("new,lens,dim,page", [([5], [3000], 128, 64), ([300, 20], [700, 20], 128, 16), ([300], [900], 64, 16),
                                               ([40], [500], 80, 2), ([9, 9], [60, 50], 64, 1)], ids=str)
def test_cached_runs_out_of_time(short_limit, new, lens, dim, page):
    k, v, table, _, _ = paged(gen(3), 2, lens, 2, dim, page, torch.bfloat16)
    q = normal(gen(4), 2, sum(new) + 2, 8, dim, dtype=torch.bfloat16)
    starts, lens = starts_of(new), i32(*lens)
    ws, out, lse = workspace(q, 2), torch.full_like(q, MARK), torch.full(q.shape[:3], MARK, device="cuda")
    run_out(lambda: B.prompt_attention_cached(q, k, v, table, starts, lens, out, lse, ws), ws, (out, lse))
    B.debug_set_fault(0)
    want = cached_forward(q, k, v, table, starts, lens)
    assert all(torch.equal(a, b) for a, b in zip(cached_forward(q, k, v, table, starts, lens, ws), want))


@pytest.mark.parametrize("lens,heads,kv,dim", [([700], 8, 1, 128), ([97], 8, 1, 128), ([1500], 16, 1, 64), ([60, 200], 6, 2, 80),
                                               ([3, 20], 6, 2, 64)], ids=str)
def test_gradient_runs_out_of_time(short_limit, lens, heads, kv, dim):
    """Rows that see one tile of keys (among 97 tokens, say) wait for one another's sums as well."""
    q, k, v, starts = prompt_inputs(2, lens, heads, kv, dim, "bf16", behind=2)
    B.debug_set_fault(0)
    out, lse = forward(q, k, v, starts)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    want = backward(q, k, v, starts, out, lse, dout)
    ws, grads = workspace(q, kv), [torch.full_like(x, MARK) for x in (q, k, k)]
    B.debug_set_fault(4)
    run_out(lambda: B.prompt_attention_backward(q, k, v, starts, out, lse, dout, *grads, ws), ws, grads)
    B.debug_set_fault(0)
    for a, b in zip(want, backward(q, k, v, starts, out, lse, dout, ws)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("limit", [2 ** 64 - 1, 2 ** 63])
def test_no_limit_at_all(limit):
    """The largest limits are limits like any other."""
    q, k, v, starts = prompt_inputs(1, [2000, 50], 8, 1, 128, "bf16")
    want = forward(q, k, v, starts)
    grads = backward(q, k, v, starts, *want, q)
    B.set_spin_timeout_ns(limit)
    try:
        got = forward(q, k, v, starts)
        again = backward(q, k, v, starts, *got, q)
    finally:
        B.set_spin_timeout_ns(0)
    assert all(torch.equal(a, b) for a, b in zip((*got, *again), (*want, *grads)))


# ---------------------------------------------------------------- what is no number
@pytest.mark.parametrize("bad", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("lens", [[3, 1, 40], [3, 1, 200]], ids=str)
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "bf16"), (80, "bf16"), (192, "bf16"), (64, "f32"), (128, "f32")], ids=str)
def test_gradient_of_one_key_that_is_no_number(dim, dtype, lens, bad):
    """A row that sees one key alone: what is infinite or NaN there shows in every gradient that the formula takes from it
    (dv takes nothing of v), in every form alike, and in no other sequence."""
    q, k, v, starts = prompt_inputs(1, lens, 4, 2, dim, dtype, seed=2)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    out, lse = forward(q, k, v, starts)
    want = backward(q, k, v, starts, out, lse, dout)
    for value in (float("nan"), float("inf")):
        x = dict(q=q.clone(), k=k.clone(), v=v.clone(), dout=dout.clone())
        x[bad][:, 3, 0] = value  # its first head: of a group of two queries, or one of them
        o, l = forward(x["q"], x["k"], x["v"], starts)
        dq, dk, dv = backward(x["q"], x["k"], x["v"], starts, o, l, x["dout"])
        heads = 1 if bad in ("q", "dout") else 2
        assert not bool(dq[:, 3, :heads].isfinite().any()) and torch.equal(dq[:, 3, heads:], want[0][:, 3, heads:])
        assert not bool(dk[:, 3, 0].isfinite().any()) and torch.equal(dk[:, 3, 1], want[1][:, 3, 1])
        if bad == "v":
            assert torch.equal(dv, want[2])
        else:
            assert not bool(dv[:, 3, 0].isfinite().any()) and torch.equal(dv[:, 3, 1], want[2][:, 3, 1])
        for a, b in zip((dq, dk, dv), want):
            assert torch.equal(a[:, :3], b[:, :3]) and torch.equal(a[:, 4:], b[:, 4:])


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.5, 0.5])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "bf16"), (192, "bf16"), (64, "f32")], ids=str)
def test_scores_that_are_no_numbers(dim, dtype, scale):
    """A query or key of NaN shows in the rows that see it, whatever the scale; another sequence's do not change."""
    q, k, v, starts = prompt_inputs(1, [40, 200, 30], 4, 2, dim, dtype, seed=2)
    want, want_lse = forward(q, k, v, starts, scale=scale)
    q[:, 50, 1], k[:, 140, 1, 5] = float("nan"), float("nan")
    out, lse = forward(q, k, v, starts, scale=scale)
    bad = torch.zeros(1, 270, 4, dtype=torch.bool, device="cuda")
    bad[:, 50, 1] = True
    bad[:, 140:240, 2:] = True
    assert torch.equal(lse.isnan(), bad) and bool(out[bad].isnan().all())
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])


# ---------------------------------------------------------------- roundings of weights
@pytest.mark.parametrize("lens", [[2, 300, 17, 1, 128, 129, 90], [5] * 70, [128, 1000, 3]], ids=str)
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_gradient_of_short_sequences_among_others(lens, dim):
    """A sequence of up to 128 tokens loses nothing to the roundings of weights, whatever it is packed with: the bound of
    a call of its own, 2^-13 of the magnitudes (2^-16 of a weight or a score's gradient is lost with what their
    roundings leave, sums of 128 binary32 products take 2^-17, the exponential of a score below 16 2^-19, lse's rounding
    2^-21; below 2^-15 in all, of terms that are multiplied twice)."""
    q, k, v, starts = prompt_inputs(2, lens, 6, 2, dim, "bf16", seed=6)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    out, lse = forward(q, k, v, starts)
    dq, dk, dv = backward(q, k, v, starts, out, lse, dout)
    bounds = starts.tolist()
    for r in range(2):
        for a, b in zip(bounds, bounds[1:]):
            if b - a > 128:
                continue
            x, key, value, g = (z[r, a:b].double() for z in (q, k, v, dout))
            x, g = (z.unflatten(1, (2, 3)) for z in (x, g))
            s, sees, _ = scores(q[r, a:b], k[r, a:b], 0, dim ** -0.5)
            p = torch.softmax(s.masked_fill(~sees, float("-inf")), -1)
            dp = torch.einsum("thgd,shd->hgts", g, value)
            dsize = torch.einsum("thgd,shd->hgts", g.abs(), value.abs())
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            size = p * (dsize + (p * dsize).sum(-1, keepdim=True)) * 2 ** -13 * dim ** -0.5
            close(dq[r, a:b], torch.einsum("hgts,shd->thgd", ds, key).flatten(1, 2) * dim ** -0.5,
                  torch.einsum("hgts,shd->thgd", size, key.abs()).flatten(1, 2), "dq")
            close(dk[r, a:b], torch.einsum("hgts,thgd->shd", ds, x) * dim ** -0.5,
                  torch.einsum("hgts,thgd->shd", size, x.abs()), "dk")
            close(dv[r, a:b], torch.einsum("hgts,thgd->shd", p, g), 2 ** -13 * torch.einsum("hgts,thgd->shd", p, g.abs()), "dv")


@pytest.mark.parametrize("new,lens,heads,kv,dim,page", [
    ([5], [3000], 16, 2, 128, 64), ([1, 16, 3], [1, 700, 41], 8, 1, 128, 16), ([9, 128, 40], [900, 128, 1000], 2, 2, 64, 16),
    ([42, 300, 1], [50, 800, 513], 6, 2, 80, 32), ([7, 2], [300, 9], 8, 2, 64, 4), ([1] * 40, list(range(1, 401, 10)), 4, 2, 64, 16),
    ([1], [30000], 100, 1, 128, 128)], ids=str)
def test_cached_requests_of_few_tokens(new, lens, heads, kv, dim, page):
    """New tokens of one tile of rows lose nothing to the weights' rounding, whatever else is in the call: a weight is off by
    2^-16 of itself (the rounding of what its rounding leaves), where attend() allows 2^-8 for others."""
    k, v, table, keys, values = paged(gen(3), 2, lens, kv, dim, page, torch.bfloat16)
    q = normal(gen(4), 2, sum(new), heads, dim, dtype=torch.bfloat16)
    starts = starts_of(new)
    out, lse = cached_forward(q, k, v, table, starts, i32(*lens))
    bounds = starts.tolist()
    for r in range(2):
        for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
            o, _, slack, _ = attend(q[r, a:b], keys[i][r], values[i][r], lens[i] - (b - a), dim ** -0.5)
            if b - a <= 128 // (heads // kv):
                s, sees, _ = scores(q[r, a:b], keys[i][r], lens[i] - (b - a), dim ** -0.5)
                p = torch.softmax(s.masked_fill(~sees, float("-inf")), -1)
                mass = torch.einsum("hgts,shd->thgd", p, values[i][r].double().abs()).flatten(1, 2)
                slack = slack - (2.0 ** -8 - 2.0 ** -16) * mass
            close(out[r, a:b], o, slack, f"{i}")


PLAIN = [(64, "f32"), (80, "f32"), (128, "f32"), (200, "f32"), (192, "bf16")]  # forms of the ordinary arithmetic units


@pytest.mark.parametrize("dim,dtype", PLAIN, ids=str)
def test_weight_of_a_score_that_is_lse(dim, dtype):
    """A score and an lse that are the same number leave a weight of 1, exactly, however large they are: dv is dout."""
    score = torch.tensor([0.0, 1.0, -3.0, 100.0, 123.25, -77.5, 1000.0, 3.0, -4096.0], device="cuda").to(DT[dtype])
    n = len(score)
    q, k = (torch.zeros(1, n, 1, dim, dtype=DT[dtype], device="cuda") for _ in range(2))
    q[0, :, 0, 3], k[0, :, 0, 3] = score, 1.0  # products and sums are exact
    v, dout = (normal(gen(i), 1, n, 1, dim, dtype=q.dtype) for i in (1, 2))
    dq, dk, dv = backward(q, k, v, starts_of([1] * n), v, score.float().view(1, n, 1), dout, scale=1.0)
    assert torch.equal(dv, dout) and bool((dq == 0).all()) and bool((dk == 0).all())


@pytest.mark.parametrize("dim,dtype", PLAIN, ids=str)
def test_gradient_of_keys_that_are_alike(dim, dtype):
    """Two equal keys of equal values have no gradient. Their dO . v are the same bits x, and so are their weights, 1/2 up to
    4 U for the exponential, 2 U for its exponent and U for lse: 1/2 (1 + d), d below 8 U. The sum of p x is x (1 + d) up to
    2 U x, so a score's gradient is below 1/2 (8 + 2 + 1) U |x|: 8 U |x|, where a sum of out . dout is off by some U of the
    sum of the magnitudes, hundreds of times |x| here. dq and dk of the second token are these, times scale and k, or q."""
    k = normal(gen(1), 1, 1, 1, dim, dtype=DT[dtype]).expand(1, 2, 1, dim).contiguous()
    v = normal(gen(2), 1, 1, 1, dim, dtype=DT[dtype]).expand(1, 2, 1, dim).contiguous()
    q = torch.zeros_like(k)  # scores of 0: lse is the logarithm of 2
    x = normal(gen(3), dim).double()
    y = v[0, 0, 0].double()
    dout = (x - (x @ y) / (y @ y) * y).to(q.dtype).expand(1, 2, 1, dim).contiguous()  # across the value, but for its rounding
    out, lse = forward(q, k, v, starts_of([2]), scale=0.5)
    dq, dk, dv = backward(q, k, v, starts_of([2]), out, lse, dout, scale=0.5)
    dot = abs(float(dout[0, 1, 0].double() @ y)) + 2 * dim * U * float((dout[0, 1, 0].double() * y).abs().sum())
    assert bool((dq[0, 1, 0].double().abs() <= 2 * 0.5 * 8 * U * dot * k[0, 1, 0].double().abs()).all())
    assert bool((dk == 0).all())  # queries of 0
