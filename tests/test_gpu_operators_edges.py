"""GPU tests of the operators at the edges of their domain: vanishing values and no
eps, sums that must neither miss nor repeat a row, zeros of both signs,
infinities and NaN in valid places. Bounds as in test_gpu_operators.py, from
binary32 roundings of the 64-bit computation's magnitudes, unless a test derives
its own."""
import pytest

torch = pytest.importorskip("torch")

from collective_communication_gb300 import binding as B
from test_gpu_operators import DT, U, attention64, attention_case, close, gen, i32, normal, run_attention, run_logprobs, \
    turn64

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()
    yield


# ------------------------------------------------------------ norm and rotation
def rope_inputs(seed, n, t, q, kv, d, rot, dtype, scale):
    g = gen(seed)
    qkv = normal(g, n, t, (q + 2 * kv) * d, dtype=DT[dtype], scale=scale)
    wq, wk = normal(g, d, dtype=DT[dtype]), normal(g, d, dtype=DT[dtype])
    angle = torch.rand((300, rot // 2), generator=g, device="cuda") * 6.3
    pos = torch.randint(0, 300, (t,), generator=g, device="cuda", dtype=torch.int32)
    grads = [normal(g, n, t, h, d, dtype=DT[dtype]) for h in (q, kv, kv)]
    return qkv, wq, wk, torch.cat([angle.cos(), angle.sin()], 1), pos, grads


def check_rope(qkv, wq, wk, cs, pos, grads, q, kv, d, inter, eps):
    """Forward and gradient against 64 bits."""
    n, t = qkv.shape[:2]
    rot = cs.shape[1]
    x = qkv.double().view(n, t, q + 2 * kv, d)[:, :, :q + kv]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = x * r
    w = torch.cat([wq.double().expand(q, d), wk.double().expand(kv, d)])
    row = cs.double()[pos.long()][None, :, None]

    def span(v):  # of the magnitudes that meet in a rotation
        return v + turn64(v, row.abs(), rot, inter).abs() + turn64(v, -row.abs(), rot, inter).abs()

    y = turn64(xh * w, row, rot, inter)
    dy = torch.cat(grads[:2], 2).double()
    z = turn64(dy, row, rot, inter, back=True)
    zs = span(dy.abs())
    a = z * w
    dx = r * (a - xh * (a * xh).mean(-1, keepdim=True))
    size = r * (zs * w.abs() + xh.abs() * (zs * w.abs() * xh.abs()).mean(-1, keepdim=True))
    ws = B.OpWorkspace(B.qk_norm_rope_workspace_bytes(n, d))
    yq, yk = (torch.full((n, t, h, d), NAN, dtype=qkv.dtype, device="cuda") for h in (q, kv))
    B.qk_norm_rope(qkv, wq, wk, cs, pos, yq, yk, ws, eps=eps, interleaved=inter)
    slack = (d / 2 + 12) * U * span((xh * w).abs())
    close(yq, y[:, :, :q], slack[:, :, :q], "q")
    close(yk, y[:, :, q:], slack[:, :, q:], "k")
    dqkv = torch.full_like(qkv, NAN)
    dwq, dwk = (torch.full((n, d), NAN, device="cuda") for _ in range(2))
    B.qk_norm_rope_backward(qkv, wq, wk, cs, pos, *grads, dqkv, dwq, dwk, ws, eps=eps, interleaved=inter)
    assert B.get_status(ws) == B.Status.OK
    got = dqkv.view(n, t, q + 2 * kv, d)
    close(got[:, :, :q + kv], dx, (2 * d + 24) * U * size, "dx")
    assert torch.equal(got[:, :, q + kv:], grads[2])
    for dw, heads in ((dwq, slice(0, q)), (dwk, slice(q, q + kv))):
        mag = (zs * xh.abs())[:, :, heads].sum((1, 2))
        close(dw, (z * xh)[:, :, heads].sum((1, 2)), (t * (q + kv) + d + 24) * U * mag, "dw")


@pytest.mark.parametrize("n,t,q,kv,d,rot,inter,dtype", [
    (1, 1, 1, 1, 64, 64, False, "f32"), (2, 1, 8, 1, 128, 128, False, "bf16"), (1, 3, 32, 4, 96, 48, True, "bf16"),
    (1, 5, 3, 1, 8, 8, False, "f32"), (2, 701, 5, 3, 80, 40, False, "f32"), (1, 3001, 12, 4, 64, 64, True, "bf16"),
    (1, 2, 4, 2, 256, 128, False, "bf16")])
def test_norm_rope_without_eps(n, t, q, kv, d, rot, inter, dtype):
    """Groups of threads that have fewer rows than their neighbours add nothing to the weights' gradient."""
    check_rope(*rope_inputs(41, n, t, q, kv, d, rot, dtype, 1.0), q, kv, d, inter, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-45, -60])
def test_norm_rope_of_vanishing_rows(power, dtype):
    """Rows so small that the third power of 1 / rms, or the second, is past binary32, while the results are not."""
    check_rope(*rope_inputs(42, 2, 9, 4, 2, 96, 48, dtype, 2.0 ** power), 4, 2, 96, False, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_rope_of_zero_rows_with_a_subnormal_eps(dtype):
    inputs = rope_inputs(43, 1, 5, 4, 2, 64, 64, dtype, 1.0)
    inputs[0][:, 2] = 0
    check_rope(*inputs, 4, 2, 64, False, 2.0 ** -140)


@pytest.mark.parametrize("n,t,q,kv,d,dtype", [
    (1, 1500, 7, 3, 128, "f32"), (2, 4097, 4, 2, 64, "bf16"), (1, 20000, 2, 1, 256, "bf16"), (1, 130, 32, 4, 80, "f32")])
def test_norm_rope_weight_gradient_counts_every_row_once(n, t, q, kv, d, dtype):
    """Elements of +-1 and whole gradients, nothing turned: each weight's gradient is a sum of whole numbers from 1 to 4,
    of either sign, that binary32 holds exactly, times a 1 / rms of 1 that is off by 4 u at most and rounded once more: less
    than 1/2 in all, where a row that was left out or added twice is 1 or more."""
    g = gen(44)

    def signs(*shape):
        return (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1).to(DT[dtype])

    def whole(h):
        return signs(n, t, h, d) * torch.randint(1, 5, (n, t, h, d), generator=g, device="cuda").to(DT[dtype])

    qkv, dq, dk = signs(n, t, (q + 2 * kv) * d), whole(q), whole(kv)
    w = torch.ones(d, dtype=DT[dtype], device="cuda")
    cs = torch.cat([torch.ones(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")], 1)
    pos = torch.zeros(t, dtype=torch.int32, device="cuda")
    assert 4 * t * max(q, kv) * 6 * U < 0.5
    ws = B.OpWorkspace(B.qk_norm_rope_workspace_bytes(n, d))
    dwq, dwk = (torch.full((n, d), NAN, device="cuda") for _ in range(2))
    B.qk_norm_rope_backward(qkv, w, w, cs, pos, dq, dk, dk, torch.empty_like(qkv), dwq, dwk, ws, eps=0.0)
    x = qkv.double().view(n, t, q + 2 * kv, d)
    for got, dy, heads in ((dwq, dq, slice(0, q)), (dwk, dk, slice(q, q + kv))):
        assert float((got.double() - (dy.double() * x[:, :, heads]).sum((1, 2))).abs().max()) < 0.5


# ------------------------------------------------------------ log probabilities
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [1, 2, 5, 9, 32])
def test_token_logprobs_alternatives_hold_both_zeros_equal(top, dtype):
    """0 and -0 are one value, so the lower index comes first, wherever they lie in a row and its parts."""
    g = gen(51)
    for widths in ([40], [33, 700], [1024] * 5, [9000, 1], [16384] * 8, [131072]):
        total = sum(widths)
        rows = 6
        x = -1 - torch.rand((rows, total), generator=g, device="cuda")
        x[0, -1], x[0, 3] = 0.0, -0.0                 # two, the negative one first
        x[1, 0], x[1, total // 2], x[1, -2] = -0.0, 0.0, -0.0
        x[2] = torch.where(torch.rand(total, generator=g, device="cuda") < 0.5, 0.0, -0.0)
        x[3] = -0.0
        x[3, total // 3:] = 0.0                       # the negative ones first
        many = torch.randperm(total, generator=g, device="cuda")[:40]
        x[4, many] = torch.where(many % 2 == 0, 0.0, -0.0)
        x[5, many] = torch.where(many % 3 == 0, 0.0, -0.0)
        x[5, many[:3]] = 2.0
        x = x.to(DT[dtype])
        parts = [p.contiguous() for p in x.split(widths, 1)]
        o, _ = run_logprobs(parts, torch.zeros(rows, dtype=torch.int32, device="cuda"), top)
        order = torch.sort(x.double(), dim=1, descending=True, stable=True)
        assert torch.equal(o["top_ids"].long(), order.indices[:, :top]), widths


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_logprobs_of_a_word_that_holds_everything(dtype):
    """A word above all others by 2e30 has the whole probability."""
    x = torch.full((2, 3000), -1e30, device="cuda")
    x[0, 5] = x[1, 2999] = 1e30
    x = x.to(DT[dtype])
    o, _ = run_logprobs([x[:, :1001].contiguous(), x[:, 1001:].contiguous()], i32(6, 2999), 2)
    assert o["entropy"].tolist() == [0, 0]
    assert float(o["logprob"][0]) <= -1e30 and float(o["logprob"][1]) == 0
    assert o["top_ids"].tolist() == [[5, 0], [2999, 0]] and o["top_values"][:, 0].tolist() == [0, 0]
    assert torch.equal(o["lse"], x.float().amax(1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("widths", [[500, 499], [20001]])
@pytest.mark.parametrize("entropy", ["none", "zero"])
@pytest.mark.parametrize("in_place", [False, True])
def test_token_logprobs_gradient_of_rows_without_a_token(widths, dtype, entropy, in_place):
    """Their log probability is the constant 0, whatever the logits are: a padding row of NaN, or with nothing but -inf,
    has the gradient 0."""
    g = gen(52)
    total = sum(widths)
    x = normal(g, 5, total, dtype=DT[dtype], scale=3.0)
    x[1] = -INF
    x[2, 7], x[3, total - 1] = NAN, INF
    tokens = i32(-1, -1, total, -5, 2)
    parts = [p.clone() for p in x.split(widths, 1)]
    o, ws = run_logprobs(parts, tokens, 0)
    assert o["logprob"][:4].tolist() == [0] * 4
    out = parts if in_place else [torch.full_like(p, NAN) for p in parts]
    grad = torch.tensor([NAN, 1.0, 2.0, INF, 0.5], device="cuda")
    h = None if entropy == "none" else torch.zeros(5, device="cuda")
    B.token_logprobs_backward(parts, tokens, o["lse"], o["entropy"], grad, h, out, ws)
    assert B.get_status(ws) == B.Status.OK
    got = torch.cat(out, 1)
    assert not bool(got[:4].any())  # NaN counts as true
    p = torch.softmax(x[4].double(), 0)
    want = 0.5 * ((torch.arange(total, device="cuda") == 2).double() - p)
    size = x[4].double().abs() + abs(float(o["lse"][4]))
    # p's exponent is off by 4 u of its terms and by lse's own error, of (4 total^(1/2) + 16) u and 4 u of its terms
    close(got[4], want, 0.5 * (p + (want > 0)) * (8 * size + 4 * total ** 0.5 + 40) * U, "the row with a token")


# -------------------------------------------------------------------- attention
ATTENTION = [(q, kv, d, dtype) for dtype in ("f32", "bf16")
             for q, kv, d in ((8, 2, 64), (16, 1, 128), (3, 1, 80), (12, 1, 192), (5, 1, 256))]


@pytest.mark.parametrize("q,kv,d,dtype", ATTENTION)
@pytest.mark.parametrize("length", [1, 16, 17, 65, 130, 5000])
def test_decode_attention_nan_in_a_valid_key(length, q, kv, d, dtype):
    """A NaN in the key of a valid token, wherever it lies among the tokens that a warp, a tile or a block takes, is in
    out and lse of its head's queries, and nowhere else."""
    lens = [length, 40, length]
    places = sorted({0, length - 1, length // 2, min(length - 1, 16), min(length - 1, 64)})
    x, k, v, table, ln = attention_case(61, 1, lens, q, kv, d, 16, dtype)
    want, wlse, tol, ltol = attention64(x, k, v, table, ln, d ** -0.5, 16)
    for t in places:
        bad = k.clone()
        bad[0, table[0, t // 16].long(), 0, t % 16, d // 2] = NAN
        out, lse, status, _ = run_attention(x, bad, v, table, ln)
        assert status == B.Status.OK
        mine = slice(0, q // kv)
        assert bool(out[0, 0, mine].isnan().all()) and bool(lse[0, 0, mine].isnan().all()), t
        rest = torch.ones((1, 3, q), dtype=torch.bool, device="cuda")
        rest[0, 0, mine] = False
        close(out[rest], want[rest], tol[rest], "out of the others")
        close(lse[rest], wlse[rest], ltol[rest], "lse of the others")


@pytest.mark.parametrize("q,kv,d,dtype", ATTENTION)
def test_decode_attention_nan_in_a_query(q, kv, d, dtype):
    lens = [1, 17, 700, 5000, 0]
    x, k, v, table, ln = attention_case(62, 1, lens, q, kv, d, 16, dtype)
    want, wlse, tol, ltol = attention64(x, k, v, table, ln, d ** -0.5, 16)
    x = x.clone()
    x[:, :, q - 1, 3] = NAN
    out, lse, status, _ = run_attention(x, k, v, table, ln)
    assert status == B.Status.OK
    assert bool(out[0, :4, q - 1].isnan().all()) and bool(lse[0, :4, q - 1].isnan().all())
    assert not bool(out[0, 4].any()) and bool((lse[0, 4] == -INF).all())  # nothing to attend to
    close(out[:, :4, :q - 1], want[:, :4, :q - 1], tol[:, :4, :q - 1], "out of the others")
    close(lse[:, :4, :q - 1], wlse[:, :4, :q - 1], ltol[:, :4, :q - 1], "lse of the others")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length", [1, 17, 3000])
def test_decode_attention_infinite_key(length, dtype):
    """A score of +inf, or in binary32 any product with an infinity, makes out and lse NaN; a score of -inf is one of no
    weight."""
    q, d = 8, 64
    x, k, v, table, ln = attention_case(63, 1, [length], q, 1, d, 16, dtype)
    t = length - 1
    x[0, 0, :, 5] = x[0, 0, :, 5].abs() + 0.5
    x[0, 0, :4, 5] *= -1
    bad = k.clone()
    bad[0, table[0, t // 16].long(), 0, t % 16, 5] = INF
    out, lse, status, _ = run_attention(x, bad, v, table, ln)
    assert status == B.Status.OK
    nan = slice(4, q) if dtype == "bf16" else slice(0, q)
    assert bool(out[0, 0, nan].isnan().all()) and bool(lse[0, 0, nan].isnan().all())
    if dtype == "bf16":
        want, wlse, tol, ltol = attention64(x, k, v, table, i32(length - 1), d ** -0.5, 16)
        close(out[:, :, :4], want[:, :, :4], tol[:, :, :4], "without the token")
        close(lse[:, :, :4], wlse[:, :, :4], ltol[:, :, :4], "lse without the token")
