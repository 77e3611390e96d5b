"""GPU tests of the prompt and training operators (attention over whole prompts and
its gradient, embedding over vocabulary shards and its gradient) against plain
64-bit implementations of their formulas.

Tolerances. u = 2^-24 is half an ulp of binary32; a binary32 sum of n terms is off by
at most n u times the sum of the terms' magnitudes in any order, and by twice that
where a matrix unit cuts instead of rounding. A score s = scale q . k of D products is
therefore off by E = 2 (D + 4) u scale sum |q_d k_d| (products of bf16 are exact, those
of binary32 are rounded: among the 4), and exp(s - lse) relatively by E plus the
roundings of the exponent, 4 u (|s| + |lse|), and a few u for the exponential: `weight`
below is the largest of that over a row's keys. Weights and score gradients of bf16
inputs may be rounded to bf16, by 2^-8 of themselves, before they meet values, queries
or keys. A weight below the smallest normal number, 2^-126, may count as 0. The gradient's
delta may be out . dout, of the out that the call is given, or the sum of p (dout . v) that
it stands for: they differ by out's rounding and what the forward call leaves, and by the
errors of p and dout . v. A result is the rounding to its type of a sum that is within these relative
errors of the magnitudes of the 64-bit computation.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")

from collective_communication_gb300 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -126
MARK = 7.0  # what outputs hold before a call


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.load_library()
    yield


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def close(got, want, slack, what=""):
    """got is the rounding to its type of some value within slack of want (64 bits, broadcast), everywhere."""
    lo, hi = ((want + d).to(got.dtype).double() for d in (-slack, slack))
    bad = ~(((lo <= got) & (got <= hi)) | (got.double() == want))
    err = (got.double() - want).abs()[bad]
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} values off, by up to {float(err.max())}"


def starts_of(lens, first=0):
    return i32(*itertools.accumulate([first] + list(lens)))


def cut(x):
    """Where a product's inputs are rounded before it, by how much of themselves."""
    return ROUND[x.dtype] if x.dtype == torch.bfloat16 else 0.0


def scores(q, k, before, scale):
    """Scores [kv, group, rows, keys] in 64 bits of one sequence, which keys each row sees, and a bound of the error."""
    t, heads, d = q.shape
    kv = k.shape[1]
    x = q.double().unflatten(1, (kv, heads // kv))
    s = torch.einsum("thgd,shd->hgts", x, k.double()) * scale
    size = torch.einsum("thgd,shd->hgts", x.abs(), k.double().abs()) * abs(scale)
    sees = torch.arange(k.shape[0], device="cuda")[None] <= before + torch.arange(t, device="cuda")[:, None]
    return s, sees, 2 * (d + 4) * U * size


def attend(q, k, v, before, scale):
    """out [rows, heads, d], lse [rows, heads] and their slacks."""
    if k.shape[0] == 0:  # no key at all: one that no row sees
        k, v, before = torch.zeros_like(k.new_empty(1, *k.shape[1:])), torch.zeros_like(v.new_empty(1, *v.shape[1:])), -len(q)
    s, sees, e = scores(q, k, before, scale)
    s = s.masked_fill(~sees, float("-inf"))
    empty = ~sees.any(-1)
    lse = torch.logsumexp(s, -1)
    p = torch.where(empty[:, None], 0.0, torch.exp(s - torch.where(empty, 0.0, lse)[..., None]))
    size = torch.where(sees, s.abs(), 0.0).amax(-1)
    err = torch.where(sees, e, 0.0).amax(-1) + 4 * U * (size + lse.nan_to_num(neginf=0.0).abs()) + 8 * U
    n = k.shape[0]
    out = torch.einsum("hgts,shd->thgd", p, v.double()).flatten(1, 2)
    mass = torch.einsum("hgts,shd->thgd", p, v.double().abs())
    rows = lambda x: x.permute(2, 0, 1)  # noqa: E731
    slack = mass * (2 * rows(err) + cut(q) + 2 * (n + 8) * U)[..., None] + TINY * v.double().abs().sum(0)[None, :, None]
    return out, rows(lse).flatten(1), slack.flatten(1, 2), rows(err + 2 * (n + 8) * U * 1.0).flatten(1)


def check_forward(q, k, v, starts, out, lse, scale=None, before=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    bounds = starts.tolist()
    touched = torch.zeros(q.shape[1], dtype=torch.bool, device="cuda")
    for r in range(q.shape[0]):
        for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if a == b:
                continue
            touched[a:b] = True
            keys, values = (x[r, a:b] if before is None else x[i][r] for x in (k, v))
            o, l, slack, lslack = attend(q[r, a:b], keys, values, 0 if before is None else before[i], scale)
            close(out[r, a:b], o, slack, f"out {r} {i}")
            if lse is not None:
                fine = l.isfinite()
                assert torch.equal(lse[r, a:b][~fine].double(), l[~fine])
                close(lse[r, a:b][fine], l[fine], lslack[fine] + U * l[fine].abs(), f"lse {r} {i}")
    assert bool((out[:, ~touched] == MARK).all())
    if lse is not None:
        assert bool((lse[:, ~touched] == MARK).all())


def workspace(q, kv):
    n, t, heads, d = q.shape
    return B.OpWorkspace(B.prompt_attention_workspace_bytes(n, t, heads, kv, d))


def prompt_inputs(ranks, lens, q_heads, kv_heads, dim, dtype, seed=0, ahead=0, behind=0, scale=1.0):
    g, t = gen(seed), ahead + sum(lens) + behind
    dtype = DT[dtype]
    q = normal(g, ranks, t, q_heads, dim, dtype=dtype, scale=scale)
    k = normal(g, ranks, t, kv_heads, dim, dtype=dtype, scale=scale)
    # values are a view of the projection's output
    v = normal(g, ranks, t, (q_heads + 2 * kv_heads) * dim, dtype=dtype)[:, :, (q_heads + kv_heads) * dim:]
    return q, k, v.unflatten(2, (kv_heads, dim)), starts_of(lens, ahead)


def forward(q, k, v, starts, with_lse=True, ws=None, **kw):
    out = torch.full_like(q, MARK)
    lse = torch.full(q.shape[:3], MARK, device="cuda") if with_lse else None
    ws = ws or workspace(q, k.shape[2])
    B.prompt_attention(q, k, v, starts, out, lse, ws, **kw)
    assert B.get_status(ws) == B.Status.OK
    return out, lse


PROMPTS = [
    (1, [1], 1, 1, 64, "bf16"), (1, [1], 8, 1, 128, "f32"), (1, [97], 8, 1, 128, "bf16"),
    (2, [0, 1, 0, 130, 64, 128, 129, 0], 4, 2, 64, "bf16"), (2, [5, 0, 70, 64], 4, 2, 64, "f32"),
    (1, [300], 4, 4, 128, "bf16"), (1, [257, 255, 256], 1, 1, 128, "bf16"), (1, [1025], 2, 1, 128, "bf16"),
    (3, [40, 33], 6, 2, 80, "bf16"), (3, [40, 33], 6, 2, 80, "f32"), (1, [50, 61], 7, 1, 96, "bf16"),
    (1, [77], 10, 2, 40, "bf16"), (1, [130], 3, 3, 8, "bf16"), (1, [130], 3, 1, 24, "f32"), (1, [201], 5, 5, 72, "bf16"),
    (2, [66, 3], 4, 2, 136, "bf16"), (2, [100], 2, 1, 192, "bf16"), (1, [140, 5], 4, 1, 256, "bf16"),
    (1, [90], 2, 2, 256, "f32"), (1, [70], 2, 2, 160, "f32"), (1, [9, 30], 130, 1, 64, "bf16"), (1, [3, 20], 128, 1, 128, "bf16"),
    (1, [11], 100, 1, 64, "f32"), (1, [45], 96, 2, 128, "bf16"), (8, [64, 300, 1, 7], 8, 1, 128, "bf16"),
    (32, [17, 9], 2, 1, 64, "bf16"), (1, [1] * 150, 8, 2, 64, "bf16"), (1, [700, 1300], 3, 1, 64, "bf16"),
    # few key heads of long sequences, whose rows are split
    (1, [1100, 30], 16, 2, 128, "bf16"), (2, [1500], 16, 1, 64, "bf16"), (1, [600, 0, 9], 16, 2, 64, "f32"),
    (1, [400], 8, 1, 192, "bf16"), (1, [333], 16, 1, 96, "f32"),
]


@pytest.mark.parametrize("ranks,lens,q_heads,kv_heads,dim,dtype", PROMPTS, ids=str)
def test_prompt(ranks, lens, q_heads, kv_heads, dim, dtype):
    q, k, v, starts = prompt_inputs(ranks, lens, q_heads, kv_heads, dim, dtype)
    out, lse = forward(q, k, v, starts)
    check_forward(q, k, v, starts, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_rows_in_no_sequence(dtype):
    """Tokens ahead of the first sequence and behind the last one: what they hold does not matter, their rows stay."""
    q, k, v, starts = prompt_inputs(2, [100, 0, 37], 4, 2, 64, dtype, ahead=5, behind=150)
    for x in (q, k, v):
        x[:, :5] = float("nan")
        x[:, 142:] = float("inf")
    out, lse = forward(q, k, v, starts)
    check_forward(q, k, v, starts, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_sequences_do_not_meet(dtype):
    """A NaN or infinity of one sequence is in no row of another."""
    q, k, v, starts = prompt_inputs(1, [70, 60, 90], 4, 2, 64, dtype)
    want, _ = forward(q, k, v, starts)
    v[:, 71:75] = float("nan")
    k[:, 80] = float("inf")
    q[:, 100] = float("nan")
    out, _ = forward(q, k, v, starts)
    assert torch.equal(out[:, :70], want[:, :70]) and torch.equal(out[:, 130:], want[:, 130:])
    assert bool(out[:, 75:130].isnan().all())


@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.3, 1.0), (1.0, 3.0), (0.02, 20.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_scales(scale, size, dtype):
    """No scale, a negative one, scores of hundreds."""
    q, k, v, starts = prompt_inputs(1, [333, 40], 4, 1, 64, dtype, seed=3, scale=size)
    out, lse = forward(q, k, v, starts, scale=scale)
    check_forward(q, k, v, starts, out, lse, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_layouts(dtype):
    """Lists of the ranks' tensors with gaps between rows, heads of one buffer side by side, no lse."""
    n, t, heads, kv, d = 3, 140, 4, 2, 64
    g = gen(1)
    dt = DT[dtype]
    buffers = [normal(g, t, (heads + 2 * kv) * d + 16, dtype=dt) for _ in range(n)]
    outs = torch.full((t, n, heads + 1, d), MARK, dtype=dt, device="cuda")
    q = [b[:, :heads * d].unflatten(1, (heads, d)) for b in buffers]
    k = [b[:, heads * d:(heads + kv) * d].unflatten(1, (kv, d)) for b in buffers]
    v = [b[:, (heads + kv) * d:(heads + 2 * kv) * d].unflatten(1, (kv, d)) for b in buffers]
    out = [outs[:, r, :heads] for r in range(n)]
    starts = starts_of([100, 40])
    ws = B.OpWorkspace(B.prompt_attention_workspace_bytes(n, t, heads, kv, d))
    B.prompt_attention(q, k, v, starts, out, None, ws)
    assert B.get_status(ws) == B.Status.OK
    check_forward(torch.stack(q), torch.stack(k), torch.stack(v), starts, torch.stack(out), None)
    assert bool((outs[:, :, heads] == MARK).all())


def paged(g, n, lens, kv, d, page, dtype, spare=3, extra_columns=1):
    """Caches with random pages of the requests, all else NaN; a table; and each request's keys and values."""
    have = [-(-v // page) for v in lens]
    pages = sum(have) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(pages)).tolist()
    k, v = (torch.full((n, pages, kv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    table, keys, values = [], [], []
    for length, count in zip(lens, have):
        mine, order = order[:count], order[count:]
        table.append(mine + [-7] * (max(have) + extra_columns - count))
        key, value = (normal(g, n, length, kv, d, dtype=dtype) for _ in range(2))
        keys.append(key)
        values.append(value)
        for c, p in enumerate(mine):
            m = min(page, length - c * page)
            k[:, p, :, :m] = key[:, c * page:c * page + m].transpose(1, 2)
            v[:, p, :, :m] = value[:, c * page:c * page + m].transpose(1, 2)
    return k, v, torch.tensor(table, dtype=torch.int32, device="cuda"), keys, values


CACHED = [
    (1, [1], [1], 8, 1, 64, 16, "bf16"), (1, [5], [3000], 16, 2, 128, 64, "bf16"), (1, [5], [3000], 16, 2, 128, 64, "f32"),
    (2, [1, 40, 130, 0, 3], [1, 40, 300, 17, 129], 4, 2, 64, 16, "bf16"), (2, [1, 40, 130, 0, 3], [1, 40, 300, 17, 129], 4, 2, 64, 16, "f32"),
    (1, [33, 64], [333, 600], 8, 1, 128, 1, "bf16"), (1, [20, 9], [60, 50], 6, 2, 80, 2, "bf16"),
    (1, [33, 64], [333, 600], 8, 1, 128, 4, "bf16"), (1, [33, 64], [333, 600], 7, 1, 96, 8, "bf16"),
    (1, [200], [700], 4, 4, 128, 256, "bf16"), (1, [200, 3], [1500, 1024], 4, 4, 64, 1024, "bf16"),
    (1, [31], [200], 4, 2, 192, 32, "bf16"), (1, [31], [200], 4, 2, 256, 128, "f32"), (8, [256, 100], [900, 4100], 8, 1, 128, 32, "bf16"),
    (1, [2], [20000], 4, 1, 128, 16, "bf16"), (1, [1, 2, 1], [5000, 9, 12345], 8, 2, 64, 16, "bf16"),
    (1, [1], [9001], 5, 1, 40, 128, "f32"),
]


def cached_forward(q, k, v, table, starts, lens, ws=None, status=B.Status.OK, **kw):
    out = torch.full_like(q, MARK)
    lse = torch.full(q.shape[:3], MARK, device="cuda")
    ws = ws or workspace(q, k.shape[2])
    B.prompt_attention_cached(q, k, v, table, starts, lens, out, lse, ws, **kw)
    assert B.get_status(ws) == status
    return out, lse


@pytest.mark.parametrize("ranks,new,lens,q_heads,kv_heads,dim,page,dtype", CACHED, ids=str)
def test_cached(ranks, new, lens, q_heads, kv_heads, dim, page, dtype):
    g = gen(len(lens) * dim)
    k, v, table, keys, values = paged(g, ranks, lens, kv_heads, dim, page, DT[dtype])
    q = normal(g, ranks, sum(new) + 2, q_heads, dim, dtype=DT[dtype])
    starts = starts_of(new)
    out, lse = cached_forward(q, k, v, table, starts, i32(*lens))
    check_forward(q, keys, values, starts, out, lse, before=[a - b for a, b in zip(lens, new)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cached_not_a_number_in_a_part(dtype):
    """A query of NaN, and a key of NaN that later rows alone see, where the keys are split over blocks."""
    new, lens = [6], [4000]
    g = gen(8)
    k, v, table, keys, values = paged(g, 1, lens, 1, 64, 16, DT[dtype])
    q = normal(g, 1, 6, 4, 64, dtype=DT[dtype])
    want, want_lse = cached_forward(q, k, v, table, starts_of(new), i32(*lens))
    q[:, 2, 1] = float("nan")
    page = int(table[0, 3997 // 16])
    k[:, page, 0, 3997 % 16] = float("nan")
    out, lse = cached_forward(q, k, v, table, starts_of(new), i32(*lens))
    bad = torch.zeros(1, 6, 4, dtype=torch.bool, device="cuda")
    bad[:, 2, 1] = True
    bad[:, 3:] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad) and torch.equal(lse.isnan(), bad)
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cached_rows_that_see_nothing(dtype):
    """Requests that were refused: their lengths are below the step's tokens, down to nothing at all."""
    new, lens = [10, 20, 5], [4, 0, 5]
    g = gen(5)
    k, v, table, keys, values = paged(g, 2, lens, 2, 64, 16, DT[dtype])
    q = normal(g, 2, sum(new), 4, 64, dtype=DT[dtype])
    starts = starts_of(new)
    out, lse = cached_forward(q, k, v, table, starts, i32(*lens))
    check_forward(q, keys, values, starts, out, lse, before=[a - b for a, b in zip(lens, new)])
    assert bool((out[:, :6] == 0).all()) and bool((lse[:, 10:30] == float("-inf")).all())


@pytest.mark.parametrize("new,lens", [([10, 20, 5], [4, 0, 5]), ([30], [11]), ([7], [0]), ([3, 0, 40, 1], [3, 9, 700, 0])])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cached_rows_that_see_nothing_in_parts(new, lens, dtype):
    """The same where the table has room for many keys, so that rows are joined from parts, most of them of no key."""
    g = gen(6)
    k, v, table, keys, values = paged(g, 1, lens, 1, 64, 16, DT[dtype], extra_columns=400)
    q = normal(g, 1, sum(new), 4, 64, dtype=DT[dtype])
    starts = starts_of(new)
    out, lse = cached_forward(q, k, v, table, starts, i32(*lens))
    check_forward(q, keys, values, starts, out, lse, before=[a - b for a, b in zip(lens, new)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cached_bad_numbers(dtype):
    """Pages that are none are left out, lengths past the table row are cut to it; the status says so, later calls run."""
    new, lens, page = [10, 150, 20], [300, 320, 100], 16
    g = gen(6)
    k, v, table, keys, values = paged(g, 1, lens, 2, 64, page, DT[dtype], extra_columns=0)
    q = normal(g, 1, sum(new), 4, 64, dtype=DT[dtype])
    starts = starts_of(new)
    good, good_lse = cached_forward(q, k, v, table, starts, i32(*lens))
    ws = workspace(q, 2)
    for bad in (-1, k.shape[1], 2 ** 31 - 1):
        broken = table.clone()
        broken[1, 3] = bad
        out, lse = cached_forward(q, k, v, broken, starts, i32(*lens), ws, B.Status.ERR_CAPACITY)
        assert torch.equal(out[:, :10], good[:, :10]) and torch.equal(out[:, 160:], good[:, 160:])
        left = [torch.cat([x[1][:, :48], x[1][:, 64:]], 1) for x in (keys, values)]
        # keys ahead of every row's position are gone: the rest as if the sequence were 16 shorter
        o, l, slack, lslack = attend(q[0, 10:160], left[0][0], left[1][0], 170 - 16, 64 ** -0.5)
        close(out[0, 10:160], o, slack)
        close(lse[0, 10:160], l, lslack + U * l.abs())
    width = table.shape[1] * page  # the second request's row is full: longer, its rows see no more than that
    out, lse = cached_forward(q, k, v, table, starts, i32(300, width + 30, 100), ws, B.Status.ERR_CAPACITY)
    o, l, slack, lslack = attend(q[0, 10:160], keys[1][0], values[1][0], 320 + 30 - 150, 64 ** -0.5)
    close(out[0, 10:160], o, slack)
    cached_forward(q, k, v, table, starts, i32(300, -3, 100), ws, B.Status.ERR_CAPACITY)
    out, lse = cached_forward(q, k, v, table, starts, i32(*lens), ws)
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("starts", [[0, 50, 20, 90], [-3, 20], [0, 500], [95, 90], [2 ** 31 - 1, 5], [0, -1, 10]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_starts(starts, dtype):
    q, k, v, good = prompt_inputs(1, [90], 4, 2, 64, dtype)
    ws = workspace(q, 2)
    out, lse = torch.full_like(q, MARK), torch.full(q.shape[:3], MARK, device="cuda")
    B.prompt_attention(q, k, v, i32(*starts), out, lse, ws)
    assert B.get_status(ws) == B.Status.ERR_CAPACITY
    grads = [torch.full_like(x, MARK) for x in (q, k, k)]
    B.prompt_attention_backward(q, k, v, i32(*starts), out, lse, q, *grads, ws)
    assert B.get_status(ws) == B.Status.ERR_CAPACITY
    out, lse = forward(q, k, v, good, ws=ws)
    check_forward(q, k, v, good, out, lse)


# ---------------------------------------------------------------- gradient
def check_backward(q, k, v, starts, out, lse, dout, dq, dk, dv, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    n, t, heads, d = q.shape
    kv, bounds = k.shape[2], starts.tolist()
    touched = torch.zeros(t, dtype=torch.bool, device="cuda")
    for r in range(n):
        for a, b in zip(bounds, bounds[1:]):
            if a == b:
                continue
            touched[a:b] = True
            x, key, value, g, o = (z[r, a:b].double() for z in (q, k, v, dout, out))
            x, g, o = (z.unflatten(1, (kv, heads // kv)) for z in (x, g, o))
            s, sees, e = scores(q[r, a:b], k[r, a:b], 0, scale)
            l = lse[r, a:b].double().unflatten(1, (kv, heads // kv)).permute(1, 2, 0)[..., None]
            p = torch.where(sees, torch.exp(s - l), 0.0)
            err = e + 4 * U * (s.abs() + l.abs()) + 8 * U
            dp = torch.einsum("thgd,shd->hgts", g, value)
            dsize = torch.einsum("thgd,shd->hgts", g.abs(), value.abs())
            delta = (g * o).sum(-1).permute(1, 2, 0)[..., None]
            lsize = (g * o).abs().sum(-1).permute(1, 2, 0)[..., None]
            ds = p * (dp - delta)
            tiny = torch.where(sees, TINY, 0.0)
            mass = torch.einsum("hgts,shd->thgd", p, value.abs())
            left = (torch.where(sees, err, 0.0).amax(-1) * 2 + cut(q) + 2 * (b - a + 8) * U).permute(2, 0, 1)[..., None] * mass
            ddelta = (g.abs() * (left + ROUND[q.dtype] * o.abs())).sum(-1).permute(1, 2, 0)[..., None] + \
                (p * (dp.abs() * err + 2 * (d + 4) * U * dsize)).sum(-1, keepdim=True)
            eds = p * (2 * (d + 4) * U * (dsize + lsize) + ddelta) + ds.abs() * (err + cut(q) + 4 * U) + tiny * (dp - delta).abs()
            ep = p * (err + cut(q)) + tiny
            rows, cols = 2 * (b - a + 8) * U, 2 * ((b - a) * (heads // kv) + 8) * U
            want = torch.einsum("hgts,shd->thgd", ds, key).flatten(1, 2) * scale
            slack = torch.einsum("hgts,shd->thgd", eds + rows * ds.abs(), key.abs()).flatten(1, 2) * abs(scale)
            close(dq[r, a:b], want, slack + 2 * U * want.abs(), "dq")
            want = torch.einsum("hgts,thgd->shd", ds, x) * scale
            slack = torch.einsum("hgts,thgd->shd", eds + cols * ds.abs(), x.abs()) * abs(scale)
            close(dk[r, a:b], want, slack + 2 * U * want.abs(), "dk")
            close(dv[r, a:b], torch.einsum("hgts,thgd->shd", p, g),
                  torch.einsum("hgts,thgd->shd", ep + cols * p, g.abs()), "dv")
    for z in (dq, dk, dv):
        assert bool((z[:, ~touched] == MARK).all())


def backward(q, k, v, starts, out, lse, dout, ws=None, **kw):
    grads = [torch.full_like(x, MARK) for x in (q, k, k)]
    ws = ws or workspace(q, k.shape[2])
    B.prompt_attention_backward(q, k, v, starts, out, lse, dout, *grads, ws, **kw)
    assert B.get_status(ws) == B.Status.OK
    return grads


@pytest.mark.parametrize("ranks,lens,q_heads,kv_heads,dim,dtype", PROMPTS, ids=str)
def test_backward(ranks, lens, q_heads, kv_heads, dim, dtype):
    q, k, v, starts = prompt_inputs(ranks, lens, q_heads, kv_heads, dim, dtype, seed=1)
    out, lse = forward(q, k, v, starts)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    check_backward(q, k, v, starts, out, lse, dout, *backward(q, k, v, starts, out, lse, dout))


@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_of_one_key(dim, dtype):
    """A sequence's first token sees one key: no gradient through its score, exactly, and dv is dout."""
    q, k, v, starts = prompt_inputs(2, [1, 0, 1, 1, 1], 3, 3, dim, dtype, seed=5)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    out, lse = forward(q, k, v, starts)
    assert torch.equal(out, v)
    dq, dk, dv = backward(q, k, v, starts, out, lse, dout)
    assert bool((dq == 0).all()) and bool((dk == 0).all())
    close(dv, dout.double(), 1e-6 * dout.double().abs())
    q, k, v, starts = prompt_inputs(1, [300, 40], 6, 2, dim, dtype, seed=5)
    out, lse = forward(q, k, v, starts)
    dq = backward(q, k, v, starts, out, lse, normal(gen(9), *q.shape, dtype=q.dtype))[0]
    assert bool((dq[:, [0, 300]] == 0).all()) and bool((dq[:, [1, 301]] != 0).any())


@pytest.mark.parametrize("lens", [[2], [3, 1, 32], [17, 0, 9, 31], [128]], ids=str)
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_backward_of_few_tokens(lens, dim):
    """Calls of up to 128 tokens lose nothing to the roundings of weights: what those leave takes part (2^-17 of a
    weight or a score's gradient is lost), next to sums of 128 binary32 products (2^-17), the exponential of a score below 16
    (2^-19) and lse's rounding (2^-21): below 2^-15 in all, of terms that are multiplied twice; 2^-13 is allowed."""
    q, k, v, starts = prompt_inputs(2, lens, 6, 2, dim, "bf16", seed=6)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    out, lse = forward(q, k, v, starts)
    dq, dk, dv = backward(q, k, v, starts, out, lse, dout)
    bounds = starts.tolist()
    for r in range(2):
        for a, b in zip(bounds, bounds[1:]):
            if a == b:
                continue
            x, key, value, g = (z[r, a:b].double() for z in (q, k, v, dout))
            x, g = (z.unflatten(1, (2, 3)) for z in (x, g))
            s, sees, _ = scores(q[r, a:b], k[r, a:b], 0, dim ** -0.5)
            p = torch.softmax(s.masked_fill(~sees, float("-inf")), -1)
            dp = torch.einsum("thgd,shd->hgts", g, value)
            dsize = torch.einsum("thgd,shd->hgts", g.abs(), value.abs())
            delta = (p * dp).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            size = p * (dsize + (p * dsize).sum(-1, keepdim=True)) * 2 ** -13 * dim ** -0.5
            close(dq[r, a:b], torch.einsum("hgts,shd->thgd", ds, key).flatten(1, 2) * dim ** -0.5,
                  torch.einsum("hgts,shd->thgd", size, key.abs()).flatten(1, 2), "dq")
            close(dk[r, a:b], torch.einsum("hgts,thgd->shd", ds, x) * dim ** -0.5,
                  torch.einsum("hgts,thgd->shd", size, x.abs()), "dk")
            close(dv[r, a:b], torch.einsum("hgts,thgd->shd", p, g), 2 ** -13 * torch.einsum("hgts,thgd->shd", p, g.abs()), "dv")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_rows_in_no_sequence(dtype):
    q, k, v, starts = prompt_inputs(2, [100, 0, 37, 130], 6, 2, 64, dtype, ahead=5, behind=150)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    for x in (q, k, v, dout):
        x[:, :5] = float("nan")
        x[:, 272:] = float("inf")
    out, lse = forward(q, k, v, starts)
    out[:, 272:], lse[:, 272:] = float("nan"), float("nan")
    check_backward(q, k, v, starts, out, lse, dout, *backward(q, k, v, starts, out, lse, dout))


@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.3, 1.0), (0.02, 20.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_scales(scale, size, dtype):
    q, k, v, starts = prompt_inputs(1, [333, 40], 4, 1, 64, dtype, seed=3, scale=size)
    out, lse = forward(q, k, v, starts, scale=scale)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    check_backward(q, k, v, starts, out, lse, dout, *backward(q, k, v, starts, out, lse, dout, scale=scale), scale)


def test_backward_into_one_buffer():
    """dq, dk and dv side by side in the gradient of the projection, and lists of ranks with gaps between rows."""
    n, t, heads, kv, d = 2, 150, 4, 2, 64
    q, k, v, starts = prompt_inputs(n, [100, 50], heads, kv, d, "bf16")
    out, lse = forward(q, k, v, starts)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    want = backward(q, k, v, starts, out, lse, dout)
    buffer = torch.full((t, n, (heads + 2 * kv) * d + 8), MARK, dtype=q.dtype, device="cuda")
    part = lambda a, b: [buffer[:, r, a * d:b * d].unflatten(1, (b - a, d)) for r in range(n)]  # noqa: E731
    dq, dk, dv = part(0, heads), part(heads, heads + kv), part(heads + kv, heads + 2 * kv)
    ws = workspace(q, kv)
    B.prompt_attention_backward(q, k, v, starts, out, lse, dout, dq, dk, dv, ws)
    assert B.get_status(ws) == B.Status.OK
    for got, w in zip((dq, dk, dv), want):
        assert torch.equal(torch.stack(got), w)
    assert bool((buffer[:, :, -8:] == MARK).all())


def test_backward_against_differences():
    """The derivative of sum(out * dout) along random directions, by differences of the 64-bit form, whose step of 1e-4
    leaves an error of order 1e-8 times the third derivative (of order of the gradient's size here); the kernel's own
    roundings, in binary32, are some 1e-6 of the sum of the magnitudes."""
    q, k, v, starts = prompt_inputs(1, [40, 23], 4, 2, 16, "f32", seed=4)
    out, lse = forward(q, k, v, starts)
    dout = normal(gen(8), *q.shape)
    grads = backward(q, k, v, starts, out, lse, dout)
    g, h = gen(7), 1e-4

    def value(x):
        total = 0.0
        for a, b in zip(starts.tolist(), starts.tolist()[1:]):
            o = attend(*(z[0, a:b] for z in x), 0, 0.25)[0]
            total += float((o * dout[0, a:b].double()).sum())
        return total

    for i in range(3):
        x = [z.double() for z in (q, k, v)]
        step = normal(g, *x[i].shape).double()
        slope = 0.0
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * h * step
            ROUND[torch.float64] = 0.0
            slope += sign * value(y) / (2 * h)
        mine = grads[i].double() * step
        assert abs(float(mine.sum()) - slope) <= 1e-5 * float(mine.abs().sum())


# ---------------------------------------------------------------- streams, graphs, repetition
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits(dtype):
    q, k, v, starts = prompt_inputs(2, [500, 77], 6, 2, 64, dtype)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    first = None
    for _ in range(5):
        out, lse = forward(q, k, v, starts)
        found = [out, lse, *backward(q, k, v, starts, out, lse, dout)]
        first = first or found
        assert all(torch.equal(a, b) for a, b in zip(first, found))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_of_a_step(dtype):
    """Embedding, attention and all gradients captured once and replayed on other tokens and other starts, on another
    stream, with one workspace; a second graph with a workspace of its own in between."""
    n, t, heads, kv, d, words = 2, 200, 4, 2, 64, 77
    hidden = (heads + 2 * kv) * d
    dt = DT[dtype]

    class Step:
        def __init__(self, seed):
            g = gen(seed)
            self.tables = normal(g, n, words, hidden, dtype=dt)
            self.tokens, self.starts = torch.zeros(t, dtype=torch.int32, device="cuda"), starts_of([0, 0, 0])
            self.x = torch.zeros(t, hidden, dtype=dt, device="cuda")
            self.out, self.dout = (torch.zeros(n, t, heads, d, dtype=dt, device="cuda") for _ in range(2))
            self.lse = torch.zeros(n, t, heads, device="cuda")
            self.dout.copy_(normal(g, n, t, heads, d))
            self.dx = torch.zeros(n, t, hidden, dtype=dt, device="cuda")
            self.dtables = torch.zeros(n, words, hidden, device="cuda")
            self.ws = B.OpWorkspace(max(B.prompt_attention_workspace_bytes(n, t, heads, kv, d),
                                        B.embed_tokens_workspace_bytes(t, hidden)))

        def parts(self, x):
            at = (0, heads * d, (heads + kv) * d, hidden)
            return [x[..., a:b].unflatten(-1, (-1, d)) for a, b in zip(at, at[1:])]

        def run(self):
            B.embed_tokens(self.tokens, self.tables, self.x, self.ws, scale=2.0)
            q, k, v = ([z] * n for z in self.parts(self.x))  # every rank attends with the same rows
            B.prompt_attention(q, k, v, self.starts, self.out, self.lse, self.ws)
            self.dx.zero_()
            B.prompt_attention_backward(q, k, v, self.starts, list(self.out), self.lse, self.dout,
                                        *self.parts(self.dx), self.ws)
            B.embed_tokens_backward(self.tokens, self.dx[0], self.dtables, self.ws, scale=2.0)

        def check(self):
            assert B.get_status(self.ws) == B.Status.OK
            flat = self.tables.flatten(0, 1)
            close(self.x, flat[self.tokens.long()].double() * 2, 0)
            q, k, v = (z[None].expand(n, *z.shape) for z in self.parts(self.x))
            a, b = self.starts.tolist()[0], self.starts.tolist()[-1]
            bounds = self.starts - a
            check_forward(q[:, a:b], k[:, a:b], v[:, a:b], bounds, self.out[:, a:b], self.lse[:, a:b])
            check_backward(q[:, a:b], k[:, a:b], v[:, a:b], bounds, self.out[:, a:b], self.lse[:, a:b], self.dout[:, a:b],
                           *(z[:, a:b] for z in self.parts(self.dx)))
            check_table_gradient(self.tokens, self.dx[0], list(self.dtables), 2.0)

    steps = [Step(1), Step(2)]
    graphs = []
    side = torch.cuda.Stream()
    for s in steps:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        graphs.append(graph)
    for turn, lens in enumerate(([100, 60, 40], [1, 0, 199], [130, 70, 0])):
        for s, graph in zip(steps, graphs):
            s.tokens.copy_(torch.randint(0, n * words, (t,), generator=gen(turn), device="cuda"))
            s.starts.copy_(starts_of(lens))
            graph.replay()
        for s in steps:
            s.check()


def test_two_streams():
    """Calls on two streams with a workspace each."""
    q, k, v, starts = prompt_inputs(1, [900], 4, 1, 64, "bf16")
    want, _ = forward(q, k, v, starts)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [workspace(q, 1) for _ in streams]
    outs = [torch.empty_like(q) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, spaces, outs):
            B.prompt_attention(q, k, v, starts, o, None, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_nothing_to_do():
    q, k, v, starts = prompt_inputs(1, [], 4, 2, 64, "bf16", behind=10)
    ws = workspace(q, 2)
    out = torch.full_like(q, MARK)
    B.prompt_attention(q, k, v, starts, out, None, ws)          # no sequences
    B.prompt_attention(q[:, :0], k[:, :0], v[:, :0], starts, out[:, :0], None, ws)  # no tokens
    B.prompt_attention(q, k, v, i32(0, 0, 0), out, None, ws)    # empty sequences
    assert B.get_status(ws) == B.Status.OK and bool((out == MARK).all())


# ---------------------------------------------------------------- embedding
def check_table_gradient(tokens, dout, dtables, scale, base=None):
    words = sum(x.shape[0] for x in dtables)
    inside = (tokens >= 0) & (tokens < words)
    at = tokens[inside].long()
    want, size = (torch.zeros(words, dout.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    want.index_add_(0, at, dout[inside].double() * scale)
    size.index_add_(0, at, dout[inside].double().abs() * abs(scale))
    count = torch.zeros(words, device="cuda", dtype=torch.float64).index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    slack = (count[:, None] + 2) * U * size
    got = torch.cat(dtables)
    if base is not None:
        want = want + base.double()
        slack = slack + U * want.abs()
        assert torch.equal(got[count == 0], base[count == 0])
    close(got, want, slack, "dtable")


EMBED = [
    (1, [1], 8, 1, "bf16"), (2, [5, 9], 16, 0, "f32"), (8, [100] * 8, 4096, 7, "bf16"), (3, [50, 1, 33], 520, 300, "bf16"),
    (3, [50, 1, 33], 1032, 300, "f32"), (32, [3] * 32, 64, 1000, "bf16"), (2, [4000, 4001], 256, 9000, "bf16"),
    (1, [3], 264, 8193, "f32"), (4, [30, 20, 10, 5], 72, 40000, "bf16"), (1, [50000], 2048, 2500, "bf16"),
]


def embed_inputs(vocab, hidden, count, dtype, seed=0):
    g, words = gen(seed), sum(vocab)
    tables = [normal(g, v, hidden, dtype=DT[dtype]) for v in vocab]
    # some words far more often than others, some tokens of no word
    tokens = ((words + 1.0) ** torch.rand(count, generator=g, device="cuda", dtype=torch.float64) - 1).int()
    tokens[::7] = -1
    tokens[3::50] = words
    return tables, tokens


@pytest.mark.parametrize("ranks,vocab,hidden,count,dtype", EMBED, ids=str)
def test_embed(ranks, vocab, hidden, count, dtype):
    tables, tokens = embed_inputs(vocab, hidden, count, dtype)
    out = torch.full((count, hidden), MARK, dtype=DT[dtype], device="cuda")
    ws = B.OpWorkspace()
    B.embed_tokens(tokens, tables, out, ws, scale=1.7)
    assert B.get_status(ws) == B.Status.OK
    words = sum(vocab)
    inside = (tokens >= 0) & (tokens < words)
    want = torch.cat(tables)[tokens.clamp(0, words - 1).long()].float() * torch.tensor(1.7, device="cuda")
    assert torch.equal(out, torch.where(inside[:, None], want, 0.0).to(out.dtype))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("ranks,vocab,hidden,count,dtype", EMBED, ids=str)
def test_embed_backward(ranks, vocab, hidden, count, dtype, accumulate):
    tables, tokens = embed_inputs(vocab, hidden, count, dtype)
    dout = normal(gen(3), count, hidden, dtype=DT[dtype])
    grads = [normal(gen(r), v, hidden) for r, v in enumerate(vocab)]
    base = torch.cat(grads).clone()
    ws = B.OpWorkspace(B.embed_tokens_workspace_bytes(count, hidden))
    B.embed_tokens_backward(tokens, dout, grads, ws, scale=0.3, accumulate=accumulate)
    assert B.get_status(ws) == B.Status.OK
    check_table_gradient(tokens, dout, grads, float(torch.tensor(0.3, dtype=torch.float32)), base if accumulate else None)
    again = [normal(gen(r), v, hidden) for r, v in enumerate(vocab)]
    B.embed_tokens_backward(tokens, dout, again, ws, scale=0.3, accumulate=accumulate)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("count", [31, 32, 33, 700, 20000])
@pytest.mark.parametrize("tokens", ["one", "two", "none", "all"])
def test_embed_backward_distributions(count, tokens):
    """One word for all tokens, two that alternate, none at all, each word once or so."""
    i = torch.arange(count, device="cuda", dtype=torch.int32)
    token = {"one": i * 0 + 4, "two": i % 2 * 6, "none": i * 0 - 1, "all": i.flip(0) % 20011}[tokens]
    vocab, hidden = [7, 20004], 264
    dout = normal(gen(3), count, hidden, dtype=torch.bfloat16)
    grads = [torch.full((v, hidden), MARK, device="cuda") for v in vocab]
    ws = B.OpWorkspace(B.embed_tokens_workspace_bytes(count, hidden))
    B.embed_tokens_backward(token, dout, grads, ws)
    check_table_gradient(token, dout, grads, 1.0)


@pytest.mark.parametrize("count,hidden", [(304, 2048), (305, 2048), (512, 64), (513, 64), (1024, 1032), (1025, 1032),
                                          (65536, 64), (65537, 64), (140001, 8)])
@pytest.mark.parametrize("words", [9, 70000])
def test_embed_backward_counts(count, hidden, words):
    """On both sides of the numbers of tokens at which another form begins; few words, and more than there are tokens."""
    vocab = [words // 3, words - words // 3]
    token = torch.randint(-1, words + 1, (count,), generator=gen(count), device="cuda").int()
    dout = normal(gen(3), count, hidden, dtype=torch.bfloat16)
    ws = B.OpWorkspace(B.embed_tokens_workspace_bytes(count, hidden))
    for accumulate in (False, True):
        grads = [normal(gen(r), v, hidden) for r, v in enumerate(vocab)]
        base = torch.cat(grads).clone()
        B.embed_tokens_backward(token, dout, grads, ws, accumulate=accumulate)
        check_table_gradient(token, dout, grads, 1.0, base if accumulate else None)
    assert B.get_status(ws) == B.Status.OK


def test_embed_layouts():
    """Rows with gaps: tables in one buffer side by side, outputs and gradients strided; infinities and NaN of words that
    no token asks for do not matter, and those of tokens that ask for nothing neither."""
    n, vocab, hidden, count = 2, 40, 64, 90
    g = gen(2)
    store = normal(g, vocab, n, hidden + 8, dtype=torch.bfloat16)
    tables = [store[:, r, :hidden] for r in range(n)]
    tokens = torch.randint(0, n * vocab, (count,), generator=g, device="cuda").int()
    tokens[tokens == 11] = 12
    tokens[5] = -4
    store[11, 0] = float("nan")
    rows = torch.full((count, hidden + 8), MARK, dtype=torch.bfloat16, device="cuda")
    ws = B.OpWorkspace(B.embed_tokens_workspace_bytes(count, hidden))
    B.embed_tokens(tokens, tables, rows[:, :hidden], ws)
    want = torch.cat(tables)[tokens.long().clamp(min=0)]
    want[5] = 0
    assert torch.equal(rows[:, :hidden], want) and bool((rows[:, hidden:] == MARK).all())
    dout = normal(g, count, hidden + 8, dtype=torch.bfloat16)
    dout[5] = float("inf")
    buffer = torch.full((vocab, n, hidden + 8), MARK, device="cuda")
    grads = [buffer[:, r, :hidden] for r in range(n)]
    B.embed_tokens_backward(tokens, dout[:, :hidden], grads, ws)
    check_table_gradient(tokens, dout[:, :hidden], [x.contiguous() for x in grads], 1.0)
    assert bool((buffer[:, :, hidden:] == MARK).all())


def test_embed_nothing():
    ws = B.OpWorkspace(1 << 20)
    grads = [torch.full((9, 64), MARK, device="cuda")]
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    rows = torch.zeros(0, 64, device="cuda")
    B.embed_tokens(none, grads, rows, ws)
    B.embed_tokens_backward(none, rows, grads, ws, accumulate=True)
    assert bool((grads[0] == MARK).all())
    B.embed_tokens_backward(none, rows, grads, ws)
    assert B.get_status(ws) == B.Status.OK and bool((grads[0] == 0).all())


MANY = [
    ([i * 37 % 190 for i in range(45)], 8, 2, 128, "bf16"), ([i * 37 % 190 for i in range(33)], 3, 1, 64, "bf16"),
    ([0, 0, 1] * 700, 4, 4, 64, "bf16"), ([i * 37 % 90 for i in range(45)], 4, 2, 64, "f32"), ([0] * 40 + [300] + [0] * 2000, 8, 1, 64, "bf16"),
]


@pytest.mark.parametrize("lens,q_heads,kv_heads,dim,dtype", MANY, ids=lambda x: None if isinstance(x, list) else str(x))
def test_many_sequences(lens, q_heads, kv_heads, dim, dtype):
    """More than a warp has lanes, which are taken in another order."""
    q, k, v, starts = prompt_inputs(2, lens, q_heads, kv_heads, dim, dtype, seed=4, ahead=3)
    out, lse = forward(q, k, v, starts)
    check_forward(q, k, v, starts, out, lse)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    check_backward(q, k, v, starts, out, lse, dout, *backward(q, k, v, starts, out, lse, dout))


@pytest.mark.parametrize("page,dtype", [(64, "bf16"), (4, "bf16"), (64, "f32")])
def test_cached_far(page, dtype):
    """Pages whose elements' numbers pass 32 bits."""
    d, kv, heads, new, lens = 128, 2, 4, [9, 200], [500, 340]
    pages = (2 ** 32 + 2 ** 20) // (kv * page * d)
    g = gen(7)
    k, v = (torch.empty(1, pages, kv, page, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    have = [-(-n // page) for n in lens]
    near, far = list(range(have[0])), [pages - 1 - i for i in range(have[1])]
    far[1] = pages // 2 - 1
    keys, values, rows = [], [], []
    for n, mine in zip(lens, (near, far)):
        key, value = (normal(g, 1, n, kv, d, dtype=DT[dtype]) for _ in range(2))
        for c, at in enumerate(mine):
            m = min(page, n - c * page)
            k[:, at, :, :m] = key[:, c * page:c * page + m].transpose(1, 2)
            v[:, at, :, :m] = value[:, c * page:c * page + m].transpose(1, 2)
        keys.append(key)
        values.append(value)
        rows.append(mine + [0] * (max(have) - len(mine)))
    q = normal(g, 1, sum(new), heads, d, dtype=DT[dtype])
    starts = starts_of(new)
    out, lse = cached_forward(q, k, v, i32(*sum(rows, [])).view(2, -1), starts, i32(*lens))
    check_forward(q, keys, values, starts, out, lse, before=[a - b for a, b in zip(lens, new)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_far_apart(dtype):
    """Rows whose elements' numbers pass 32 bits, of all tensors in one buffer."""
    t, heads, kv, d = 150, 4, 2, 64
    stride = 2 ** 32 // 140
    stride -= stride % 8
    buffer = torch.empty(t * stride, dtype=DT[dtype], device="cuda")
    q, k, v, starts = prompt_inputs(1, [20, 130], heads, kv, d, dtype)
    dout = normal(gen(9), *q.shape, dtype=q.dtype)
    out, lse = forward(q, k, v, starts)
    want = [out, *backward(q, k, v, starts, out, lse, dout)]
    at = 0

    def place(x):
        nonlocal at
        view = buffer.as_strided(x.shape, (t * stride, stride, d, 1), at)
        at += x.shape[2] * d
        return view.copy_(x)

    q, k, v, dout = (place(x) for x in (q, k, v, dout))
    out, dq, dk, dv = (place(torch.full_like(x, MARK)) for x in want)
    ws = workspace(q, kv)
    B.prompt_attention(q, k, v, starts, out, lse, ws)
    B.prompt_attention_backward(q, k, v, starts, out, lse, dout, dq, dk, dv, ws)
    assert B.get_status(ws) == B.Status.OK
    for got, w in zip((out, dq, dk, dv), want):
        assert torch.equal(got, w)


def test_embed_far():
    """A table, outputs and a gradient whose elements' numbers pass 32 bits."""
    words, hidden = 2 ** 32 // 4096 + 100, 4096
    table = torch.empty(words, hidden, dtype=torch.bfloat16, device="cuda")
    tokens = torch.randint(0, words, (3000,), generator=gen(1), device="cuda").int()
    tokens[:3] = i32(words - 1, words, 0)
    tokens[7] = words - 1
    used = tokens[tokens < words].long()
    table[used] = normal(gen(2), len(used), hidden, dtype=torch.bfloat16)
    ws = B.OpWorkspace(B.embed_tokens_workspace_bytes(len(tokens), hidden))
    out = torch.full((len(tokens), hidden), MARK, dtype=torch.bfloat16, device="cuda")
    B.embed_tokens(tokens, [table], out, ws)
    want = table[tokens.long().clamp(max=words - 1)]
    want[1] = 0
    assert torch.equal(out, want)
    del table
    grad = torch.full((words, hidden), MARK, device="cuda")
    B.embed_tokens_backward(tokens, out, [grad], ws)
    assert B.get_status(ws) == B.Status.OK
    row, place = torch.unique(used, return_inverse=True)
    part = torch.zeros(len(row), hidden, dtype=torch.float64, device="cuda").index_add_(0, place, out[tokens < words].double())
    size = torch.zeros_like(part).index_add_(0, place, out[tokens < words].double().abs())
    close(grad[row], part, 5 * U * size, "dtable")
    grad[row] = 0
    assert not bool(grad.any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspace_that_is_not_initialised(dtype):
    """The kernels write nothing but the status."""
    q, k, v, starts = prompt_inputs(1, [300, 20], 4, 2, 64, dtype)
    ws = workspace(q, 2)
    ws.buf.zero_()
    out, lse = torch.full_like(q, MARK), torch.full(q.shape[:3], MARK, device="cuda")
    B.prompt_attention(q, k, v, starts, out, lse, ws)
    assert B.get_status(ws) == B.Status.ERR_WORKSPACE
    grads = [torch.full_like(x, MARK) for x in (q, k, k)]
    B.prompt_attention_backward(q, k, v, starts, out, lse, q, *grads, ws)
    assert B.get_status(ws) == B.Status.ERR_WORKSPACE
    rows, tables = torch.full((20, 64), MARK, device="cuda"), torch.full((1, 9, 64), MARK, device="cuda")
    tokens = torch.zeros(20, dtype=torch.int32, device="cuda")
    B.embed_tokens(tokens, torch.zeros_like(tables), rows, ws)
    assert B.get_status(ws) == B.Status.ERR_WORKSPACE
    B.embed_tokens_backward(tokens, torch.zeros(20, 64, device="cuda"), tables, ws)
    assert B.get_status(ws) == B.Status.ERR_WORKSPACE
    for x in (out, lse, *grads, rows, tables):
        assert bool((x == MARK).all())
