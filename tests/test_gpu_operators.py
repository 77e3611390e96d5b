"""GPU tests of the operators around the collectives (page tables, norm and
rotation, decode attention, token log probabilities) against plain 64-bit
implementations of their formulas.

Tolerances. A result is the rounding to its type of a value whose distance from
the 64-bit one is bounded. u = 2^-24 is half an ulp of binary32: a binary32 sum of n terms is off by at most
about n u times the sum of the terms' magnitudes in any order; the bounds below
use that n (or, where partial sums are joined, a larger one) with the magnitudes
of the 64-bit computation, plus a few u for each exp, log, root and division.
"""
import pytest

torch = pytest.importorskip("torch")

from collective_communication_gb300 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def ints(n, fill=-7):
    return torch.full((n,), fill, dtype=torch.int32, device="cuda")


def close(got, want, slack, what=""):
    """got is the rounding to its type of some value within slack of want (64 bits, broadcast), everywhere."""
    lo, hi = ((want + d).to(got.dtype).double() for d in (-slack, slack))
    bad = ~(((lo <= got) & (got <= hi)) | (got.double() == want))
    err = (got.double() - want).abs()[bad]
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} values off, by up to {float(err.max())}"


# ---------------------------------------------------------------- page tables
def tables_by_hand(lens, new, free, count, table, page, capacity):
    table = [list(row) for row in table]
    width = len(table[0]) * page
    left, total, slots, positions, starts, out = count, 0, [], [], [], []
    blocked_pages = False
    for r, (have, more) in enumerate(zip(lens, new)):
        starts.append(total)
        valid = have >= 0 and more >= 0 and have + more <= width
        if not valid:
            out.append(have)
            continue
        columns = range(-(-have // page), -(-(have + more) // page))
        fits_pages = not columns or (not blocked_pages and len(columns) <= left)
        fits = fits_pages and total + more <= capacity
        if columns and not fits_pages:
            blocked_pages = True
        if fits:
            for c in columns:
                left -= 1
                table[r][c] = free[left]
        out.append(have + more if fits else have)
        for j in range(more):
            if total + j < capacity:
                positions.append(have + j if fits else 0)
                slots.append(table[r][(have + j) // page] * page + (have + j) % page if fits else -1)
        total += more
    starts.append(total)
    pad = capacity - len(slots)
    return table, out, starts, positions + [0] * pad, slots + [-1] * pad, left


def run_tables(lens, new, free, count, table, page, capacity, num_pages, stride=None):
    n = len(lens)
    t = torch.full((max(n, 1), stride or len(table[0])), -9, dtype=torch.int32, device="cuda")[:n, :len(table[0])]
    if n:
        t.copy_(torch.tensor(table, dtype=torch.int32))
    ws = B.OpWorkspace()
    outs = dict(lens_out=ints(n), starts=ints(n + 1), positions=ints(capacity), slots=ints(capacity),
                free_count_out=ints(1))
    B.page_tables(i32(*lens), i32(*new), i32(*free), i32(count), t, page, num_pages, workspace=ws, **outs)
    status = B.get_status(ws)
    return t, outs, status


@pytest.mark.parametrize("requests,page,most_new,slack,stride", [
    (1, 16, 1, 0, None), (1, 1, 5, 3, None), (3, 16, 40, 5, 64), (33, 8, 3, 0, None), (257, 32, 200, 100, None),
    (4096, 16, 2, 7, None), (4097, 64, 5, 0, 60), (9001, 16, 9, 1, None)])
def test_page_tables(requests, page, most_new, slack, stride):
    g = torch.Generator().manual_seed(requests)
    lens = torch.randint(0, 200, (requests,), generator=g).tolist()
    new = torch.randint(0, most_new + 1, (requests,), generator=g).tolist()
    blocks = -(-(200 + most_new) // page)
    used = sum(-(-v // page) for v in lens)
    pages = used + sum(new) // page + requests + 2
    order = torch.randperm(pages, generator=g).tolist()
    table, at = [], 0
    for v in lens:
        k = -(-v // page)
        table.append(order[at:at + k] + [-5] * (blocks - k))
        at += k
    free = order[at:]
    stride = None if stride is not None and stride < blocks else stride
    want = tables_by_hand(lens, new, free, len(free), table, page, sum(new) + slack)
    t, o, status = run_tables(lens, new, free, len(free), table, page, sum(new) + slack, pages, stride)
    assert status == B.Status.OK
    assert t.tolist() == want[0]
    got = [o[k].tolist() for k in ("lens_out", "starts", "positions", "slots")] + [int(o["free_count_out"])]
    assert got == list(want[1:])


@pytest.mark.parametrize("count,capacity,lens,new", [
    (2, 100, [16, 16, 16, 5], [1, 20, 1, 1]),    # the second wants two pages, one is left; the last needs none
    (9, 10, [3, 15, 0, 2], [4, 4, 5, 1]),        # the third does not fit the step's tokens
    (9, 100, [-1, 15, 3, 2], [4, -4, 46, 1]),    # negative length, negative count, longer than the table row
])
def test_page_tables_shortage(count, capacity, lens, new):
    page, blocks = 16, 3
    free = list(range(20, 20 + count))
    table = [[r * 3, r * 3 + 1, r * 3 + 2] for r in range(4)]
    want = tables_by_hand(lens, new, free, count, table, page, capacity)
    t, o, status = run_tables(lens, new, free, count, table, page, capacity, 64)
    assert status == B.Status.ERR_CAPACITY
    assert t.tolist() == want[0]
    got = [o[k].tolist() for k in ("lens_out", "starts", "positions", "slots")] + [int(o["free_count_out"])]
    assert got == list(want[1:])


def test_page_tables_bad_pages_and_count():
    # a page number past the cache in the free list and one in the table
    t, o, status = run_tables([16, 3], [1, 1], [99], 1, [[0, -1], [77, -1]], 16, 4, 64)
    assert status == B.Status.ERR_CAPACITY
    assert o["slots"].tolist() == [-1, -1, -1, -1] and t.tolist() == [[0, -1], [77, -1]]
    # a free count past the list is taken as the list's length
    t, o, status = run_tables([16], [1], [5], 3, [[0, -1]], 16, 1, 64)
    assert status == B.Status.ERR_CAPACITY and t.tolist() == [[0, 5]] and int(o["free_count_out"]) == 0


def test_page_tables_empty_and_replayed():
    t, o, status = run_tables([], [], [1, 2], 2, [[0, 0]], 16, 5, 64)
    assert status == B.Status.OK and o["slots"].tolist() == [-1] * 5 and o["starts"].tolist() == [0]
    assert int(o["free_count_out"]) == 2
    lens, new, table = i32(5, 16), i32(1, 1), torch.tensor([[3, 0], [4, 0]], dtype=torch.int32, device="cuda")
    outs = [ints(2), ints(3), ints(4), ints(4), ints(1)]
    ws = B.OpWorkspace()
    args = (lens, new, i32(8, 9), i32(2), table, 16, 64, *outs, ws)
    B.page_tables(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.page_tables(*args)
    lens.copy_(i32(15, 31))
    new.copy_(i32(3, 1))
    graph.replay()
    torch.cuda.synchronize()
    assert table.tolist() == [[3, 9], [4, 9]]  # 4, 9 from the first call: that page is listed already
    assert outs[3].tolist() == [3 * 16 + 15, 9 * 16, 9 * 16 + 1, 9 * 16 + 15]


# ------------------------------------------------------------ norm and rotation
def turn64(x, row, rot, interleaved, back=False):
    half = rot // 2
    c, s = row[..., :half], row[..., half:]
    s = -s if back else s
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope_case(seed, n, t, q, kv, d, rot, dtype, extra=0, zero_rows=False):
    g = gen(seed)
    width = (q + 2 * kv) * d
    buf = normal(g, n, max(t, 1), width + extra, dtype=DT[dtype], scale=1.5)[:, :t]
    qkv = buf[:, :, :width]
    if zero_rows and t:
        qkv[:, 0].zero_()
    wq, wk = normal(g, d, dtype=DT[dtype]), normal(g, d, dtype=DT[dtype])
    angle = torch.rand((300, rot // 2), generator=g, device="cuda") * 6.3
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    pos = torch.randint(0, 300, (t,), generator=g, device="cuda", dtype=torch.int32)
    return qkv, wq, wk, cos_sin, pos


def rope64(qkv, wq, wk, cos_sin, pos, q, kv, d, interleaved, eps):
    n, t = qkv.shape[:2]
    x = qkv.double().reshape(n, t, q + 2 * kv, d)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    w = torch.cat([wq.double().expand(q, d), wk.double().expand(kv, d)])
    z = x[:, :, :q + kv] * r[:, :, :q + kv] * w
    row = cos_sin.double()[pos.long()][None, :, None]
    y = turn64(z, row, cos_sin.shape[1], interleaved)
    size = turn64(z.abs(), row.abs(), cos_sin.shape[1], interleaved).abs() + \
        turn64(z.abs(), -row.abs(), cos_sin.shape[1], interleaved).abs() + z.abs()
    # sum of d squares (d u), root, three products, two products and a sum of the rotation
    return y[:, :, :q], y[:, :, q:], x[:, :, q + kv:], (d / 2 + 12) * U * size


ROPE = [  # n, tokens, q heads, kv heads, dim, rot, interleaved, dtype, extra columns
    (1, 1, 1, 1, 64, 64, False, "bf16", 0), (2, 5, 8, 1, 128, 128, False, "bf16", 0),
    (3, 7, 3, 1, 80, 80, False, "f32", 8), (1, 130, 5, 5, 96, 48, True, "bf16", 16),
    (2, 33, 6, 2, 256, 64, True, "f32", 0), (8, 17, 4, 2, 192, 192, False, "bf16", 0),
    (1, 65, 2, 1, 8 * 9, 32, False, "bf16", 0), (2, 9, 1, 1, 8 * 31, 16, True, "bf16", 8),
    (32, 3, 2, 1, 16, 16, False, "f32", 0), (1, 3, 1, 1, 24, 16, False, "bf16", 0),
    (2, 11, 3, 2, 80, 40, False, "bf16", 0), (1, 6, 9, 5, 8, 8, False, "f32", 0), (2, 5, 5, 3, 120, 24, True, "f32", 8)]


@pytest.mark.parametrize("n,t,q,kv,d,rot,inter,dtype,extra", ROPE)
def test_norm_rope(n, t, q, kv, d, rot, inter, dtype, extra):
    qkv, wq, wk, cs, pos = rope_case(3, n, t, q, kv, d, rot, dtype, extra, zero_rows=True)
    yq, yk, v, slack = rope64(qkv, wq, wk, cs, pos, q, kv, d, inter, 1e-5)
    ws = B.OpWorkspace()
    # queries of all ranks side by side in one row
    q_all = torch.zeros((t, n, q, d), dtype=DT[dtype], device="cuda")
    k_out = torch.empty((n, t, kv, d), dtype=DT[dtype], device="cuda")
    B.qk_norm_rope(qkv, wq, wk, cs, pos, [q_all[:, r] for r in range(n)], k_out, ws, eps=1e-5, interleaved=inter)
    assert B.get_status(ws) == B.Status.OK
    close(q_all.transpose(0, 1), yq, slack[:, :, :q], "q")
    close(k_out, yk, slack[:, :, q:], "k")

    page = 8
    pages = t // page + 2
    g = gen(5)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].to(torch.int32)
    if t > 2:
        slots[1] = -1  # a padding token
    k_cache = normal(g, n, pages, kv, page, d, dtype=DT[dtype])
    v_cache = normal(g, n, pages, kv, page, d, dtype=DT[dtype])
    k_old, v_old = k_cache.clone(), v_cache.clone()
    q_out = qkv.as_strided((n, t, q, d), (qkv.stride(0), qkv.stride(1), d, 1), qkv.storage_offset())
    B.qk_norm_rope_cached(qkv, wq, wk, cs, pos, slots, q_out, k_cache, v_cache, ws, eps=1e-5, interleaved=inter)
    assert B.get_status(ws) == B.Status.OK
    close(q_out, yq, slack[:, :, :q], "q in place")
    live = slots >= 0
    at, off = (slots[live] // page).long(), (slots[live] % page).long()
    close(k_cache[:, at, :, off].permute(1, 0, 2, 3), yk[:, live], slack[:, live][:, :, q:], "key cache")
    assert torch.equal(v_cache[:, at, :, off].permute(1, 0, 2, 3).double(), v[:, live])
    k_cache[:, at, :, off] = k_old[:, at, :, off]
    v_cache[:, at, :, off] = v_old[:, at, :, off]
    assert torch.equal(k_cache, k_old) and torch.equal(v_cache, v_old), "a row outside the slots was written"


@pytest.mark.parametrize("n,t,q,kv,d,rot,inter,dtype,extra", ROPE + [(2, 1500, 7, 3, 128, 128, False, "f32", 0),
                                                                     (1, 0, 2, 1, 64, 32, True, "bf16", 0)])
def test_norm_rope_backward(n, t, q, kv, d, rot, inter, dtype, extra):
    eps = 1e-5
    qkv, wq, wk, cs, pos = rope_case(4, n, t, q, kv, d, rot, dtype, extra)
    g = gen(6)
    dq, dk, dv = (normal(g, n, t, h, d, dtype=DT[dtype]) for h in (q, kv, kv))
    x = qkv.double().reshape(n, t, q + 2 * kv, d)[:, :, :q + kv]
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = x * r
    w = torch.cat([wq.double().expand(q, d), wk.double().expand(kv, d)])
    row = cs.double()[pos.long()][None, :, None]
    dy = torch.cat([dq, dk], 2).double()
    z = turn64(dy, row, rot, inter, back=True)
    a = z * w
    dot = (a * xh).mean(-1, keepdim=True)
    dx = r * (a - xh * dot)
    zs = dy.abs() + turn64(dy.abs(), row.abs(), rot, inter).abs() + turn64(dy.abs(), -row.abs(), rot, inter).abs()
    size = r * (zs * w.abs() + xh.abs() * (zs * w.abs() * xh.abs()).mean(-1, keepdim=True))
    ws = B.OpWorkspace(B.qk_norm_rope_workspace_bytes(n, d))
    dqkv = torch.empty((n, t, (q + 2 * kv) * d), dtype=DT[dtype], device="cuda")
    dwq = torch.full((n, d), float("nan"), device="cuda")
    dwk = torch.full((n, d), float("nan"), device="cuda")
    args = (qkv, wq, wk, cs, pos, dq, dk, dv, dqkv, dwq, dwk, ws)
    B.qk_norm_rope_backward(*args, eps=eps, interleaved=inter)
    assert B.get_status(ws) == B.Status.OK
    got = dqkv.view(n, t, q + 2 * kv, d)
    close(got[:, :, :q + kv], dx, (2 * d + 24) * U * size, "dx")
    assert torch.equal(got[:, :, q + kv:], dv)
    for dw, heads in ((dwq, slice(0, q)), (dwk, slice(q, q + kv))):
        terms = (z * xh)[:, :, heads]
        mag = (zs * xh.abs())[:, :, heads].sum((1, 2))
        close(dw, terms.sum((1, 2)), (t * (q + kv) + d + 24) * U * mag, "dw")
    first = [v.clone() for v in (dqkv, dwq, dwk)]
    B.qk_norm_rope_backward(*args, eps=eps, interleaved=inter)
    assert all(torch.equal(u, v) for u, v in zip(first, (dqkv, dwq, dwk))), "not the same bits twice"


def test_norm_rope_gradient_by_differences():
    """The directional derivative of sum(c y) from the forward kernel in f32,
    central differences of step h: h^2 times the third derivative (values of
    order one) plus the forward's rounding over h."""
    n, t, q, kv, d, rot = 1, 6, 3, 1, 64, 32
    qkv, wq, wk, cs, pos = rope_case(8, n, t, q, kv, d, rot, "f32")
    g = gen(9)
    cq, ck = normal(g, n, t, q, d), normal(g, n, t, kv, d)
    ws = B.OpWorkspace(B.qk_norm_rope_workspace_bytes(n, d))
    dqkv, dwq, dwk = torch.empty_like(qkv), torch.empty((n, d), device="cuda"), torch.empty((n, d), device="cuda")
    B.qk_norm_rope_backward(qkv, wq, wk, cs, pos, cq, ck, torch.zeros_like(ck), dqkv, dwq, dwk, ws)
    ex, eq, ek = normal(g, *qkv.shape), normal(g, d), normal(g, d)
    ex[..., (q + kv) * d:] = 0

    def loss(step):
        yq, yk = torch.empty_like(cq), torch.empty_like(ck)
        B.qk_norm_rope(qkv + step * ex, wq + step * eq, wk + step * ek, cs, pos, yq, yk, ws)
        return float((yq.double() * cq.double()).sum() + (yk.double() * ck.double()).sum())

    h = 2.0 ** -7
    want = (loss(h) - loss(-h)) / (2 * h)
    got = float((dqkv.double() * ex.double()).sum() + (dwq.double() * eq).sum() + (dwk.double() * ek).sum())
    terms = t * (q + kv) * d
    scale = terms ** 0.5 * 8  # a sum of independent products of a few normals each
    assert abs(got - want) <= scale * (8 * h * h + 64 * U / h)


def test_norm_rope_reports_bad_positions_and_slots():
    qkv, wq, wk, cs, pos = rope_case(1, 1, 4, 2, 1, 64, 64, "bf16")
    ws = B.OpWorkspace()
    q_out = torch.empty((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((2, 1, 3, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    for p, s in ((300, 0), (-1, 0), (0, 48)):
        pos2, slots = pos.clone(), i32(1, 2, 3, 4)
        pos2[2], slots[1] = p, s
        B.qk_norm_rope_cached(qkv, wq, wk, cs, pos2, slots, q_out, cache[0], cache[1], ws)
        assert B.get_status(ws) == B.Status.ERR_CAPACITY
        assert B.get_status(ws) == B.Status.OK


# ------------------------------------------------------------- decode attention
def attention_case(seed, n, lens, q, kv, d, page, dtype, poison=True, spare=3):
    g = gen(seed)
    batch = len(lens)
    need = [-(-v // page) for v in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, max(max(need), 1)), 2 ** 30, dtype=torch.int32, device="cuda")
    k = normal(g, n, pages, kv, page, d, dtype=DT[dtype])
    v = normal(g, n, pages, kv, page, d, dtype=DT[dtype])
    live = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        for j in range(m):
            live[order[at + j].long(), :min(page, lens[b] - j * page)] = True
        at += m
    if poison:  # everything that no length covers
        bad = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda")
        fill = bad[torch.randint(0, 3, (pages, page, d), generator=g, device="cuda")].to(DT[dtype])
        dead = ~live[None, :, None, :, None]
        k = torch.where(dead, fill[None, :, None], k)
        v = torch.where(dead, fill[None, :, None], v)
    x = normal(g, n, batch, q, d, dtype=DT[dtype])
    return x, k.contiguous(), v.contiguous(), table, i32(*lens)


def attention64(x, k, v, table, lens, scale, page):
    n, batch, q, d = x.shape
    kv = k.shape[2]
    out = torch.zeros((n, batch, q, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, batch, q), float("-inf"), dtype=torch.float64, device="cuda")
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, length in enumerate(lens.tolist()):
        if length == 0:
            continue
        t = torch.arange(length, device="cuda")
        rows = table[b].long()[t // page], t % page
        kk = k[:, rows[0], :, rows[1]].double().permute(1, 2, 0, 3)  # n, kv, t, d
        vv = v[:, rows[0], :, rows[1]].double().permute(1, 2, 0, 3)
        qq = x[:, b].double().view(n, kv, q // kv, d)
        s = torch.einsum("nkgd,nktd->nkgt", qq, kk) * scale
        size = torch.einsum("nkgd,nktd->nkgt", qq.abs(), kk.abs()) * abs(scale)
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - l[..., None])
        out[:, b] = torch.einsum("nkgt,nktd->nkgd", p, vv).reshape(n, q, d)
        lse[:, b] = l.reshape(n, q)
        # a score is off by (d + 4) u of its terms' magnitudes and by the 2 u of the exponent's scaling; the weighted
        # sum of up to `length` terms and its division add (length^(1/2) * 4 + 16) u: partial sums in any order
        ds = (d + 4) * U * size.amax(-1) + 4 * U * (s.abs().amax(-1) + l.abs())
        out_tol[:, b] = ((2 * ds + (4 * length ** 0.5 + 16) * U)[..., None]
                         * torch.einsum("nkgt,nktd->nkgd", p, vv.abs())).reshape(n, q, d)
        lse_tol[:, b] = (ds + (4 * length ** 0.5 + 16) * U).reshape(n, q)
    return out, lse, out_tol, lse_tol


def run_attention(x, k, v, table, lens, scale=None, want_lse=True):
    n, batch, q, d = x.shape
    ws = B.OpWorkspace(B.decode_attention_workspace_bytes(n, batch, q, k.shape[2], d))
    out = torch.full_like(x, float("nan"))
    lse = torch.full((n, batch, q), float("nan"), device="cuda") if want_lse else None
    B.decode_attention(x, k, v, table, lens, out, lse, ws, scale=scale)
    return out, lse, B.get_status(ws), ws


ODD = [0, 1, 2, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200]
ATTENTION = [  # n, lens, q heads, kv heads, dim, page, dtype
    (1, [1], 1, 1, 64, 16, "bf16"), (2, ODD, 8, 1, 128, 16, "bf16"), (1, ODD, 4, 4, 64, 8, "bf16"),
    (1, ODD, 16, 1, 128, 32, "bf16"), (2, ODD, 12, 2, 96, 1, "bf16"), (1, ODD, 40, 2, 80, 64, "bf16"),
    (1, ODD, 7, 1, 256, 16, "bf16"), (1, ODD, 24, 2, 192, 128, "bf16"), (3, ODD, 3, 3, 8, 4, "bf16"),
    (1, ODD, 33, 1, 136, 16, "bf16"), (2, ODD, 8, 1, 128, 16, "f32"), (1, ODD, 10, 2, 80, 32, "f32"),
    (1, ODD, 5, 1, 256, 2, "f32"), (1, ODD, 32, 2, 64, 16, "f32"), (2, ODD, 2, 1, 24, 1024, "f32"),
    (1, [100000, 3, 0, 4097], 8, 1, 128, 16, "bf16"), (1, [50001], 3, 1, 64, 128, "f32"),
    (1, [0, 0], 8, 2, 128, 16, "bf16"), (32, [40, 1300], 4, 2, 64, 16, "bf16"),
    (1, [i % 300 for i in range(1111)], 2, 1, 64, 16, "bf16"), (1, ODD, 16, 1, 256, 16, "bf16"),
    (1, ODD, 20, 2, 128, 16, "f32"), (1, ODD, 12, 1, 96, 16, "f32"), (1, ODD, 9, 1, 192, 8, "f32"),
    (1, [30000, 5], 16, 1, 192, 64, "bf16"), (2, [0, 70001], 12, 1, 88, 32, "f32")]


@pytest.mark.parametrize("n,lens,q,kv,d,page,dtype", ATTENTION)
def test_decode_attention(n, lens, q, kv, d, page, dtype):
    x, k, v, table, ln = attention_case(11, n, lens, q, kv, d, page, dtype)
    out, lse, status, ws = run_attention(x, k, v, table, ln)
    assert status == B.Status.OK
    want, wlse, tol, ltol = attention64(x, k, v, table, ln, d ** -0.5, page)
    close(out, want, tol, "out")
    close(lse, wlse, ltol, "lse")
    again = torch.empty_like(out)
    B.decode_attention(x, k, v, table, ln, again, None, ws)
    assert torch.equal(out, again), "not the same bits twice"


def test_decode_attention_weights_sum_to_one():
    """Values of 1: a result is the sum of the weights over itself. Each of the two sums adds up to 144 tiles a warp (512
    requests and ranks of 128 tiles over 456 blocks), the block's warps and the joins, every addition rounded: at most u
    each. A sum that truncates drifts by half of that in one direction for each of a tile's several products."""
    g = gen(16)
    n, batch, d, page, length = 8, 64, 64, 128, 8192
    blocks = length // page
    k = normal(g, n, batch * blocks, 1, page, d)
    v = torch.ones_like(k)
    table = torch.randperm(batch * blocks, generator=g, device="cuda").to(torch.int32).view(batch, blocks)
    lens = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    out, _, status, _ = run_attention(normal(g, n, batch, 8, d), k, v, table, lens)
    assert status == B.Status.OK
    assert float((out.double() - 1).abs().max()) <= (2 * 144 + 32) * U / 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_attention_large_scores(dtype):
    """Scores in the hundreds, rising along the cache: the running maximum moves all the way."""
    lens = [1500, 77]
    x, k, v, table, ln = attention_case(12, 1, lens, 8, 1, 64, 16, dtype)
    ramp = torch.linspace(0.1, 3, lens[0], device="cuda")
    t = torch.arange(lens[0], device="cuda")
    at, off = table[0].long()[t // 16], t % 16
    k[:, at, :, off] = (k[:, at, :, off].float() * ramp[:, None, None, None] * 4).to(k.dtype)
    out, lse, status, _ = run_attention(x, k, v, table, ln, scale=1.0)
    want, wlse, tol, ltol = attention64(x, k, v, table, ln, 1.0, 16)
    close(out, want, tol, "out")
    close(lse, wlse, ltol, "lse")


def test_decode_attention_strides_streams_graph():
    n, lens, q, kv, d, page = 2, [70, 129, 5], 8, 2, 128, 16
    x, k, v, table, ln = attention_case(13, n, lens, q, kv, d, page, "bf16")
    want, wlse, tol, ltol = attention64(x, k, v, table, ln, d ** -0.5, page)
    wide = torch.zeros((3, n, q + 4, d), dtype=torch.bfloat16, device="cuda")  # rows of both ranks, with a gap
    xs = [wide[:, r, :q] for r in range(n)]
    for r in range(n):
        xs[r].copy_(x[r])
    big = torch.zeros((3, n, q, d), dtype=torch.bfloat16, device="cuda")
    outs = [big[:, r] for r in range(n)]
    tables = torch.full((3, table.shape[1] + 5), 7, dtype=torch.int32, device="cuda")
    tables[:, :table.shape[1]] = table
    ws = B.OpWorkspace(B.decode_attention_workspace_bytes(n, 3, q, kv, d))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    args = (xs, [k[r] for r in range(n)], [v[r] for r in range(n)], tables[:, :table.shape[1]], ln, outs, None, ws)
    B.decode_attention(*args, stream=stream)
    stream.synchronize()
    close(big.transpose(0, 1), want, tol, "other stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.decode_attention(*args)
    for new in ([70, 129, 5], [1, 0, 33], [80, 100, 16]):
        ln.copy_(i32(*new))
        big.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, _, tol, _ = attention64(x, k.nan_to_num(), v.nan_to_num(), table, i32(*[min(a, b) for a, b in
                                                                                  zip(new, lens)]), d ** -0.5, page)
        ok = [b for b in range(3) if new[b] <= lens[b]]
        close(big.transpose(0, 1)[:, ok], want[:, ok], tol[:, ok], "replayed")


def test_decode_attention_past_32_bits():
    """Cache rows whose element offset, and byte offset, pass 2^31 and 2^32."""
    page, d, kv = 64, 128, 1
    pages = (2 ** 32 // (page * d)) + 9
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    k = torch.zeros((1, pages, kv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((1, pages, kv, page, d), dtype=torch.bfloat16, device="cuda")
    g = gen(14)
    used = [pages - 1, 3, pages // 2 + 1, pages - 5]
    for p in used:
        k[0, p] = normal(g, kv, page, d).bfloat16()
        v[0, p] = normal(g, kv, page, d).bfloat16()
    table = i32(*used).view(1, -1)
    x = normal(g, 1, 1, 8, d, dtype=torch.bfloat16)
    out, lse, status, _ = run_attention(x, k, v, table, i32(250))
    assert status == B.Status.OK
    want, wlse, tol, ltol = attention64(x, k, v, table, i32(250), d ** -0.5, page)
    close(out, want, tol, "out")
    close(lse, wlse, ltol, "lse")


def test_decode_attention_reports_bad_tables():
    x, k, v, table, ln = attention_case(15, 1, [40, 40], 8, 1, 128, 16, "bf16")
    good, _, status, _ = run_attention(x, k, v, table, ln)
    assert status == B.Status.OK
    for value in (-1, k.shape[1], 2 ** 30):
        t2 = table.clone()
        t2[0, 1] = value
        out, _, status, ws = run_attention(x, k, v, t2, ln)
        assert status == B.Status.ERR_CAPACITY
        assert torch.equal(out[:, 1], good[:, 1]) and bool(out.isfinite().all())
        # without the 16 tokens of the page that is not there
        out2, _, status, _ = run_attention(x, k, v, table[:, [0, 2, 1]].contiguous(), i32(24, 40))
        close(out[:, 0], out2[:, 0].double(), 2.0 ** -7 * out2[:, 0].abs().double() + 8 * U, "left out")
    for length in (-3, 49):
        out, _, status, _ = run_attention(x, k.nan_to_num(), v.nan_to_num(), table.clamp(max=k.shape[1] - 1), i32(length, 40))
        assert status == B.Status.ERR_CAPACITY and torch.equal(out[:, 1], good[:, 1])
        if length < 0:
            assert not bool(out[:, 0].any())


# ------------------------------------------------------- token log probabilities
def logits_case(seed, n, rows, widths, dtype, offset=0, banned=True, ties=False):
    g = gen(seed)
    parts = []
    for w in widths:
        buf = normal(g, rows * (w + 5) + offset + 1, dtype=DT[dtype], scale=3.0)
        if ties:
            buf = buf.float().round().to(DT[dtype])
        x = buf[offset:offset + rows * (w + 5)].view(rows, w + 5)[:, :w]
        if banned and w > 3:
            x[:, torch.randint(0, w, (w // 4,), generator=g, device="cuda")] = float("-inf")
        parts.append(x)
    total = sum(widths)
    tokens = torch.randint(0, total, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return parts, tokens


def run_logprobs(parts, tokens, top):
    rows = parts[0].shape[0]
    ws = B.OpWorkspace(B.token_logprobs_workspace_bytes(rows, top))
    o = {k: torch.full((rows,), float("nan"), device="cuda") for k in ("logprob", "entropy", "lse")}
    o["top_values"] = torch.full((rows, top), float("nan"), device="cuda")
    o["top_ids"] = torch.full((rows, top), -1, dtype=torch.int32, device="cuda")
    B.token_logprobs(parts, tokens, workspace=ws, **o)
    assert B.get_status(ws) == B.Status.OK
    return o, ws


def check_logprobs(parts, tokens, o, top):
    x = torch.cat([p.double() for p in parts], 1)
    rows, total = x.shape
    lse = torch.logsumexp(x, 1)
    y = x - lse[:, None]
    p = torch.exp(y)
    size = x.masked_fill(x.isinf(), 0).abs().amax(1) + lse.abs()
    # exponents to 4 u of their magnitude, a sum of at most `total` terms joined from partial sums, one log
    tol = (4 * size + 4 * total ** 0.5 + 16) * U
    close(o["lse"], lse, tol, "lse")
    asked = (tokens >= 0) & (tokens < total)
    lp = torch.where(asked, y.gather(1, tokens.long().clamp(0, total - 1)[:, None])[:, 0], torch.zeros_like(lse))
    close(o["logprob"], lp, tol, "logprob")
    entropy = torch.special.entr(p).sum(1)
    mean = (p * y.masked_fill(p == 0, 0).abs()).sum(1)
    close(o["entropy"], entropy, tol * (1 + mean) + 16 * U * mean, "entropy")
    if top:
        order = torch.sort(x, dim=1, descending=True, stable=True)
        assert torch.equal(o["top_ids"].long(), order.indices[:, :top])
        close(o["top_values"], order.values[:, :top] - lse[:, None], tol[:, None], "top")


LOGPROBS = [  # rows, widths, dtype, top, offset, ties
    (1, [1], "f32", 1, 0, False), (1, [7], "bf16", 7, 1, False), (3, [1000], "bf16", 5, 0, False),
    (5, [33, 1, 64, 500], "f32", 32, 3, False), (2, [16384] * 8, "bf16", 8, 0, False),
    (7, [16003] * 4, "bf16", 20, 1, False), (300, [501, 499], "bf16", 3, 7, True), (2000, [128, 131], "f32", 0, 1, False),
    (9, [20000, 3], "f32", 1, 2, True), (1, [5003] * 32, "bf16", 31, 0, True), (1, [262145], "f32", 16, 0, False),
    (600, [4099], "bf16", 20, 1, True), (1300, [2048, 2048], "f32", 8, 0, False)]


@pytest.mark.parametrize("rows,widths,dtype,top,offset,ties", LOGPROBS)
def test_token_logprobs(rows, widths, dtype, top, offset, ties):
    parts, tokens = logits_case(21, len(widths), rows, widths, dtype, offset, ties=ties)
    if rows > 2:
        tokens[0], tokens[1] = -1, sum(widths)
    # words with a probability, so that no log probability is -inf where a number is compared
    o, ws = run_logprobs(parts, tokens, top)
    check_logprobs(parts, tokens, o, top)
    o2, _ = run_logprobs(parts, tokens, top)
    for k in o:
        assert torch.equal(o[k], o2[k]), k


def test_token_logprobs_edge_rows():
    """All words alike; one word only; nothing allowed; a NaN; +inf; a peak that holds all the probability."""
    v, inf, nan = 3000, float("inf"), float("nan")
    x = torch.zeros((7, v), device="cuda")
    x[1] = -inf
    x[1, 1234] = 5.0
    x[2] = -inf
    x[3, 17] = nan
    x[4, 18] = inf
    x[5, 2999] = 200.0
    x[6] = -1e30
    x[6, 5] = 1e30
    for dtype in ("f32", "bf16"):
        y = x.to(DT[dtype])
        parts = [y[:, :1001].contiguous(), y[:, 1001:].contiguous()]
        tokens = i32(2999, 1234, 0, 5, 18, 2999, 6)
        o, _ = run_logprobs(parts, tokens, 4)
        assert o["top_ids"][0].tolist() == [0, 1, 2, 3]
        assert o["top_ids"][1].tolist() == [1234, 0, 1, 2] and o["logprob"][1] == 0 and o["entropy"][1] == 0
        assert o["top_values"][1].tolist() == [0, -inf, -inf, -inf]
        for r in (2, 3, 4):
            assert o["entropy"][r].isnan() and o["logprob"][r].isnan()
        assert o["lse"][2] == -inf and o["top_ids"][2].tolist() == [0, 1, 2, 3]
        assert o["lse"][3].isnan() and int(o["top_ids"][3, 0]) == 17
        assert int(o["top_ids"][4, 0]) == 18
        assert o["logprob"][5] == 0 and o["entropy"][5] == 0 and int(o["top_ids"][5, 0]) == 2999
        assert o["entropy"][6] == 0 and o["logprob"][6] == -inf or o["logprob"][6] <= -1e30
        close(o["entropy"][:1], torch.full((1,), float(torch.tensor(float(v)).double().log()), dtype=torch.float64,
                                           device="cuda"), torch.tensor(64 * U, device="cuda"), "uniform")


@pytest.mark.parametrize("rows,widths,dtype,offset", [
    (1, [1], "f32", 0), (3, [1000], "bf16", 0), (5, [33, 1, 64, 500], "f32", 3), (7, [4003] * 4, "bf16", 1),
    (2, [16384] * 8, "bf16", 0), (300, [501, 499], "bf16", 7), (1, [100001], "f32", 2)])
@pytest.mark.parametrize("with_entropy", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
def test_token_logprobs_backward(rows, widths, dtype, offset, with_entropy, in_place):
    parts, tokens = logits_case(22, len(widths), rows, widths, dtype, offset)
    if rows > 2:
        tokens[0], tokens[1] = -1, sum(widths)
    g = gen(23)
    gl, gh = normal(g, rows), normal(g, rows)
    x = torch.cat([p.double() for p in parts], 1)
    total = x.shape[1]
    lse, H = torch.logsumexp(x, 1).float(), torch.special.entr(torch.softmax(x, 1)).sum(1).float()
    y = x - lse.double()[:, None]
    p = torch.exp(y)
    asked = (tokens >= 0) & (tokens < total)
    gg = torch.where(asked, gl, torch.zeros_like(gl)).double()[:, None]
    gl = torch.where(asked, gl, torch.full_like(gl, float("nan")))  # must not be read
    h = gh.double()[:, None] if with_entropy else torch.zeros_like(gg)
    picked = (torch.arange(total, device="cuda")[None] == tokens.long()[:, None]).double()
    y0 = y.masked_fill(p == 0, 0)
    want = gg * (picked - p) - h * p * (y0 + H.double()[:, None])
    size = gg.abs() * (picked + p) + h.abs() * p * (y0.abs() + H.double()[:, None])
    # p is off by its exponent's rounding: 4 u of (|x| + |lse|); and a few products
    tol = size * U * (4 * (x.masked_fill(x.isinf(), 0).abs() + lse.double().abs()[:, None]) + 16)
    ws = B.OpWorkspace()
    out = parts if in_place else [torch.empty_like(q) for q in parts]
    B.token_logprobs_backward(parts, tokens, lse, H, gl, gh if with_entropy else None, out, ws)
    assert B.get_status(ws) == B.Status.OK
    close(torch.cat(out, 1), want, tol + 1e-40, "dlogits")


def test_token_logprobs_gradient_by_differences():
    """Central differences of the forward kernel in f32, step h: the third
    derivative is of order one, the forward's values are off by their rounding."""
    rows, widths = 4, [65, 100]
    parts, tokens = logits_case(24, 2, rows, widths, "f32", banned=False)
    parts = [q.contiguous() for q in parts]
    g = gen(25)
    gl, gh = normal(g, rows), normal(g, rows)
    o, ws = run_logprobs(parts, tokens, 0)
    d = [torch.empty_like(q) for q in parts]
    B.token_logprobs_backward(parts, tokens, o["lse"], o["entropy"], gl, gh, d, ws)
    e = [normal(g, rows, w) for w in widths]
    h = 2.0 ** -6

    def loss(step):
        q, _ = run_logprobs([x + step * y for x, y in zip(parts, e)], tokens, 0)
        return float((q["logprob"].double() * gl.double()).sum() + (q["entropy"].double() * gh.double()).sum())

    want = (loss(h) - loss(-h)) / (2 * h)
    got = sum(float((a.double() * b.double()).sum()) for a, b in zip(d, e))
    assert abs(got - want) <= rows * 16 * (16 * h * h + 256 * U / h)


def test_operators_share_a_workspace_and_empty_calls():
    """One workspace serves all operators in any order; empty calls change nothing."""
    x, k, v, table, ln = attention_case(31, 1, [3000, 5], 8, 1, 64, 16, "bf16")
    parts, tokens = logits_case(32, 2, 3, [30000, 30000], "f32")
    qkv, wq, wk, cs, pos = rope_case(33, 1, 700, 4, 1, 64, 64, "f32")
    ws = B.OpWorkspace(max(B.decode_attention_workspace_bytes(1, 2, 8, 1, 64), B.token_logprobs_workspace_bytes(3, 9),
                           B.qk_norm_rope_workspace_bytes(1, 64)))
    ref, _, _, _ = run_attention(x, k, v, table, ln)
    lref, _ = run_logprobs(parts, tokens, 9)
    g = gen(34)
    dq, dk = normal(g, 1, 700, 4, 64), normal(g, 1, 700, 1, 64)
    last = None
    for _ in range(3):
        out = torch.empty_like(x)
        B.decode_attention(x, k, v, table, ln, out, None, ws)
        o = {key: torch.empty_like(t) for key, t in lref.items()}
        B.token_logprobs(parts, tokens, workspace=ws, **o)
        grads = [torch.empty_like(qkv), torch.empty((1, 64), device="cuda"), torch.empty((1, 64), device="cuda")]
        B.qk_norm_rope_backward(qkv, wq, wk, cs, pos, dq, dk, dk, *grads, ws)
        assert torch.equal(out, ref) and all(torch.equal(o[key], lref[key]) for key in o)
        assert last is None or all(torch.equal(a, b) for a, b in zip(last, grads))
        last = grads
    empty = torch.empty((1, 0, 8, 64), dtype=torch.bfloat16, device="cuda")
    B.decode_attention(empty, k, v, table[:0], ln[:0], empty, None, ws)
    none = torch.empty((0,), device="cuda")
    B.token_logprobs([p[:0] for p in parts], tokens[:0], none, none, none, None, None, ws)
    assert B.get_status(ws) == B.Status.OK


def test_uninitialised_workspace_is_reported():
    x, k, v, table, ln = attention_case(35, 1, [40], 8, 1, 64, 16, "bf16")
    ws = B.OpWorkspace(B.decode_attention_workspace_bytes(1, 1, 8, 1, 64))
    ws.buf.zero_()
    out = torch.full_like(x, 7.0)
    B.decode_attention(x, k, v, table, ln, out, None, ws)
    assert B.get_status(ws) == B.Status.ERR_WORKSPACE and bool((out == 7.0).all())


@pytest.mark.parametrize("way", ["one stream", "two streams", "graph", "torch between"])
def test_operators_follow_one_another(way):
    """A kernel may come up before the one ahead of it has ended, and has to wait for its results: steps whose
    operators each read what the last one wrote, and write over what it read, give the bits of the same steps with
    a synchronisation after every operator."""
    n, rows, q, kv, d, page, steps = 4, 40, 8, 2, 64, 4, 18
    g = gen(91)
    qkv = normal(g, steps, n, rows, (q + 2 * kv) * d, dtype=torch.bfloat16)
    weights = [normal(g, d, dtype=torch.bfloat16) for _ in range(2)]
    angles = torch.rand((64, d // 2), generator=g, device="cuda") * 6
    cos_sin = torch.cat([angles.cos(), angles.sin()], 1).contiguous()
    tokens = torch.randint(0, n * q * d, (rows,), generator=g, device="cuda", dtype=torch.int32)
    blocks = -(-steps // page)
    pages = rows * blocks + 3
    ones = ints(rows, 1)
    gradient = torch.full((rows,), 0.5, device="cuda")

    def f32(*shape):
        return torch.zeros(shape, device="cuda")

    def bf16(*shape):
        return torch.zeros(shape, device="cuda", dtype=torch.bfloat16)

    def prepared():
        return dict(lens=ints(2 * rows, 0).view(2, rows), count=i32(pages, 0).view(2, 1),
                    free=torch.arange(pages, device="cuda", dtype=torch.int32),
                    table=torch.zeros((rows, blocks), device="cuda", dtype=torch.int32), starts=ints(rows + 1),
                    positions=ints(rows), slots=ints(rows), queries=bf16(n, rows, q, d), out=bf16(n, rows, q, d),
                    k=bf16(n, pages, kv, page, d), v=bf16(n, pages, kv, page, d), dk=bf16(n, rows, kv, d),
                    dqkv=bf16(n, rows, (q + 2 * kv) * d), logprob=f32(steps, rows), entropy=f32(steps, rows),
                    lse=f32(steps, rows), values=f32(steps, rows, 5),
                    ids=torch.zeros((steps, rows, 5), device="cuda", dtype=torch.int32), dw=f32(steps, 2, n, d),
                    ws=B.OpWorkspace(max(B.decode_attention_workspace_bytes(n, rows, q, kv, d),
                                         B.token_logprobs_workspace_bytes(rows, 5),
                                         B.qk_norm_rope_workspace_bytes(n, d))))

    def run(s, call):
        for i in range(steps):
            logits, now, next = s["out"].view(n, rows, q * d), i % 2, 1 - i % 2
            lens = s["lens"][next]
            call(B.page_tables, s["lens"][now], ones, s["free"], s["count"][now], s["table"], page, pages, lens, s["starts"],
                 s["positions"], s["slots"], s["count"][next], s["ws"])
            call(B.qk_norm_rope_cached, qkv[i], *weights, cos_sin, s["positions"], s["slots"], s["queries"], s["k"], s["v"],
                 s["ws"])
            call(B.decode_attention, s["queries"], s["k"], s["v"], s["table"], lens, s["out"], None, s["ws"])
            call(B.token_logprobs, logits, tokens, s["logprob"][i], s["entropy"][i], s["lse"][i], s["values"][i],
                 s["ids"][i], s["ws"])
            call(B.token_logprobs_backward, logits, tokens, s["lse"][i], s["entropy"][i], gradient, None, logits, s["ws"])
            call(B.qk_norm_rope_backward, qkv[i], *weights, cos_sin, s["positions"], s["out"], s["dk"], s["dk"], s["dqkv"],
                 s["dw"][i, 0], s["dw"][i, 1], s["ws"])

    def apart(f, *args):
        f(*args)
        torch.cuda.synchronize()

    want = prepared()
    run(want, apart)
    got = prepared()
    torch.cuda.synchronize()
    if way == "one stream":
        run(got, lambda f, *args: f(*args))
    elif way == "two streams":
        streams = [torch.cuda.Stream() for _ in range(2)]

        def alternate(f, *args):
            f(*args, stream=streams[0])
            streams[1].wait_stream(streams[0])
            streams.reverse()

        run(got, alternate)
    elif way == "graph":
        first = {k: v.clone() for k, v in got.items() if k != "ws"}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(got, lambda f, *args: f(*args))
        for _ in range(3):
            for k, v in first.items():
                got[k].copy_(v)
            graph.replay()
    else:
        def between(f, *args):
            f(*args)
            got["dk"].add_(0)

        run(got, between)
    torch.cuda.synchronize()
    assert B.get_status(want["ws"]) == B.Status.OK and B.get_status(got["ws"]) == B.Status.OK
    assert want["lens"][steps % 2].tolist() == [steps] * rows
    for k in want:
        if k != "ws":
            assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [1, 2, 5, 6, 7, 8, 9, 31, 32])
def test_token_logprobs_alternatives(top, dtype):
    """One part a row to more than 128, words in rising and falling order, many alike, rows of -inf: every way in which
    alternatives are found and joined gives the first of a stable sort."""
    for seed, widths in enumerate(([40], [700, 900], [1024] * 5, [1700] * 4, [3000] * 5, [9000, 1], [16384] * 8,
                                   [32768] * 5)):
        total = sum(widths)
        parts, tokens = logits_case(60 + seed, len(widths), 6, widths, dtype, seed % 3, ties=seed % 2 == 1)
        ramp = torch.arange(total, device="cuda").float() * 0.125
        at = 0
        for p in parts:
            p[0] = ramp[at:at + p.shape[1]]
            p[1] = -ramp[at:at + p.shape[1]]
            p[2] = 1.5
            p[3] = float("-inf")
            at += p.shape[1]
        o, _ = run_logprobs(parts, tokens, top)
        x = torch.cat([p.double() for p in parts], 1)
        order = torch.sort(x, dim=1, descending=True, stable=True)
        assert torch.equal(o["top_ids"].long(), order.indices[:, :top]), widths


@pytest.mark.parametrize("rows,widths,dtype,offset", [
    (700, [501, 499], "bf16", 7), (1300, [2051], "f32", 1), (1217, [3071], "f32", 0), (409, [1, 700, 2049], "bf16", 0),
    (2500, [8], "bf16", 0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_token_logprobs_backward_of_many_narrow_rows(rows, widths, dtype, offset, in_place):
    test_token_logprobs_backward(rows, widths, dtype, offset, True, in_place)


@pytest.mark.parametrize("q,d,dtype", [(8, 128, "bf16"), (16, 64, "bf16"), (9, 192, "bf16"), (5, 80, "f32")])
def test_decode_attention_cuts(q, d, dtype):
    """Lengths for which the blocks' ranges begin and end at every kind of place: in an item, at its first or last
    tile, and between items."""
    rng = torch.Generator().manual_seed(17)
    for seed, (batch, longest) in enumerate([(1, 65), (2, 30000), (3, 64 * 500), (40, 700), (150, 130), (300, 64),
                                             (450, 128), (700, 200), (911, 65), (913, 100)]):
        lens = torch.randint(0, longest + 1, (batch,), generator=rng).tolist()
        x, k, v, table, ln = attention_case(70 + seed, 1, lens, q, 1, d, 16, dtype)
        out, lse, status, _ = run_attention(x, k, v, table, ln)
        assert status == B.Status.OK
        want, wlse, tol, ltol = attention64(x, k, v, table, ln, d ** -0.5, 16)
        close(out, want, tol, "out")
        close(lse, wlse, ltol, "lse")


@pytest.mark.parametrize("rows,widths,dtype,top", [
    (5000, [1100, 30], "bf16", 5), (9731, [700], "f32", 20), (6000, [1030, 1027], "bf16", 0), (5001, [16400], "bf16", 1),
    (4864, [333], "bf16", 2), (4865, [20, 1300], "f32", 3), (11000, [8200], "bf16", 0)])
def test_token_logprobs_of_many_rows(rows, widths, dtype, top):
    test_token_logprobs(rows, widths, dtype, top, 1, False)


@pytest.mark.parametrize("n,t,q,kv,d,rot,inter,dtype,extra", [
    (1, 3, 32, 4, 192, 96, False, "bf16", 0), (4, 2, 32, 8, 64, 32, True, "bf16", 8), (1, 1, 7, 3, 128, 128, False, "f32", 0),
    (8, 117, 32, 16, 80, 80, True, "f32", 0), (1, 703, 16, 2, 192, 192, False, "bf16", 0), (2, 64, 12, 9, 96, 48, False, "f32", 0),
    (1, 40, 1024, 2, 8, 8, False, "bf16", 0)])
def test_norm_rope_backward_of_few_tokens(n, t, q, kv, d, rot, inter, dtype, extra):
    """A token's heads shared by several groups of threads."""
    test_norm_rope_backward(n, t, q, kv, d, rot, inter, dtype, extra)


def test_operators_follow_copies():
    """A kernel that may come up early waits for a copy ahead of it all the same, and a copy behind it for its results."""
    rows, vocab, n = 64, 40000, 12
    g = torch.Generator().manual_seed(5)
    given = [torch.randn((1, rows, vocab), generator=g).pin_memory() for _ in range(n)]
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32).cuda()
    x = torch.zeros((1, rows, vocab), device="cuda")
    d = torch.zeros_like(x)
    o = {k: torch.zeros((rows,), device="cuda") for k in ("logprob", "entropy", "lse")}
    ws = B.OpWorkspace(B.token_logprobs_workspace_bytes(rows, 0))
    read = [torch.zeros((2, rows)).pin_memory() for _ in range(n)]
    grads = [torch.zeros((1, rows, vocab)).pin_memory() for _ in range(n)]
    ones = torch.ones((rows,), device="cuda")
    torch.cuda.synchronize()
    for i in range(n):
        B.token_logprobs(x, tokens, workspace=ws, top_values=None, top_ids=None, **o)  # of the last logits; overwritten
        x.copy_(given[i], non_blocking=True)
        B.token_logprobs(x, tokens, workspace=ws, top_values=None, top_ids=None, **o)
        B.token_logprobs_backward(x, tokens, o["lse"], o["entropy"], ones, ones, d, ws)
        grads[i].copy_(d, non_blocking=True)
        read[i][0].copy_(o["logprob"], non_blocking=True)
        read[i][1].copy_(o["lse"], non_blocking=True)
    torch.cuda.synchronize()
    for i in range(n):
        want = {k: torch.zeros((rows,), device="cuda") for k in o}
        x.copy_(given[i])
        B.token_logprobs(x, tokens, workspace=ws, top_values=None, top_ids=None, **want)
        torch.cuda.synchronize()
        B.token_logprobs_backward(x, tokens, want["lse"], want["entropy"], ones, ones, d, ws)
        assert torch.equal(read[i][0], want["logprob"].cpu()) and torch.equal(read[i][1], want["lse"].cpu())
        assert torch.equal(grads[i], d.cpu())
