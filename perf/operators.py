"""Cases of the decode and scoring operators over virtual ranks: page tables, query/key norm with rotary positions,
attention of one new token over a paged cache, and log probabilities over vocabulary shards.

Every tensor that belongs to a rank has the rank as its first dimension (N ranks in one GPU): heads and vocabulary are
split over the ranks, request lengths, tables and positions are shared by all of them.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # a decode step of eight requests: one token each, the smallest call of a serving loop
        dict(name="pages_decode_8", op="pages", requests=8, tokens=8, page=16, max_len=4096),
        # a large mixed step: thousands of decoding requests and chunked prefills among them
        dict(name="pages_mixed_4096", op="pages", requests=4096, tokens=262144, page=16, max_len=8192),
        # one decode step of a small batch on eight ranks (64 query heads, 8 key heads in all)
        dict(name="rope_decode_5", op="rope_cached", ranks=8, tokens=5, q_heads=8, kv_heads=1, dim=128, rot=128,
             interleaved=False, dtype="bf16", page=16, max_pos=8192),
        # a prefill of 8192 tokens on eight ranks into the cache: limited by memory
        dict(name="rope_prefill_8192", op="rope_cached", ranks=8, tokens=8192, q_heads=8, kv_heads=1, dim=128, rot=128,
             interleaved=False, dtype="bf16", page=64, max_pos=32768),
        # the same operator in a training step: gradients, interleaved pairs, half of the head rotated, odd length
        dict(name="rope_backward_4097", op="rope_backward", ranks=4, tokens=4097, q_heads=12, kv_heads=4, dim=96, rot=48,
             interleaved=True, dtype="bf16", max_pos=8192),
        # one chat request of a few hundred tokens: latency
        dict(name="attention_one_777", op="attention", ranks=1, batch=1, q_heads=8, kv_heads=1, dim=128, max_len=777,
             ragged=False, page=16, dtype="bf16"),
        # a ragged batch on eight ranks, lengths from 0 to 16384
        dict(name="attention_ragged_64", op="attention", ranks=8, batch=64, q_heads=8, kv_heads=1, dim=128, max_len=16384,
             ragged=True, page=16, dtype="bf16"),
        # one long document on one rank: the cache's length is all there is to split
        dict(name="attention_long_262145", op="attention", ranks=1, batch=1, q_heads=16, kv_heads=2, dim=128,
             max_len=262145, ragged=False, page=64, dtype="bf16"),
        # 32 bits, a head size and a group that are no powers of two
        dict(name="attention_f32_33", op="attention", ranks=2, batch=33, q_heads=10, kv_heads=2, dim=80, max_len=3001,
             ragged=True, page=32, dtype="f32"),
        # scores of a decode step over eight vocabulary shards
        dict(name="logprobs_decode_3", op="logprobs", ranks=8, rows=3, vocab=16384, top=8, dtype="bf16"),
        # scores of a whole batch of sequences, shards of an odd size (rows start on odd addresses)
        dict(name="logprobs_rows_2048", op="logprobs", ranks=8, rows=2048, vocab=16003, top=5, dtype="bf16"),
        # the gradient of a policy or language model loss with an entropy term
        dict(name="logprobs_backward_2048", op="logprobs_backward", ranks=8, rows=2048, vocab=16384, dtype="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        v = min(max(v, lo), hi)
        return v + 1 if v == 3072 else v

    op = rng.choice(["pages", "rope_cached", "rope", "rope_backward", "attention", "attention", "logprobs",
                     "logprobs_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ranks = rng.choice([1, 2, 4, 8])
    if op == "pages":
        requests = spread(1, 4096)
        return dict(op=op, requests=requests, tokens=requests + spread(1, 250000), page=rng.choice([8, 16, 32, 64, 128]),
                    max_len=spread(16, 8192))
    if op.startswith("rope"):
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        kv = rng.choice([1, 2, 4])
        q = kv * rng.choice([1, 2, 3, 4, 8])
        most = 8 * 8192 * 10 * 128 // (ranks * (q + 2 * kv) * dim) // (2 if dtype == "f32" else 1)
        if op != "rope_cached":
            most = most // 2
        case = dict(op=op, ranks=ranks, tokens=spread(1, max(2, most)), q_heads=q, kv_heads=kv, dim=dim,
                    rot=rng.choice([r for r in (dim, dim // 2, 32) if r % 16 == 0]),
                    interleaved=rng.random() < 0.5, dtype=dtype, max_pos=spread(64, 32768))
        if op == "rope_cached":
            case["page"] = rng.choice([8, 16, 32, 64, 128])
        return case
    if op == "attention":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        kv = rng.choice([1, 1, 2, 4])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        batch = spread(1, 256)
        size = 2 if dtype == "bf16" else 4
        most = 2 ** 30 // (ranks * kv * dim * size * 2 * batch)
        return dict(op=op, ranks=ranks, batch=batch, q_heads=kv * group, kv_heads=kv, dim=dim,
                    max_len=spread(1, max(2, min(most, 131072))), ragged=rng.random() < 0.7,
                    page=rng.choice([8, 16, 32, 64, 128]), dtype=dtype)
    vocab = spread(1000, 150000 // ranks)
    most = 2 ** 27 // (ranks * vocab)
    case = dict(op=op, ranks=ranks, rows=spread(1, max(2, most)), vocab=vocab, dtype=dtype)
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 8, 20])
    return case


def _lengths(case):
    """Lengths of the cached requests: all alike, or spread evenly from 0 to the longest."""
    batch, longest = case["batch"], case["max_len"]
    if not case["ragged"] or batch == 1:
        return [longest] * batch
    return [longest * i // (batch - 1) for i in range(batch)]


def _new_tokens(case):
    """New tokens of each request: one for most, the rest of the step's tokens spread over every eighth as prefill."""
    requests, tokens = case["requests"], case["tokens"]
    new = [1] * requests
    prefills = list(range(0, requests, 8))
    left = tokens - requests
    for i, r in enumerate(prefills):
        new[r] += left * (i + 1) // len(prefills) - left * i // len(prefills)
    return new


def work(case):
    op = case["op"]
    if op == "pages":
        r, t = case["requests"], case["tokens"]
        # lengths and new tokens in, lengths and starts out, one table entry read a request; positions and slots; new pages
        return {"bytes": 20 * r + 8 * t + 8 * (t // case["page"]), "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    if op.startswith("rope"):
        heads = case["q_heads"] + case["kv_heads"]
        rows = case["ranks"] * case["tokens"]
        table = min(case["tokens"], case["max_pos"]) * case["rot"] * 4
        if op == "rope_cached":
            moved = 2 * rows * (heads + case["kv_heads"])
        elif op == "rope":
            moved = 2 * rows * heads
        else:
            moved = rows * (heads + 2 * (heads + case["kv_heads"]))
        return {"bytes": moved * case["dim"] * size + table + 8 * case["tokens"],
                "flops": rows * heads * case["dim"] * (8 if op != "rope_backward" else 20)}
    if op == "attention":
        tokens = sum(_lengths(case)) * case["ranks"]
        io = 2 * case["ranks"] * case["batch"] * case["q_heads"] * case["dim"] * size
        return {"bytes": 2 * tokens * case["kv_heads"] * case["dim"] * size + io + 4 * (tokens // case["page"]),
                "flops": 4 * tokens * case["q_heads"] * case["dim"]}
    values = case["ranks"] * case["rows"] * case["vocab"]
    if op == "logprobs":
        return {"bytes": values * size + case["rows"] * (16 + 8 * case["top"]), "flops": 5 * values}
    return {"bytes": 2 * values * size + 20 * case["rows"], "flops": 7 * values}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=dtype) * scale).to(dtype)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)

    op = case["op"]
    s = dict(case=case)
    if op == "pages":
        requests, page = case["requests"], case["page"]
        new = torch.tensor(_new_tokens(case), dtype=torch.int32, device="cuda")[shuffled(requests).long()]
        lens = ints(0, case["max_len"] + 1, requests)
        max_blocks = (case["max_len"] + max(_new_tokens(case)) + page - 1) // page
        have = (lens + page - 1) // page
        pages = requests * ((case["max_len"] + page - 1) // page) + case["tokens"] // page + 2 * requests
        order = shuffled(pages)
        columns = torch.arange(max_blocks, device="cuda", dtype=torch.int32)
        first = torch.cumsum(have, 0, dtype=torch.int32) - have
        at = (first[:, None] + columns[None]).clamp(max=pages - 1).long()
        s["table"] = torch.where(columns[None] < have[:, None], order[at], torch.full_like(columns, -1)[None])
        used = int(have.sum())
        s["free"] = order[used:].contiguous()
        s["free_count"] = torch.tensor([pages - used], dtype=torch.int32, device="cuda")
        s["lens"], s["new"], s["num_pages"] = lens, new, pages
        s["capacity"] = (case["tokens"] + 63) // 64 * 64
        return s
    dtype = DTYPES[case["dtype"]]
    n = case["ranks"]
    if op.startswith("rope"):
        t, q, kv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        s["qkv"] = normal(n, t, (q + 2 * kv) * d, dtype=dtype, scale=1.5)
        s["wq"] = (1 + 0.2 * normal(d)).to(dtype)
        s["wk"] = (1 + 0.2 * normal(d)).to(dtype)
        half = case["rot"] // 2
        angle = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)[None]
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = ints(0, case["max_pos"], t)
        if op == "rope_cached":
            page = case["page"]
            pages = (t + page - 1) // page + 3
            s["slots"] = shuffled(pages * page)[:t].contiguous()
            s["k_cache"] = normal(n, pages, kv, page, d, dtype=dtype)
            s["v_cache"] = normal(n, pages, kv, page, d, dtype=dtype)
        if op == "rope_backward":
            s["dq"] = normal(n, t, q, d, dtype=dtype)
            s["dk"] = normal(n, t, kv, d, dtype=dtype)
            s["dv"] = normal(n, t, kv, d, dtype=dtype)
        return s
    if op == "attention":
        batch, d, kv, page = case["batch"], case["dim"], case["kv_heads"], case["page"]
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[shuffled(batch).long()]
        max_blocks = (case["max_len"] + page - 1) // page
        have = (lens + page - 1) // page
        pages = sum((v + page - 1) // page for v in _lengths(case)) + 5
        order = shuffled(pages)
        first = torch.cumsum(have, 0) - have
        columns = torch.arange(max_blocks, device="cuda")
        at = (first[:, None] + columns[None]).clamp(max=pages - 1)
        s["table"] = torch.where(columns[None] < have[:, None], order[at], torch.full((1, 1), -1, dtype=torch.int32, device="cuda"))
        s["lens"] = lens
        s["q"] = normal(n, batch, case["q_heads"], d, dtype=dtype)
        s["k_cache"] = normal(n, pages, kv, page, d, dtype=dtype)
        s["v_cache"] = normal(n, pages, kv, page, d, dtype=dtype)
        return s
    rows, vocab = case["rows"], case["vocab"]
    logits = normal(n, rows, vocab, dtype=dtype, scale=3.0)
    # a few words that the sampler's rules forbid
    banned = ints(0, vocab, n, max(1, vocab // 1000)).long()
    logits.scatter_(2, banned[:, None].expand(n, rows, -1), float("-inf"))
    s["logits"] = logits
    tokens = ints(0, n * vocab, rows)
    forbidden = logits[(tokens // vocab).long(), torch.arange(rows, device="cuda"), (tokens % vocab).long()].isinf()
    s["tokens"] = torch.where(forbidden, torch.full_like(tokens, -1), tokens)
    if op == "logprobs_backward":
        y = logits.permute(1, 0, 2).reshape(rows, n * vocab).double()
        lse = torch.logsumexp(y, 1)
        y = (y - lse[:, None]).exp_()
        s["lse"], s["entropy"] = lse.float(), torch.special.entr(y).sum(1).float()
        s["grad_logprob"] = normal(rows)
        s["grad_entropy"] = 0.1 * normal(rows)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from collective_communication_gb300 import binding as B

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    op = case["op"]
    need = 0
    if op == "pages":
        r = case["requests"]
        s["lens_out"], s["starts"] = empty(r, dtype=torch.int32), empty(r + 1, dtype=torch.int32)
        s["positions"] = empty(s["capacity"], dtype=torch.int32)
        s["slots"] = empty(s["capacity"], dtype=torch.int32)
        s["free_out"] = empty(1, dtype=torch.int32)
    elif op in ("rope", "rope_cached"):
        n, t, d = case["ranks"], case["tokens"], case["dim"]
        s["q_out"] = empty(n, t, case["q_heads"], d, dtype=s["qkv"].dtype)
        if op == "rope":
            s["k_out"] = empty(n, t, case["kv_heads"], d, dtype=s["qkv"].dtype)
    elif op == "rope_backward":
        n, d = case["ranks"], case["dim"]
        s["dqkv"] = torch.empty_like(s["qkv"])
        s["dwq"], s["dwk"] = empty(n, d), empty(n, d)
        need = B.qk_norm_rope_workspace_bytes(n, d)
    elif op == "attention":
        n, batch, q = case["ranks"], case["batch"], case["q_heads"]
        s["out"], s["lse"] = torch.empty_like(s["q"]), empty(n, batch, q)
        need = B.decode_attention_workspace_bytes(n, batch, q, case["kv_heads"], case["dim"])
    elif op == "logprobs":
        rows, top = case["rows"], case["top"]
        s["logprob"], s["entropy"], s["lse"] = empty(rows), empty(rows), empty(rows)
        s["top_values"], s["top_ids"] = empty(rows, top), empty(rows, top, dtype=torch.int32)
        need = B.token_logprobs_workspace_bytes(rows, top)
    else:
        s["dlogits"] = torch.empty_like(s["logits"])
    s["workspace"] = B.OpWorkspace(need)
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from collective_communication_gb300 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "pages":
        B.page_tables(s["lens"], s["new"], s["free"], s["free_count"], s["table"], case["page"], s["num_pages"],
                      s["lens_out"], s["starts"], s["positions"], s["slots"], s["free_out"], s["workspace"])
        return dict(table=s["table"], lens=s["lens_out"], starts=s["starts"], positions=s["positions"], slots=s["slots"],
                    free=s["free_out"])
    if op == "rope_cached":
        B.qk_norm_rope_cached(s["qkv"], s["wq"], s["wk"], s["cos_sin"], s["positions"], s["slots"], s["q_out"],
                              s["k_cache"], s["v_cache"], s["workspace"], eps=EPS, interleaved=case["interleaved"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if op == "rope":
        B.qk_norm_rope(s["qkv"], s["wq"], s["wk"], s["cos_sin"], s["positions"], s["q_out"], s["k_out"], s["workspace"],
                       eps=EPS, interleaved=case["interleaved"])
        return dict(q=s["q_out"], k=s["k_out"])
    if op == "rope_backward":
        B.qk_norm_rope_backward(s["qkv"], s["wq"], s["wk"], s["cos_sin"], s["positions"], s["dq"], s["dk"], s["dv"],
                                s["dqkv"], s["dwq"], s["dwk"], s["workspace"], eps=EPS, interleaved=case["interleaved"])
        return dict(dqkv=s["dqkv"], dwq=s["dwq"], dwk=s["dwk"])
    if op == "attention":
        B.decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"], s["lse"], s["workspace"],
                           scale=case["dim"] ** -0.5)
        return dict(out=s["out"], lse=s["lse"])
    if op == "logprobs":
        B.token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["lse"], s["top_values"], s["top_ids"],
                         s["workspace"])
        out = dict(logprob=s["logprob"], entropy=s["entropy"], lse=s["lse"])
        if case["top"]:
            out.update(top_values=s["top_values"], top_ids=s["top_ids"])
        return out
    B.token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["grad_logprob"], s["grad_entropy"],
                              s["dlogits"], s["workspace"])
    return dict(dlogits=s["dlogits"])


def _plain_pages(s):
    page = s["case"]["page"]
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"]
    have = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - have
    off = torch.cumsum(need, 0) - need
    columns = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (columns >= have[:, None]) & (columns < (have + need)[:, None])
    at = s["free_count"].long()[0] - 1 - (off[:, None] + columns - have[:, None])
    table = torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table)
    starts = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    token = torch.arange(s["capacity"], device="cuda")
    request = torch.searchsorted(starts[1:].contiguous(), token, right=True).clamp(max=lens.numel() - 1)
    position = lens[request] + token - starts[request]
    live = token < starts[-1]
    position = torch.where(live, position, torch.zeros_like(position))
    slot = table[request, (position // page).clamp(max=table.shape[1] - 1)].long() * page + position % page
    slot = torch.where(live, slot, torch.full_like(slot, -1))
    return dict(table=table, lens=(lens + new).int(), starts=starts.int(), positions=position.int(), slots=slot.int(),
                free=(s["free_count"] - need.sum()).int())


def _rotate(x, cos, sin, rot, interleaved):
    """Rotates the first rot elements of the last dimension by the angles of cos and sin (rot / 2 each)."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _normed(s):
    """Query and key heads in 32 bits, their weights by head, and the reciprocal of their root mean squares."""
    case = s["case"]
    q, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    n, t = s["qkv"].shape[:2]
    x = s["qkv"].view(n, t, q + 2 * kv, d)[:, :, :q + kv].float()
    w = torch.cat([s["wq"].float().expand(q, d), s["wk"].float().expand(kv, d)])
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    turn = s["cos_sin"][s["positions"].long()][None, :, None]
    return x, w, r, turn[..., :case["rot"] // 2], turn[..., case["rot"] // 2:]


def _plain_rope(s):
    case = s["case"]
    x, w, r, cos, sin = _normed(s)
    y = _rotate(x * r * w, cos, sin, case["rot"], case["interleaved"]).to(s["qkv"].dtype)
    return dict(q=y[:, :, :case["q_heads"]].contiguous(), k=y[:, :, case["q_heads"]:].contiguous())


def _plain_rope_cached(s):
    case = s["case"]
    y = _plain_rope(s)
    q, kv, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    n, t = s["qkv"].shape[:2]
    v = s["qkv"].view(n, t, q + 2 * kv, d)[:, :, q + kv:]
    at, off = (s["slots"] // page).long(), (s["slots"] % page).long()
    s["k_cache"][:, at, :, off] = y["k"].permute(1, 0, 2, 3)
    s["v_cache"][:, at, :, off] = v.permute(1, 0, 2, 3)
    return dict(q=y["q"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_rope_backward(s):
    case = s["case"]
    q, kv = case["q_heads"], case["kv_heads"]
    x, w, r, cos, sin = _normed(s)
    n, t = x.shape[:2]
    dy = torch.cat([s["dq"].float(), s["dk"].float()], 2)
    dz = _rotate(dy, cos, -sin, case["rot"], case["interleaved"])
    xh = x * r
    dw = dz * xh
    a = dz * w
    dx = r * (a - xh * (a * xh).mean(-1, keepdim=True))
    dqkv = torch.cat([dx, s["dv"].float()], 2).reshape(n, t, -1).to(s["qkv"].dtype)
    return dict(dqkv=dqkv, dwq=dw[:, :, :q].sum((1, 2)), dwk=dw[:, :, q:].sum((1, 2)))


def _plain_attention(s):
    case = s["case"]
    n, batch, q, d = s["q"].shape
    kv, page = case["kv_heads"], case["page"]
    blocks = s["table"].shape[1]
    at = s["table"].clamp(min=0).long()
    query = s["q"].float().view(n, batch, kv, q // kv, d) * d ** -0.5
    # [n, batch, blocks, kv, page, d] -> [n, batch, kv, blocks * page, d]
    k = s["k_cache"][:, at].permute(0, 1, 3, 2, 4, 5).reshape(n, batch, kv, blocks * page, d).float()
    scores = torch.matmul(query, k.transpose(-1, -2))
    del k
    live = torch.arange(blocks * page, device="cuda")[None] < s["lens"][:, None]
    scores = torch.where(live[None, :, None, None], scores, torch.full((), float("-inf"), device="cuda"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    v = s["v_cache"][:, at].permute(0, 1, 3, 2, 4, 5).reshape(n, batch, kv, blocks * page, d).float()
    out = torch.matmul(p, v).reshape(n, batch, q, d).to(s["q"].dtype)
    return dict(out=out, lse=(top + torch.log(total)).reshape(n, batch, q))


def _plain_logprobs(s):
    n, rows, vocab = s["logits"].shape
    x = s["logits"].permute(1, 0, 2).reshape(rows, n * vocab).float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1)
    lse = top[:, 0] + torch.log(total)
    t = torch.where(e > 0, x - top, torch.zeros_like(x))
    entropy = torch.log(total) - (e * t).sum(1) / total
    asked = s["tokens"] >= 0
    logprob = x.gather(1, s["tokens"].clamp(min=0).long()[:, None])[:, 0] - lse
    out = dict(logprob=torch.where(asked, logprob, torch.zeros_like(logprob)), entropy=entropy, lse=lse)
    if s["case"]["top"]:
        del e, t
        best, ids = torch.sort(x, dim=1, descending=True, stable=True)
        k = s["case"]["top"]
        out.update(top_values=best[:, :k] - lse[:, None], top_ids=ids[:, :k].int())
    return out


def _plain_logprobs_backward(s):
    n, rows, vocab = s["logits"].shape
    y = s["logits"].float() - s["lse"][None, :, None]
    p = torch.exp(y)
    asked = s["tokens"] >= 0
    g = torch.where(asked, s["grad_logprob"], torch.zeros_like(s["grad_logprob"]))
    y = torch.where(p > 0, y, torch.zeros_like(y))
    d = -p * (g[None, :, None] + s["grad_entropy"][None, :, None] * (y + s["entropy"][None, :, None]))
    at = s["tokens"].clamp(min=0).long()
    d.index_put_((at // vocab, torch.arange(rows, device="cuda"), at % vocab), g, accumulate=True)
    return dict(dlogits=d.to(s["logits"].dtype))


_PLAIN = dict(pages=_plain_pages, rope=_plain_rope, rope_cached=_plain_rope_cached, rope_backward=_plain_rope_backward,
              attention=_plain_attention, logprobs=_plain_logprobs, logprobs_backward=_plain_logprobs_backward)


def exact(case, seed):
    """The definitions in 64 bits, a request or a block of rows at a time."""
    s = _inputs(case, seed)
    return {"pages": _exact_pages, "attention": _exact_attention, "logprobs": _exact_logprobs,
            "logprobs_backward": _exact_logprobs_backward}.get(case["op"], _exact_rope)(s)


def _exact_pages(s):
    page = s["case"]["page"]
    lens, new, free = s["lens"].tolist(), s["new"].tolist(), s["free"].tolist()
    table = s["table"].cpu().clone()
    left = int(s["free_count"])
    starts, positions, slots = [0], [], []
    for r, (have, more) in enumerate(zip(lens, new)):
        for column in range(-(-have // page), -(-(have + more) // page)):
            left -= 1
            table[r, column] = free[left]
        at = torch.arange(have, have + more)
        positions.append(at)
        slots.append(table[r, at // page].long() * page + at % page)
        starts.append(starts[-1] + more)
    pad = s["capacity"] - starts[-1]
    positions = torch.cat(positions + [torch.zeros(pad, dtype=torch.int64)])
    slots = torch.cat(slots + [torch.full((pad,), -1, dtype=torch.int64)])
    return dict(table=table, lens=torch.tensor([a + b for a, b in zip(lens, new)]).int(), starts=torch.tensor(starts).int(),
                positions=positions.int(), slots=slots.int(), free=torch.tensor([left]).int())


def _exact_rope(s):
    """Heads as complex numbers turned by e^(i angle); the gradient by the transposed Jacobian's two parts."""
    case = s["case"]
    q, kv, d, rot = case["q_heads"], case["kv_heads"], case["dim"], case["rot"]
    n, t = s["qkv"].shape[:2]
    half = rot // 2
    rows = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(rows[:, :half], rows[:, half:])
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    qkv = s["qkv"].double().view(n, t, q + 2 * kv, d)
    out, dqkv, dws = [], torch.zeros_like(qkv) if "dq" in s else None, []
    for lo, hi, name, weight in ((0, q, "dq", s["wq"].double()), (q, q + kv, "dk", s["wk"].double())):
        x = qkv[:, :, lo:hi]
        root = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
        unit = x / root
        if "dq" not in s:
            y = unit * weight
            z = torch.complex(y[..., first], y[..., second]) * turn[None, :, None]
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
            continue
        g = s[name].double()
        z = torch.complex(g[..., first], g[..., second]) * turn[None, :, None].conj()
        g[..., first], g[..., second] = z.real, z.imag
        dws.append((g * unit).sum((1, 2)))
        g = g * weight
        dqkv[:, :, lo:hi] = (g - unit * (g * unit).sum(-1, keepdim=True) / d) / root
    if "dq" in s:
        dqkv[:, :, q + kv:] = s["dv"].double()
        return dict(dqkv=dqkv.reshape(n, t, -1), dwq=dws[0], dwk=dws[1])
    if case["op"] == "rope":
        return dict(q=out[0], k=out[1])
    page = case["page"]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    at, off = (s["slots"] // page).long(), (s["slots"] % page).long()
    for h in range(kv):
        k_cache[:, at, h, off] = out[1][:, :, h]
        v_cache[:, at, h, off] = qkv[:, :, q + kv + h]
    return dict(q=out[0], k_cache=k_cache, v_cache=v_cache)


def _exact_attention(s):
    case = s["case"]
    n, batch, q, d = s["q"].shape
    kv, page = case["kv_heads"], case["page"]
    out = torch.zeros(n, batch, q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, batch, q), float("-inf"), dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        at = torch.arange(length, device="cuda")
        pages, off = s["table"][b].long()[at // page], at % page
        for h in range(kv):
            mine = slice(h * (q // kv), (h + 1) * (q // kv))
            k = s["k_cache"][:, pages, h, off].double()
            y = torch.einsum("ngd,ntd->ngt", s["q"][:, b, mine].double(), k) / math.sqrt(d)
            lse[:, b, mine] = torch.logsumexp(y, -1)
            weights = torch.exp(y - lse[:, b, mine, None])
            out[:, b, mine] = torch.einsum("ngt,ntd->ngd", weights, s["v_cache"][:, pages, h, off].double())
    return dict(out=out, lse=lse)


def _exact_logprobs(s):
    n, rows, vocab = s["logits"].shape
    found = dict(logprob=[], entropy=[], lse=[], top_values=[], top_ids=[])
    top = s["case"]["top"]
    for i in range(0, rows, 128):
        x = torch.cat(list(s["logits"][:, i:i + 128].double()), 1)
        y = torch.log_softmax(x, 1)
        token = s["tokens"][i:i + 128].long()
        mine = y[torch.arange(len(token), device="cuda"), token.clamp(min=0)]
        found["logprob"].append(torch.where(token < 0, 0.0, mine))
        found["entropy"].append(torch.special.entr(y.exp()).sum(1))
        found["lse"].append(torch.logsumexp(x, 1))
        left = x.clone()
        for _ in range(top):
            best = left.amax(1, keepdim=True)
            at = torch.where(left == best, torch.arange(n * vocab, device="cuda"), n * vocab).amin(1, keepdim=True)
            found["top_values"].append(y.gather(1, at))
            found["top_ids"].append(at.int())
            left.scatter_(1, at, float("nan"))
            left.nan_to_num_(nan=float("-inf"), neginf=float("-inf"), posinf=float("inf"))
    out = {k: torch.cat(found[k]) for k in ("logprob", "entropy", "lse")}
    if top:
        for k in ("top_values", "top_ids"):
            out[k] = torch.cat([torch.cat(found[k][j:j + top], 1) for j in range(0, len(found[k]), top)])
    return out


def _exact_logprobs_backward(s):
    n, rows, vocab = s["logits"].shape
    out = torch.empty(n, rows, vocab, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 128):
        mine = slice(i, i + 128)
        y = torch.cat(list(s["logits"][:, mine].double()), 1) - s["lse"][mine].double()[:, None]
        p = torch.exp(y)
        token = s["tokens"][mine].long()
        g = torch.where(token < 0, 0.0, s["grad_logprob"][mine].double())[:, None]
        picked = (torch.arange(n * vocab, device="cuda")[None] == token[:, None]).double()
        # d entropy / d x = -p (log p + entropy) = entr(p) - p entropy
        d = g * (picked - p) + s["grad_entropy"][mine].double()[:, None] * \
            (torch.special.entr(p) - p * s["entropy"][mine].double()[:, None])
        out[:, mine] = d.view(len(token), n, vocab).permute(1, 0, 2)
    return dict(dlogits=out)
