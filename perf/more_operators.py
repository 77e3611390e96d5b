"""Cases of the prompt and training operators over virtual ranks: causal attention over whole prompts (dense, and over a
paged cache that holds earlier tokens) with its gradient, and the embedding lookup over vocabulary shards with its gradient.

Every tensor that belongs to a rank has the rank as its first dimension (N ranks in one GPU): heads and vocabulary are
split over the ranks; sequences, tables, tokens and the embedded rows are shared by all of them.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the first message of a chat on one rank: latency
        dict(name="prompt_one_97", op="prompt", ranks=1, tokens=97, sequences=1, q_heads=8, kv_heads=1, dim=128, dtype="bf16"),
        # packed prompts of 28 to 936 tokens on eight ranks (64 query heads, 8 key heads in all)
        dict(name="prompt_packed_8192", op="prompt", ranks=8, tokens=8192, sequences=17, q_heads=8, kv_heads=1, dim=128,
             dtype="bf16"),
        # one long document on two ranks
        dict(name="prompt_long_16384", op="prompt", ranks=2, tokens=16384, sequences=1, q_heads=8, kv_heads=1, dim=128,
             dtype="bf16"),
        # 32 bits, a head size and a group that are no powers of two
        dict(name="prompt_f32_2777", op="prompt", ranks=2, tokens=2777, sequences=5, q_heads=6, kv_heads=2, dim=80,
             dtype="f32"),
        # chunks of six requests' prompts behind what the paged cache holds of them, on eight ranks
        dict(name="cached_chunks_2048", op="cached", ranks=8, tokens=2048, sequences=6, history=8192, q_heads=8, kv_heads=1,
             dim=128, page=16, dtype="bf16"),
        # a few drafted tokens to be verified behind a long context: the cache's length is all there is to split
        dict(name="cached_verify_5", op="cached", ranks=1, tokens=5, sequences=1, history=30011, q_heads=16, kv_heads=2,
             dim=128, page=64, dtype="bf16"),
        # gradients of a training step over packed sequences, four ranks, odd number of tokens
        dict(name="backward_packed_4097", op="backward", ranks=4, tokens=4097, sequences=9, q_heads=8, kv_heads=2, dim=128,
             dtype="bf16"),
        # gradients of one long sequence, head size 64
        dict(name="backward_long_8192", op="backward", ranks=2, tokens=8192, sequences=1, q_heads=8, kv_heads=2, dim=64,
             dtype="bf16"),
        # the words of a decode step of seven requests
        dict(name="embed_decode_7", op="embed", ranks=8, tokens=7, vocab=16384, hidden=4096, dtype="bf16"),
        # the words of packed prompts, shards of an odd size
        dict(name="embed_prompt_16384", op="embed", ranks=8, tokens=16384, vocab=16003, hidden=7168, dtype="bf16"),
        # the gradient of a small model's table
        dict(name="embed_backward_300", op="embed_backward", ranks=2, tokens=300, vocab=1001, hidden=512, dtype="f32"),
        # the gradient of a training step: words as often as they are in texts
        dict(name="embed_backward_16385", op="embed_backward", ranks=8, tokens=16385, vocab=4001, hidden=4096, dtype="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return min(max(v, lo), hi)

    op = rng.choice(["prompt", "prompt", "cached", "cached", "backward", "backward", "embed", "embed_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ranks = rng.choice([1, 2, 4, 8])
    if op.startswith("embed"):
        vocab, hidden = spread(500, 150000 // ranks), 8 * spread(8, 1024)
        if op == "embed_backward":
            hidden = 8 * max(1, min(hidden, 2 ** 28 // (ranks * vocab)) // 8)
        return dict(op=op, ranks=ranks, tokens=spread(1, max(2, 2 ** 26 // hidden)), vocab=vocab, hidden=hidden, dtype=dtype)
    kv = rng.choice([1, 1, 2, 4])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dim = rng.choice([40, 64, 64, 80, 96, 128, 128])
    heads = ranks * kv * group
    case = dict(op=op, ranks=ranks, q_heads=kv * group, kv_heads=kv, dim=dim, dtype=dtype)
    most = 2 ** 30 if op != "backward" else 2 ** 28  # scores of all heads, masked ones among them
    if op == "cached":
        case["sequences"] = spread(1, 32)
        case["tokens"] = case["sequences"] + spread(1, 2048)
        keys = max(1, most // (heads * case["tokens"]) - case["tokens"])
        case["history"] = spread(1, max(2, min(131072, 2 * keys // (case["sequences"] + 1))))
        case["page"] = rng.choice([8, 16, 32, 64, 128])
        return case
    case["tokens"] = spread(1, max(2, math.isqrt(most // heads)))
    case["sequences"] = spread(1, min(64, case["tokens"]))
    return case


def _lengths(case):
    """Lengths of the packed sequences: they grow evenly from short to long ones."""
    n = case["sequences"]
    least = 1 if case["op"] == "cached" else 0  # every request of a step adds a token or more; a packed row may be empty
    more = case["tokens"] - least * n
    ends = [more * i * i // (n * n) for i in range(n + 1)]
    return [least + b - a for a, b in zip(ends, ends[1:])]


def _histories(case):
    """Cached tokens before the step of each request: the single request's is the longest, several are spread from 0."""
    n, longest = case["sequences"], case["history"]
    return [longest] if n == 1 else [longest * i // (n - 1) for i in range(n)]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    n, t = case["ranks"], case["tokens"]
    if case["op"] == "embed":
        # the tokens' numbers in, and once each row that any of them asks for; a row out for each token
        rank = torch.arange(1, n * case["vocab"] + 1, dtype=torch.float64)
        often = torch.log1p(1 / rank) / math.log(n * case["vocab"] + 1)
        rows = int((1 - (1 - often) ** t).sum())
        return {"bytes": 4 * t + (rows + t) * case["hidden"] * size, "flops": t * case["hidden"]}
    if case["op"] == "embed_backward":
        return {"bytes": 4 * t + t * case["hidden"] * size + 4 * n * case["vocab"] * case["hidden"],
                "flops": 2 * t * case["hidden"]}
    q, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    lengths = _lengths(case)
    if case["op"] == "cached":
        histories = _histories(case)
        pairs = sum(a * h + a * (a + 1) // 2 for a, h in zip(lengths, histories))
        keys = sum(lengths) + sum(histories)
        extra = 4 * (keys // case["page"]) + 8 * case["sequences"]
    else:
        pairs, keys, extra = sum(a * (a + 1) // 2 for a in lengths), t, 4 * case["sequences"]
    if case["op"] == "backward":
        moved = n * size * d * (4 * t * q + 4 * t * kv) + 4 * n * t * q
        return {"bytes": moved + extra, "flops": 10 * n * q * pairs * d}
    return {"bytes": n * size * d * (2 * t * q + 2 * keys * kv) + 4 * n * t * q + extra, "flops": 4 * n * q * pairs * d}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device="cuda")

    s = dict(case=case)
    n, t, dtype = case["ranks"], case["tokens"], DTYPES[case["dtype"]]
    if case["op"].startswith("embed"):
        words, hidden = n * case["vocab"], case["hidden"]
        # the k-th most frequent word about 1 / k as often as the first; a few padding tokens
        u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
        tokens = ((words + 1.0) ** u - 1.0).long().clamp(max=words - 1)
        padding = torch.rand(t, generator=gen, device="cuda") < 1 / 64
        s["tokens"] = torch.where(padding, torch.full_like(tokens, -1), tokens).int()
        s["scale"] = math.sqrt(hidden)
        if case["op"] == "embed":
            s["tables"] = normal(n, case["vocab"], hidden, dtype=dtype, scale=hidden ** -0.5)
        else:
            s["dout"] = normal(t, hidden, dtype=dtype)
        return s
    q, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    order = shuffled(case["sequences"])
    lengths = torch.tensor(_lengths(case), device="cuda")[order]
    s["starts"] = torch.cat([torch.zeros_like(lengths[:1]), torch.cumsum(lengths, 0)]).int()
    if case["op"] == "cached":
        s["q"] = normal(n, t, q, d, dtype=dtype)
        page = case["page"]
        lens = lengths + torch.tensor(_histories(case), device="cuda")[order]
        have = (lens + page - 1) // page
        most = int(have.max())
        pages = int(have.sum()) + 5
        mix = shuffled(pages)
        first = torch.cumsum(have, 0) - have
        columns = torch.arange(most, device="cuda")
        at = (first[:, None] + columns[None]).clamp(max=pages - 1)
        s["table"] = torch.where(columns[None] < have[:, None], mix[at], torch.full_like(at, -1)).int()
        s["lens"] = lens.int()
        s["keys"] = sum(_lengths(case)) + sum(_histories(case))
        s["k_cache"] = normal(n, pages, kv, page, d, dtype=dtype)
        s["v_cache"] = normal(n, pages, kv, page, d, dtype=dtype)
        return s
    # queries and keys have been normed and rotated into tensors of their own, values are where the projection left them
    s["q"], s["k"] = normal(n, t, q, d, dtype=dtype), normal(n, t, kv, d, dtype=dtype)
    s["v"] = normal(n, t, (q + 2 * kv) * d, dtype=dtype)[:, :, (q + kv) * d:].unflatten(2, (kv, d))
    if case["op"] == "backward":
        s["out"], s["lse"] = _plain_attention(s).values()
        s["dout"] = normal(n, t, q, d, dtype=dtype)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from collective_communication_gb300 import binding as B
    n, t = case["ranks"], case["tokens"]
    if case["op"] == "embed":
        s["embedded"] = torch.empty(t, case["hidden"], dtype=s["tables"].dtype, device="cuda")
        need = 0
    elif case["op"] == "embed_backward":
        s["dtables"] = torch.empty(n, case["vocab"], case["hidden"], device="cuda")
        need = B.embed_tokens_workspace_bytes(t, case["hidden"])
    else:
        if case["op"] == "backward":
            s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
            s["dv"] = torch.empty_like(s["k"])
        else:
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(n, t, case["q_heads"], device="cuda")
        need = B.prompt_attention_workspace_bytes(n, t, case["q_heads"], case["kv_heads"], case["dim"])
    s["workspace"] = B.OpWorkspace(need)
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from collective_communication_gb300 import binding as B
    case = s["case"]
    if case["op"] == "embed":
        B.embed_tokens(s["tokens"], s["tables"], s["embedded"], s["workspace"], scale=s["scale"])
        return dict(embedded=s["embedded"])
    if case["op"] == "embed_backward":
        B.embed_tokens_backward(s["tokens"], s["dout"], s["dtables"], s["workspace"], scale=s["scale"])
        return dict(dtables=s["dtables"])
    if case["op"] == "prompt":
        B.prompt_attention(s["q"], s["k"], s["v"], s["starts"], s["out"], s["lse"], s["workspace"])
        return dict(out=s["out"], lse=s["lse"])
    if case["op"] == "cached":
        B.prompt_attention_cached(s["q"], s["k_cache"], s["v_cache"], s["table"], s["starts"], s["lens"], s["out"], s["lse"],
                                  s["workspace"])
        return dict(out=s["out"], lse=s["lse"])
    B.prompt_attention_backward(s["q"], s["k"], s["v"], s["starts"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"], s["dv"],
                                s["workspace"])
    return dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])


def _flat(s):
    """Queries [n, kv_heads, group * tokens, dim], keys and values [n, kv_heads, keys, dim] of all sequences in 32 bits, and
    which query token sees which key."""
    case = s["case"]
    n, t, q, d = s["q"].shape
    kv = case["kv_heads"]
    starts = s["starts"].long()
    token = torch.arange(t, device="cuda")
    sequence = torch.searchsorted(starts[1:].contiguous(), token, right=True)
    if case["op"] == "cached":
        lens, page = s["lens"].long(), case["page"]
        position = lens[sequence] - (starts[sequence + 1] - starts[sequence]) + token - starts[sequence]
        ends = torch.cumsum(lens, 0)
        key = torch.arange(s["keys"], device="cuda")
        owner = torch.searchsorted(ends, key, right=True)
        place = key - (ends - lens)[owner]
        at = s["table"].long()[owner, place // page]
        k, v = (c[:, at, :, place % page].permute(1, 2, 0, 3).float() for c in (s["k_cache"], s["v_cache"]))
    else:
        position = token - starts[sequence]
        owner, place = sequence, position
        k, v = s["k"].permute(0, 2, 1, 3).float(), s["v"].permute(0, 2, 1, 3).float()
    sees = (sequence[:, None] == owner[None]) & (place[None] <= position[:, None])
    return _grouped(s["q"], kv), k, v, sees


def _grouped(x, kv):
    n, t, q, d = x.shape
    return x.float().view(n, t, kv, q // kv, d).permute(0, 2, 3, 1, 4).reshape(n, kv, (q // kv) * t, d)


def _ungrouped(x, t):
    """[n, kv_heads, group * tokens, dim] back to [n, tokens, q_heads, dim]."""
    n, kv, _, d = x.shape
    return x.view(n, kv, -1, t, d).permute(0, 3, 1, 2, 4).reshape(n, t, -1, d)


def _scores(query, k, sees):
    scores = torch.matmul(query * query.shape[-1] ** -0.5, k.transpose(-1, -2))
    t = sees.shape[0]
    scores.view(*scores.shape[:2], -1, t, scores.shape[-1]).masked_fill_(~sees, float("-inf"))
    return scores


def _plain_attention(s):
    query, k, v, sees = _flat(s)
    scores = _scores(query, k, sees)
    top = scores.amax(-1, keepdim=True)
    e = scores.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / total
    t = sees.shape[0]
    lse = _ungrouped(top + torch.log(total), t)[..., 0]
    return dict(out=_ungrouped(out, t).to(s["q"].dtype), lse=lse.contiguous())


def _plain_backward(s):
    kv, dtype, t = s["case"]["kv_heads"], s["q"].dtype, s["q"].shape[1]
    query, k, v, sees = _flat(s)
    p = _scores(query, k, sees).sub_(_grouped(s["lse"][..., None], kv)).exp_()
    dout = _grouped(s["dout"], kv)
    dv = torch.matmul(p.transpose(-1, -2), dout)
    dp = torch.matmul(dout, v.transpose(-1, -2))
    dp -= (p * dp).sum(-1, keepdim=True)
    ds = p.mul_(dp).mul_(query.shape[-1] ** -0.5)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(-1, -2), query)
    return dict(dq=_ungrouped(dq, t).to(dtype), dk=dk.permute(0, 2, 1, 3).to(dtype).contiguous(),
                dv=dv.permute(0, 2, 1, 3).to(dtype).contiguous())


def _plain_embed(s):
    tokens, tables = s["tokens"].long(), s["tables"]
    rows = tables.view(-1, tables.shape[-1])[tokens.clamp(min=0)].float() * s["scale"]
    return dict(embedded=torch.where(tokens[:, None] >= 0, rows, torch.zeros_like(rows)).to(tables.dtype))


def _plain_embed_backward(s):
    case, tokens = s["case"], s["tokens"].long()
    rows = torch.where(tokens[:, None] >= 0, s["dout"].float() * s["scale"], torch.zeros((), device="cuda"))
    grad = torch.zeros(case["ranks"] * case["vocab"], case["hidden"], device="cuda")
    grad.index_add_(0, tokens.clamp(min=0), rows)
    return dict(dtables=grad.view(case["ranks"], case["vocab"], case["hidden"]))


_PLAIN = dict(prompt=_plain_attention, cached=_plain_attention, backward=_plain_backward, embed=_plain_embed,
              embed_backward=_plain_embed_backward)


def exact(case, seed):
    """The definitions in 64 bits: a sequence and a rank at a time, gradients by differentiating the forward form."""
    s = _inputs(case, seed)
    if case["op"] == "embed":
        word = s["tokens"].long()
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        for r in range(case["ranks"]):
            mine = (word // case["vocab"] == r).nonzero()[:, 0]
            out[mine] = s["tables"][r].index_select(0, word[mine] % case["vocab"]).double() * s["scale"]
        return dict(embedded=out)
    if case["op"] == "embed_backward":
        word, at = torch.sort(s["tokens"].long())
        grad = torch.zeros(case["ranks"] * case["vocab"], case["hidden"], dtype=torch.float64, device="cuda")
        used, counts = torch.unique_consecutive(word, return_counts=True)
        rows = s["dout"].double().index_select(0, at) * s["scale"]
        for w, part in zip(used.tolist(), torch.split(rows, counts.tolist())):
            if w >= 0:
                grad[w] = part.sum(0)
        return dict(dtables=grad.view(case["ranks"], case["vocab"], -1))
    n, t, q, d = s["q"].shape
    kv, bounds = case["kv_heads"], s["starts"].tolist()
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    found = dict(out=zeros(n, t, q, d), lse=zeros(n, t, q), dq=zeros(n, t, q, d), dk=zeros(n, t, kv, d), dv=zeros(n, t, kv, d))
    for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        for r in range(n):
            x = s["q"][r, a:b].double()
            if case["op"] == "cached":
                length = int(s["lens"][i])
                place = torch.arange(length, device="cuda")
                pages, off = s["table"][i].long()[place // case["page"]], place % case["page"]
                k, v = s["k_cache"][r][pages, :, off].double(), s["v_cache"][r][pages, :, off].double()
            else:
                length = b - a
                k, v = s["k"][r, a:b].double(), s["v"][r, a:b].double()
            later = torch.ones(b - a, length, dtype=torch.bool, device="cuda").triu(length - (b - a) + 1)
            leaves = [z.requires_grad_(case["op"] == "backward") for z in (x, k, v)]
            y = torch.einsum("thgd,shd->hgts", x.unflatten(1, (kv, q // kv)), k) / math.sqrt(d)
            y = y.masked_fill(later, float("-inf"))
            lse = torch.logsumexp(y, -1)
            out = torch.einsum("hgts,shd->thgd", torch.softmax(y, -1), v).flatten(1, 2)
            if case["op"] == "backward":
                grads = torch.autograd.grad(out, leaves, s["dout"][r, a:b].double())
                for name, g in zip(("dq", "dk", "dv"), grads):
                    found[name][r, a:b] = g
            else:
                found["out"][r, a:b] = out
                found["lse"][r, a:b] = lse.permute(2, 0, 1).flatten(1)
    return {k: found[k] for k in (("dq", "dk", "dv") if case["op"] == "backward" else ("out", "lse"))}
