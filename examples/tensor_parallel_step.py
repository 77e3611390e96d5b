"""Steps of a small tensor-parallel language model over virtual ranks, from page
tables to the all-reduced gradient.

Each of N ranks holds some query heads, one key head and a range of the
vocabulary of a one-layer model with random weights. A step of decoding:

  page_tables          pages and cache slots of the requests' next tokens
  embed_tokens         their rows, over the ranks' shards of the table
  (torch)              each rank's query, key and value projection
  qk_norm_rope_cached  norm and rotation; keys and values into the paged cache
  decode_attention     one new token per request over the cache
  (torch)              each rank's part of the output projection
  oneshot              AllReduce of the parts, to every rank
  (torch)              each rank's shard of the logits
  token_logprobs       the next token of each request, its log probability and
                       the entropy, over the shards

The first step's kernels are captured into a CUDA graph and replayed for the
others: lengths, tables and tokens are device tensors that the graph updates
itself. After the last step, the gradient of the log probabilities goes back
through the logits, and the norm weights' gradient, a part on every rank, is
summed by the ring AllReduce.

With prompts, a step of their own comes first: all tokens of all prompts at once,
with prompt_attention_cached in the place of decode_attention. train() is a step of
training on packed sequences: the dense forms of the same operators forward, and
the gradients of all weights, with AllReduces of what the ranks hold parts of.

Usage: python examples/tensor_parallel_step.py [--ranks 8] [--requests 6] [--steps 20] [--prompt 40]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

from collective_communication_gb300 import binding as B

HEADS, DIM, PAGE, HIDDEN, WORDS, MAX_TOKENS = 4, 64, 16, 256, 501, 256  # per rank: query heads, head size, words
EPS = 1e-6


class Model:
    """Weights of the ranks, stacked with the rank first."""

    def __init__(self, ranks, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

        self.ranks, self.dtype = ranks, dtype
        self.embed = normal(ranks * WORDS, HIDDEN, scale=1.0)
        self.wqkv = normal(ranks, HIDDEN, (HEADS + 2) * DIM, scale=HIDDEN ** -0.5)
        self.wo = normal(ranks, HEADS * DIM, HIDDEN, scale=(ranks * HEADS * DIM) ** -0.5)
        self.head = normal(ranks, HIDDEN, WORDS, scale=2 * HIDDEN ** -0.5)
        self.wq, self.wk = normal(DIM, scale=0.2) + 1, normal(DIM, scale=0.2) + 1
        angle = torch.arange(MAX_TOKENS, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(DIM // 2, device="cuda") / (DIM // 2))[None]
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()


class Decoder:
    """The requests' state, the buffers of a step and the step itself."""

    def __init__(self, model, requests):
        n, dt, r = model.ranks, model.dtype, requests
        self.model, self.requests = model, r

        def empty(*shape, dtype=dt):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        def ints(*shape):
            return empty(*shape, dtype=torch.int32)

        pages = r * MAX_TOKENS // PAGE
        self.pages = pages
        self.lens, self.new = ints(r), torch.ones(r, dtype=torch.int32, device="cuda")
        self.table = ints(r, MAX_TOKENS // PAGE)
        self.free = torch.randperm(pages, device="cuda").to(torch.int32)
        self.free_count = torch.tensor([pages], dtype=torch.int32, device="cuda")
        self.lens_out, self.starts, self.positions, self.slots = ints(r), ints(r + 1), ints(r), ints(r)
        self.free_out = ints(1)
        self.tokens = torch.arange(r, dtype=torch.int32, device="cuda")
        self.x = empty(r, HIDDEN)
        self.qkv = empty(n, r, (HEADS + 2) * DIM)
        self.q, self.attended = empty(n, r, HEADS, DIM), empty(n, r, HEADS, DIM)
        self.k_cache, self.v_cache = empty(n, pages, 1, PAGE, DIM), empty(n, pages, 1, PAGE, DIM)
        self.parts, self.sums = empty(n, r * HIDDEN), empty(n, r * HIDDEN)
        self.logits = empty(n, r, WORDS)
        self.logprob, self.entropy, self.lse = (empty(r, dtype=torch.float32) for _ in range(3))
        self.top_values, self.top_ids = empty(r, 3, dtype=torch.float32), ints(r, 3)
        self.workspace = B.OpWorkspace(max(B.decode_attention_workspace_bytes(n, r, HEADS, 1, DIM),
                                           B.prompt_attention_workspace_bytes(n, r * MAX_TOKENS, HEADS, 1, DIM),
                                           B.token_logprobs_workspace_bytes(r, 3),
                                           B.qk_norm_rope_workspace_bytes(n, DIM)))

    def step(self):
        m, r, n = self.model, self.requests, self.model.ranks
        B.page_tables(self.lens, self.new, self.free, self.free_count, self.table, PAGE, self.pages, self.lens_out,
                      self.starts, self.positions, self.slots, self.free_out, self.workspace)
        x = self.x
        B.embed_tokens(self.tokens, m.embed.view(n, WORDS, HIDDEN), x, self.workspace)
        torch.matmul(x, m.wqkv, out=self.qkv)
        B.qk_norm_rope_cached(self.qkv, m.wq, m.wk, m.cos_sin, self.positions, self.slots, self.q, self.k_cache,
                              self.v_cache, self.workspace, eps=EPS)
        B.decode_attention(self.q, self.k_cache, self.v_cache, self.table, self.lens_out, self.attended, None,
                           self.workspace)
        torch.matmul(self.attended.view(n, r, HEADS * DIM), m.wo, out=self.parts.view(n, r, HIDDEN))
        B.oneshot(list(self.parts), list(self.sums))  # every rank gets the sum
        hidden = x + self.sums.view(n, r, HIDDEN)
        torch.matmul(hidden, m.head, out=self.logits)
        # the most likely word is the next token; its log probability is that of the first alternative
        B.token_logprobs(self.logits, self.tokens, self.logprob, self.entropy, self.lse, self.top_values, self.top_ids,
                         self.workspace)
        self.tokens.copy_(self.top_ids[:, 0])
        self.lens.copy_(self.lens_out)
        self.free_count.copy_(self.free_out)

    def prefill(self, prompts):
        """All tokens of the prompts (one for each request) at once; leaves the decoder with the next token of each."""
        m, r, n, dt = self.model, self.requests, self.model.ranks, self.model.dtype
        t = sum(len(p) for p in prompts)
        tokens = torch.tensor([w for p in prompts for w in p], dtype=torch.int32, device="cuda")
        new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        positions, slots = (torch.zeros(t, dtype=torch.int32, device="cuda") for _ in range(2))
        B.page_tables(self.lens, new, self.free, self.free_count, self.table, PAGE, self.pages, self.lens_out, self.starts,
                      positions, slots, self.free_out, self.workspace)
        x = torch.empty(t, HIDDEN, dtype=dt, device="cuda")
        B.embed_tokens(tokens, m.embed.view(n, WORDS, HIDDEN), x, self.workspace)
        qkv = torch.matmul(x, m.wqkv)
        q, attended = (torch.empty(n, t, HEADS, DIM, dtype=dt, device="cuda") for _ in range(2))
        B.qk_norm_rope_cached(qkv, m.wq, m.wk, m.cos_sin, positions, slots, q, self.k_cache, self.v_cache, self.workspace,
                              eps=EPS)
        B.prompt_attention_cached(q, self.k_cache, self.v_cache, self.table, self.starts, self.lens_out, attended, None,
                                  self.workspace)
        ends = self.starts[1:].long() - 1  # the prompts' last tokens are all that the next words need
        parts = torch.matmul(attended[:, ends].reshape(n, r, HEADS * DIM), m.wo)
        B.oneshot(list(parts.view(n, -1)), list(self.sums))
        torch.matmul(x[ends] + self.sums.view(n, r, HIDDEN), m.head, out=self.logits)
        B.token_logprobs(self.logits, self.tokens, self.logprob, self.entropy, self.lse, self.top_values, self.top_ids,
                         self.workspace)
        self.tokens.copy_(self.top_ids[:, 0])
        self.lens.copy_(self.lens_out)
        self.free_count.copy_(self.free_out)

    def backward(self):
        """The gradient of the tokens' log probabilities with respect to the logits, and, for a gradient of the queries
        and keys, the norm weights' gradient summed over the ranks."""
        m, r, n = self.model, self.requests, self.model.ranks
        ones = torch.ones(r, device="cuda")
        dlogits = torch.empty_like(self.logits)
        B.token_logprobs_backward(self.logits, self.tokens, self.lse, self.entropy, ones, None, dlogits, self.workspace)
        dhidden = torch.matmul(dlogits, m.head.transpose(1, 2))
        dq = torch.matmul(dhidden, m.wo.transpose(1, 2)).view(n, r, HEADS, DIM)
        dk = dq[:, :, :1].contiguous()
        dqkv = torch.empty_like(self.qkv)
        dwq, dwk = (torch.empty((n, DIM), device="cuda") for _ in range(2))
        B.qk_norm_rope_backward(self.qkv, m.wq, m.wk, m.cos_sin, self.positions, dq, dk, dk, dqkv, dwq, dwk,
                                self.workspace, eps=EPS)
        grads = torch.cat([dwq, dwk], 1)
        summed = torch.empty_like(grads)
        ring = B.Workspace(n, 0x1, "Simple", 65536)
        B.allreduce(list(grads), list(summed), list(range(n)), 0x1, "Simple", ring, 65536, 4)
        status = B.get_status(ring)
        if status != B.Status.OK:
            raise RuntimeError(f"ring AllReduce reported {status.name}")
        return dlogits, dqkv, grads, summed


def plain_step(model, keys, values, tokens, position):
    """The same step with elementary operations in 64 bits, all ranks' heads together; appends to keys and values."""
    m = model
    x = m.embed[tokens.long()].double()
    qkv = torch.einsum("rh,nhw->rnw", x, m.wqkv.double()).view(len(tokens), m.ranks, HEADS + 2, DIM)

    def turn(z, weight):
        z = z / (z.square().mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
        c, s = m.cos_sin[position].double().chunk(2)
        a, b = z.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q = turn(qkv[:, :, :HEADS], m.wq)
    keys.append(turn(qkv[:, :, HEADS], m.wk))
    values.append(qkv[:, :, HEADS + 1])
    k, v = torch.stack(keys, 2), torch.stack(values, 2)
    p = torch.softmax(torch.einsum("rngd,rntd->rngt", q, k) * DIM ** -0.5, -1)
    o = torch.einsum("rngt,rntd->rngd", p, v).flatten(2)
    hidden = x + torch.einsum("rnw,nwh->rh", o, m.wo.double())
    return torch.log_softmax(torch.einsum("rh,nhw->rnw", hidden, m.head.double()).flatten(1), 1)


def plain_model(weights, tokens, starts, positions, cos_sin):
    """Log probabilities [tokens, words] of packed sequences with elementary operations; weights by name."""
    w = weights
    ranks = w["wqkv"].shape[0]
    x = w["embed"][tokens]
    qkv = torch.einsum("th,nhw->tnw", x, w["wqkv"]).unflatten(2, (HEADS + 2, DIM))
    c, s = cos_sin[positions][:, None, None].chunk(2, -1)

    def turn(z, weight):
        z = z / (z.square().mean(-1, keepdim=True) + EPS).sqrt() * weight
        a, b = z.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k, v = turn(qkv[:, :, :HEADS], w["wq"]), turn(qkv[:, :, HEADS:HEADS + 1], w["wk"])[:, :, 0], qkv[:, :, HEADS + 1]
    outs = []
    for a, b in zip(starts, starts[1:]):
        y = torch.einsum("tngd,snd->ngts", q[a:b], k[a:b]) * DIM ** -0.5
        y = y.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device=y.device).triu(1), float("-inf"))
        outs.append(torch.einsum("ngts,snd->tngd", torch.softmax(y, -1), v[a:b]))
    o = torch.cat(outs).reshape(len(tokens), ranks, HEADS * DIM)
    hidden = x + torch.einsum("tnw,nwh->th", o, w["wo"])
    return torch.log_softmax(torch.einsum("th,nhw->tnw", hidden, w["head"]).flatten(1), 1)


class Trainer:
    """Buffers of a training step on `tokens` packed tokens of up to `sequences` sequences, and the step."""

    def __init__(self, model, tokens, sequences):
        n, dt, t = model.ranks, model.dtype, tokens
        self.model = model

        def empty(*shape, dtype=dt):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        def ints(*shape):
            return empty(*shape, dtype=torch.int32)

        f32 = torch.float32
        self.tokens, self.targets, self.positions, self.starts = ints(t), ints(t), ints(t), ints(sequences + 1)
        self.x = empty(t, HIDDEN)
        self.qkv, self.dqkv = empty(n, t, (HEADS + 2) * DIM), empty(n, t, (HEADS + 2) * DIM)
        self.q, self.k, self.out = empty(n, t, HEADS, DIM), empty(n, t, 1, DIM), empty(n, t, HEADS, DIM)
        self.dq, self.dk, self.dv = empty(n, t, HEADS, DIM), empty(n, t, 1, DIM), empty(n, t, 1, DIM)
        self.lse = empty(n, t, HEADS, dtype=f32)
        self.parts, self.sums = empty(n, t * HIDDEN), empty(n, t * HIDDEN)
        self.logits, self.dlogits = empty(n, t, WORDS), empty(n, t, WORDS)
        self.logprob, self.entropy, self.word_lse = (empty(t, dtype=f32) for _ in range(3))
        self.grad = empty(t, dtype=f32)
        self.norm_grads, self.norm_sums = empty(n, 2, DIM, dtype=f32), empty(n, 2, DIM, dtype=f32)
        self.table_grad = empty(n, WORDS, HIDDEN, dtype=f32)
        self.grads = {}
        self.workspace = B.OpWorkspace(max(B.prompt_attention_workspace_bytes(n, t, HEADS, 1, DIM),
                                           B.qk_norm_rope_workspace_bytes(n, DIM), B.token_logprobs_workspace_bytes(t, 0),
                                           B.embed_tokens_workspace_bytes(t, HIDDEN)))
        self.ring = B.Workspace(n, 0x1, "Simple", 65536)

    def reduce(self):
        """The sum of the ranks' parts, which every rank gets; the first one's."""
        B.oneshot(list(self.parts), list(self.sums))
        return self.sums[0].view(-1, HIDDEN)

    def step(self):
        """Log probabilities of the targets, and the gradients of their sum weighted by `grad`."""
        m, n, ws = self.model, self.model.ranks, self.workspace
        t = self.tokens.numel()
        tables = m.embed.view(n, WORDS, HIDDEN)
        B.embed_tokens(self.tokens, tables, self.x, ws)
        torch.matmul(self.x, m.wqkv, out=self.qkv)
        B.qk_norm_rope(self.qkv, m.wq, m.wk, m.cos_sin, self.positions, self.q, self.k, ws, eps=EPS)
        v = self.qkv[:, :, (HEADS + 1) * DIM:].unflatten(2, (1, DIM))
        B.prompt_attention(self.q, self.k, v, self.starts, self.out, self.lse, ws)
        attended = self.out.view(n, t, HEADS * DIM)
        torch.matmul(attended, m.wo, out=self.parts.view(n, t, HIDDEN))
        hidden = self.x + self.reduce()
        torch.matmul(hidden, m.head, out=self.logits)
        B.token_logprobs(self.logits, self.targets, self.logprob, self.entropy, self.word_lse, None, None, ws)
        # backward
        B.token_logprobs_backward(self.logits, self.targets, self.word_lse, self.entropy, self.grad, None, self.dlogits, ws)
        self.grads["head"] = torch.matmul(hidden.t(), self.dlogits)
        torch.matmul(self.dlogits, m.head.transpose(1, 2), out=self.parts.view(n, t, HIDDEN))
        dhidden = self.reduce().clone()
        self.grads["wo"] = torch.matmul(attended.transpose(1, 2), dhidden)
        dout = torch.matmul(dhidden, m.wo.transpose(1, 2)).view(n, t, HEADS, DIM)
        B.prompt_attention_backward(self.q, self.k, v, self.starts, self.out, self.lse, dout, self.dq, self.dk, self.dv, ws)
        B.qk_norm_rope_backward(self.qkv, m.wq, m.wk, m.cos_sin, self.positions, self.dq, self.dk, self.dv, self.dqkv,
                                self.norm_grads[:, 0], self.norm_grads[:, 1], ws, eps=EPS)
        self.grads["wqkv"] = torch.matmul(self.x.t(), self.dqkv)
        torch.matmul(self.dqkv, m.wqkv.transpose(1, 2), out=self.parts.view(n, t, HIDDEN))
        dx = dhidden + self.reduce()
        B.embed_tokens_backward(self.tokens, dx, self.table_grad, ws)
        self.grads["embed"] = self.table_grad.view(-1, HIDDEN)
        B.allreduce(list(self.norm_grads.view(n, -1)), list(self.norm_sums.view(n, -1)), list(range(n)), 0x1, "Simple",
                    self.ring, 65536, 4)
        self.grads["wq"], self.grads["wk"] = self.norm_sums[0, 0], self.norm_sums[0, 1]


def train(ranks=4, lens=(50, 1, 77), dtype=torch.float32, seed=1, graph=True):
    """A training step, captured and replayed; returns the log probabilities' largest difference from the plain form's in
    64 bits and each weight's gradient's, relative to its norm."""
    model = Model(ranks, dtype)
    trainer = Trainer(model, sum(lens), len(lens))
    g = torch.Generator(device="cuda").manual_seed(seed)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    if graph:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            trainer.step()  # library handles are made outside of the capture
        torch.cuda.current_stream().wait_stream(stream)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            trainer.step()
    trainer.tokens.copy_(torch.randint(0, ranks * WORDS, (starts[-1],), generator=g, device="cuda"))
    targets = torch.cat([trainer.tokens[1:], trainer.tokens[:1]])
    targets[[b - 1 for b in starts[1:] if b > 0]] = -1  # nothing follows a sequence's last token
    trainer.targets.copy_(targets)
    trainer.positions.copy_(ints([i for n in lens for i in range(n)]))
    trainer.starts.copy_(ints(starts))
    trainer.grad.copy_(-torch.rand(starts[-1], generator=g, device="cuda"))
    if graph:
        captured.replay()
    else:
        trainer.step()
    for workspace in (trainer.workspace, trainer.ring):
        status = B.get_status(workspace)
        if status != B.Status.OK:
            raise RuntimeError(f"the training step reported {status.name}")
    names = ("embed", "wqkv", "wo", "head", "wq", "wk")
    weights = {k: getattr(model, k).double().requires_grad_() for k in names}
    y = plain_model(weights, trainer.tokens.long(), starts, trainer.positions.long(), model.cos_sin.double())
    asked = trainer.targets >= 0
    logprob = torch.where(asked, y.gather(1, trainer.targets.long().clamp(min=0)[:, None])[:, 0], 0.0)
    want = torch.autograd.grad((logprob * trainer.grad.double()).sum(), [weights[k] for k in names])
    off = {k: float((trainer.grads[k].double() - w).norm() / w.norm()) for k, w in zip(names, want)}
    return float((trainer.logprob.double() - logprob.detach()).abs().max()), off


def run(ranks=8, requests=6, steps=20, dtype=torch.float32, check=True, prompts=None):
    """Decodes `steps` tokens, behind the prompts if there are any; with check, returns the largest difference of the top
    alternatives' log probabilities from the plain form's."""
    model = Model(ranks, dtype)
    decoder = Decoder(model, requests)
    start = (decoder.lens, decoder.free_count, decoder.tokens, decoder.table)
    kept = [t.clone() for t in start]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        decoder.step()  # library handles and workspaces are made outside of the capture
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decoder.step()
    for t, old in zip(start, kept):
        t.copy_(old)
    worst, keys, values = 0.0, [], []
    texts = [list(p) for p in prompts] if prompts else None

    def compare_texts():
        """The last words' log probabilities of the texts so far, a text at a time."""
        weights = {k: getattr(model, k).double() for k in ("embed", "wqkv", "wo", "head", "wq", "wk")}
        off = 0.0
        for i, text in enumerate(texts):
            at = torch.tensor(text, device="cuda")
            y = plain_model(weights, at, [0, len(text)], torch.arange(len(text), device="cuda"), model.cos_sin.double())[-1]
            off = max(off, float((decoder.top_values[i].double() - y[decoder.top_ids[i].long()]).abs().max()),
                      float(y.max() - y[decoder.top_ids[i, 0].long()]),
                      abs(float(decoder.entropy[i].double() + (y.exp() * y).sum())))
        return off

    if prompts:
        decoder.prefill(prompts)
        worst = compare_texts()
    for position in range(steps):
        before = decoder.tokens.clone()
        graph.replay()
        if check and texts:
            for text, word in zip(texts, before.tolist()):
                text.append(word)
            worst = max(worst, compare_texts())
        elif check:
            y = plain_step(model, keys, values, before, position)
            at = decoder.top_ids.long()
            worst = max(worst, float((decoder.top_values.double() - y.gather(1, at)).abs().max()))
            best = y.amax(1)
            worst = max(worst, float((best - y.gather(1, at[:, :1])[:, 0]).max()))
            worst = max(worst, float((decoder.entropy.double() + (y.exp() * y).sum(1)).abs().max()))
    status = B.get_status(decoder.workspace)
    if status != B.Status.OK:
        raise RuntimeError(f"the operators reported {status.name}")
    decoder.backward()
    torch.cuda.synchronize()
    return decoder, worst


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--prompt", type=int, default=0, help="tokens of the longest prompt")
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    dtype = torch.float32 if a.dtype == "f32" else torch.bfloat16
    prompts = [[(7 * i + 3 * r) % (a.ranks * WORDS) for i in range(max(1, a.prompt * (r + 1) // a.requests))]
               for r in range(a.requests)] if a.prompt else None
    decoder, worst = run(a.ranks, a.requests, a.steps, dtype, prompts=prompts)
    print("tokens", decoder.tokens.tolist())
    print("log probabilities", [round(float(v), 4) for v in decoder.top_values[:, 0]])
    print("largest difference from 64 bits", worst)
    print("training step, gradients' differences from 64 bits", train(a.ranks, dtype=dtype))


if __name__ == "__main__":
    main()
