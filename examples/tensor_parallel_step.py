"""Steps of a small tensor-parallel language model over virtual ranks, from page
tables to the all-reduced gradient.

Each of N ranks holds some query heads, one key head and a range of the
vocabulary of a one-layer model with random weights. A step of decoding:

  page_tables          pages and cache slots of the requests' next tokens
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

Usage: python examples/tensor_parallel_step.py [--ranks 8] [--requests 6] [--steps 20]
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
        self.qkv = empty(n, r, (HEADS + 2) * DIM)
        self.q, self.attended = empty(n, r, HEADS, DIM), empty(n, r, HEADS, DIM)
        self.k_cache, self.v_cache = empty(n, pages, 1, PAGE, DIM), empty(n, pages, 1, PAGE, DIM)
        self.parts, self.sums = empty(n, r * HIDDEN), empty(n, r * HIDDEN)
        self.logits = empty(n, r, WORDS)
        self.logprob, self.entropy, self.lse = (empty(r, dtype=torch.float32) for _ in range(3))
        self.top_values, self.top_ids = empty(r, 3, dtype=torch.float32), ints(r, 3)
        self.workspace = B.OpWorkspace(max(B.decode_attention_workspace_bytes(n, r, HEADS, 1, DIM),
                                           B.token_logprobs_workspace_bytes(r, 3),
                                           B.qk_norm_rope_workspace_bytes(n, DIM)))

    def step(self):
        m, r, n = self.model, self.requests, self.model.ranks
        B.page_tables(self.lens, self.new, self.free, self.free_count, self.table, PAGE, self.pages, self.lens_out,
                      self.starts, self.positions, self.slots, self.free_out, self.workspace)
        x = m.embed.index_select(0, self.tokens)
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


def run(ranks=8, requests=6, steps=20, dtype=torch.float32, check=True):
    """Decodes `steps` tokens; with check, returns the largest difference of the top alternatives' log probabilities from
    the plain form's."""
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
    for position in range(steps):
        before = decoder.tokens.clone()
        graph.replay()
        if check:
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
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    decoder, worst = run(a.ranks, a.requests, a.steps, torch.float32 if a.dtype == "f32" else torch.bfloat16)
    print("tokens", decoder.tokens.tolist())
    print("log probabilities", [round(float(v), 4) for v in decoder.top_values[:, 0]])
    print("largest difference from 64 bits", worst)


if __name__ == "__main__":
    main()
