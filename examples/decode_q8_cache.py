"""Text from a small random-weight transformer whose every projection is a 4-bit MatMulNBits weight and whose
keys and values live in the 8-bit paged cache:

    python examples/decode_q8_cache.py [--layers 4] [--steps 64]

  1. the prompts, of different lengths, go through the model packed into one batch
     (mnb_run, mnb_kv_write, mnb_attn), and each one's last logits pick its first token;
  2. a decode step for all sequences is captured once in a CUDA graph and replayed: the cache's
     lengths, the tokens and their log probabilities (mnb_logprobs) advance on the GPU alone;
  3. the finished texts are scored in one pass over a second cache (mnb_logprobs of each next token),
     and the two sets of log probabilities are compared.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402


class Linear:
    """A 4-bit projection with random codes (1..15: none on average about the zero point 8) and one FP16 scale per
    32 inputs, outputs of unit deviation."""

    def __init__(self, n, k, gen):
        self.proj = mnb.Projection(n, k, 4, max_rank=0)
        lo, hi = (torch.randint(1, 16, (n, k // 32, 16), dtype=torch.uint8, device="cuda", generator=gen)
                  for _ in range(2))
        self.Wq = lo | hi << 4
        self.scales = (torch.rand(n, k // 32, device="cuda", generator=gen) * 0.3 + 0.85).mul_(0.2315 / k ** 0.5).half()

    def __call__(self, x):
        return self.proj(x, self.Wq, self.scales)


class Model:
    """Pre-norm layers of grouped-query attention and a gated MLP, rotary positions."""

    def __init__(self, layers=4, hidden=576, q_heads=9, kv_heads=3, head_dim=64, mlp=1536, vocab=49152, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.dim, self.vocab = hidden, q_heads, kv_heads, head_dim, vocab
        q, kv = q_heads * head_dim, kv_heads * head_dim
        self.embed = torch.randn(vocab, hidden, device="cuda", generator=gen).half()
        self.layers = [dict(qkv=Linear(q + 2 * kv, hidden, gen), out=Linear(hidden, q, gen),
                            up=Linear(2 * mlp, hidden, gen), down=Linear(hidden, mlp, gen)) for _ in range(layers)]
        self.head = Linear(vocab, hidden, gen)
        self.freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda") / head_dim)

    def caches(self, pages, page_size):
        return [mnb.KVCache.empty(pages, page_size, self.kv_heads, self.dim) for _ in self.layers]

    def workspace(self, cache, batch):
        return mnb.attn_workspace(cache, batch, self.q_heads)

    @staticmethod
    def norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).half()

    def rotate(self, x, heads, pos):
        """The first `heads` heads of x turned in place by their positions."""
        x = x[:, :heads * self.dim].unflatten(1, (heads, self.dim))
        a = (pos[:, None] * self.freq)[:, None]
        lo, hi = x.float().chunk(2, -1)
        x.copy_(torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1))

    def hidden_states(self, tokens, pos, caches, batch, ws):
        """The last layer's output for the batch's tokens, whose keys and values join the caches."""
        x = self.embed[tokens]
        q, kv = self.q_heads * self.dim, self.kv_heads * self.dim
        att = torch.empty(len(tokens), q, dtype=torch.float16, device="cuda")
        for layer, cache in zip(self.layers, caches):
            qkv = layer["qkv"](self.norm(x))  # queries, keys and values stay side by side in one row
            self.rotate(qkv, self.q_heads + self.kv_heads, pos)
            mnb.mnb_kv_write(cache, batch, qkv[:, q:q + kv], qkv[:, q + kv:])
            mnb.mnb_attn(cache, batch, qkv[:, :q], att, ws=ws)
            x = x + layer["out"](att)
            gate, up = layer["up"](self.norm(x)).chunk(2, -1)
            x = x + layer["down"]((torch.nn.functional.silu(gate) * up).contiguous())
        return self.norm(x)


def packed(lens, table, page_size):
    """Positions and KVBatch of sequences that come whole."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    return pos, mnb.KVBatch(table, i32(lens), i32(start), start[-1], max(lens), max(lens))


def generate(model, prompts, steps, page_size=16):
    """Greedy continuation of the prompts: tokens and log probabilities [steps, sequences], milliseconds a step."""
    S = len(prompts)
    lens = [len(p) for p in prompts]
    per_seq = -(-(max(lens) + steps) // page_size)
    table = torch.randperm(S * per_seq, device="cuda").to(torch.int32).view(S, per_seq)  # pages in any order
    caches = model.caches(S * per_seq, page_size)

    pos, batch = packed(lens, table, page_size)
    x = model.hidden_states(torch.cat(prompts), pos, caches, batch, model.workspace(caches[0], batch))
    logits = model.head(x[batch.q_start[1:].long() - 1])

    # the decode step: one token a sequence, everything it reads and advances lives on the GPU
    kv_len = batch.kv_len.clone()
    step = mnb.KVBatch(table, kv_len, torch.arange(S + 1, dtype=torch.int32, device="cuda"), S, 1, max(lens) + steps)
    ws = model.workspace(caches[0], step)
    top, top_lp = torch.empty(S, 1, dtype=torch.int32, device="cuda"), torch.empty(S, 1, device="cuda")
    tokens, logps = [torch.empty(steps, S, dtype=t, device="cuda") for t in (torch.int64, torch.float32)]
    at = torch.zeros(1, dtype=torch.int64, device="cuda")

    def pick(logits):
        mnb.mnb_logprobs(logits, top_ids=top, top_logprobs=top_lp)
        tokens.index_copy_(0, at, top.view(1, S).long())
        logps.index_copy_(0, at, top_lp.view(1, S))
        at.add_(1)

    def advance():
        kv_len.add_(1)
        pick(model.head(model.hidden_states(top.view(S).long(), kv_len - 1, caches, step, ws)))

    pick(logits)
    if steps > 1:
        advance()
    if steps <= 2:
        return tokens, logps, 0.0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        advance()
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(steps - 2):
        graph.replay()
    torch.cuda.synchronize()
    return tokens, logps, (time.perf_counter() - begin) * 1e3 / (steps - 2)


def score(model, texts, page_size=64):
    """Log probability of each token after the first of every text, and the entropies, in one pass."""
    lens = [len(t) for t in texts]
    per_seq = -(-max(lens) // page_size)
    table = torch.arange(len(texts) * per_seq, dtype=torch.int32, device="cuda").view(len(texts), per_seq)
    caches = model.caches(len(texts) * per_seq, page_size)
    pos, batch = packed(lens, table, page_size)
    logits = model.head(model.hidden_states(torch.cat(texts), pos, caches, batch, model.workspace(caches[0], batch)))
    # a text's last row has no next token: -1 asks for none
    target = torch.cat([torch.cat((t[1:], t.new_full((1,), -1))) for t in texts])
    logp, entropy = torch.empty(len(target), device="cuda"), torch.empty(len(target), device="cuda")
    mnb.mnb_logprobs(logits, target, logp, entropy)
    return [x[:-1] for x in logp.split(lens)], [x[:-1] for x in entropy.split(lens)]


def run(layers=4, steps=64, prompt_lens=(5, 130, 37, 300), seed=0, **sizes):
    """Generate, then score: (tokens, greedy log probabilities, their difference from the scores, ms a step)."""
    model = Model(layers=layers, seed=seed, **sizes)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    prompts = [torch.randint(0, model.vocab, (n,), device="cuda", generator=gen) for n in prompt_lens]
    tokens, logps, ms = generate(model, prompts, steps)
    texts = [torch.cat((p, tokens[:, s])) for s, p in enumerate(prompts)]
    scored, entropy = score(model, texts)
    apart = torch.stack([x[-steps:] for x in scored], 1) - logps
    return tokens, logps, apart, ms, torch.cat(entropy).mean().item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    tokens, logps, apart, ms, entropy = run(args.layers, args.steps)
    print(f"{tokens.shape[1]} sequences, {tokens.shape[0]} tokens each, {ms:.3f} ms a decode step of all of them")
    print(f"mean log probability {logps.mean().item():.3f}, mean entropy of the scored texts {entropy:.3f}")
    print(f"scored in one pass against step by step: {apart.abs().max().item():.3g} apart at most")
