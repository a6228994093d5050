"""A decode step as a model makes it: the queries and keys of a fused projection normed and turned in place, the cache
written, attention over it, a mixture of experts, logits and a drawn token, eager and as one captured graph, each stage
against its definition in 64 bits on what the stage before gave."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from step_helpers import Experts, rope_ref, sample_ref  # noqa: E402

from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_q8_cache  # noqa: E402

pytestmark = pytest.mark.gpu

S, HQ, HK, D, PAGE, VOCAB = 5, 6, 2, 64, 16, 1000
LENS = [1, 17, 40, 64, 9]


class Step:
    def __init__(self):
        r = self.rng = np.random.default_rng(31)
        pages = sum(-(-(n + 3) // PAGE) for n in LENS)
        table = np.full((S, 5), -1, np.int32)
        order = iter(r.permutation(pages))
        for s, n in enumerate(LENS):
            for j in range(-(-(n + 3) // PAGE)):
                table[s, j] = next(order)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.cache = mnb.KVCache.empty(pages, PAGE, HK, D)
        self.kv_len = dev(np.int32(LENS))
        self.table = dev(table)
        one = dev(np.arange(S + 1, dtype=np.int32))
        self.batch = mnb.KVBatch(self.table, self.kv_len, one, S, 1, max(LENS) + 3)
        self.freq = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
        self.gains = [r.uniform(0.5, 1.5, D).astype(np.float16) for _ in range(2)]
        self.rope = mnb.Rope(D, dev(self.freq), q_weight=dev(self.gains[0]), k_weight=dev(self.gains[1]))
        self.experts = Experts(32, HQ * D, 160, 6, 4, True)
        self.layer = self.experts.layer(torch, mnb, 2, True)
        self.moe_ws = mnb.moe_workspace(self.layer, S)
        self.head = dev((r.standard_normal((VOCAB, HQ * D)) * 0.2).astype(np.float16))
        self.qkv = torch.empty(S, (HQ + 2 * HK) * D, dtype=torch.float16, device="cuda")
        self.att, self.y = (torch.empty(S, HQ * D, dtype=torch.float16, device="cuda") for _ in range(2))
        self.u, self.temperature, self.top_p = (torch.empty(S, device="cuda") for _ in range(3))
        self.token, self.logp = torch.empty(S, dtype=torch.int64, device="cuda"), torch.empty(S, device="cuda")
        self.logits = torch.empty(S, VOCAB, dtype=torch.float16, device="cuda")
        # what is cached already
        old = [n - 1 for n in LENS]
        before = mnb.KVBatch(self.table, dev(np.int32(old)), dev(np.concatenate([[0], np.cumsum(old)]).astype(np.int32)),
                             sum(old), max(old), max(LENS))
        k, v = (dev(r.standard_normal((sum(old), HK, D)).astype(np.float16)) for _ in range(2))
        mnb.mnb_kv_write(self.cache, before, k, v)
        self.ws = mnb.attn_workspace(self.cache, self.batch, HQ)

    def inputs(self, seed):
        r = np.random.default_rng(seed)
        self.raw = r.standard_normal(tuple(self.qkv.shape)).astype(np.float16)
        self.us = r.uniform(0, 1, S).astype(np.float32)
        self.ts = np.float32([0.0, 0.7, 1.0, 1.3, 0.9])
        self.ps = np.float32([1.0, 0.9, 0.5, 1.0, 0.99])
        for dst, src in ((self.qkv, self.raw), (self.u, self.us), (self.temperature, self.ts), (self.top_p, self.ps)):
            dst.copy_(torch.from_numpy(src))

    def run(self):
        q, k = HQ * D, HK * D
        mnb.mnb_qk_rope(self.rope, self.batch, self.qkv[:, :q], self.qkv[:, q:q + k])
        mnb.mnb_kv_write(self.cache, self.batch, self.qkv[:, q:q + k], self.qkv[:, q + k:])
        mnb.mnb_attn(self.cache, self.batch, self.qkv[:, :q], self.att, ws=self.ws)
        mnb.mnb_moe(self.layer, self.att, self.y, ws=self.moe_ws)
        torch.mm(self.y, self.head.t(), out=self.logits)
        mnb.mnb_sample(self.logits, self.u, self.token, self.logp, self.temperature, top_p=self.top_p)

    def check(self):
        torch.cuda.synchronize()
        lens = self.kv_len.cpu().numpy()
        qkv = self.qkv.cpu().numpy()
        for lo, heads, gain in ((0, HQ, self.gains[0]), (HQ * D, HK, self.gains[1])):
            want, tol = rope_ref(self.raw[:, lo:lo + heads * D].reshape(S, heads, D), lens - 1, self.freq, False, gain)
            assert np.all(np.abs(qkv[:, lo:lo + heads * D].reshape(S, heads, D) - want) <= tol)
        assert np.array_equal(qkv[:, (HQ + HK) * D:], self.raw[:, (HQ + HK) * D:])
        # attention over what the cache holds now; its own tests have the tolerance of a row
        total = int(lens.sum())
        start = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        k, v = (torch.empty(total, HK, D, dtype=torch.float16, device="cuda") for _ in range(2))
        mnb.mnb_kv_read(self.cache, mnb.KVBatch(self.table, self.kv_len, start, total, int(lens.max()), int(lens.max())), k, v)
        k, v, att = (x.cpu().numpy().astype(np.float64) for x in (k, v, self.att))
        at = 0
        for s, n in enumerate(lens):
            for h in range(HQ):
                kk, vv = k[at:at + n, h // (HQ // HK)], v[at:at + n, h // (HQ // HK)]
                x = kk @ qkv[s, h * D:(h + 1) * D].astype(np.float64) / D ** 0.5
                w = np.exp(x - x.max())
                # probabilities and result in FP16, values read back in FP16, the scores' 2^-11 of each key
                tol = 4 * 2.0 ** -11 * (1 + np.abs(x).max()) * np.abs(vv).max()
                assert np.all(np.abs(att[s, h * D:(h + 1) * D] - w @ vv / w.sum()) <= tol)
            at += n
        want = self.experts.ref(self.att.cpu().numpy(), 2, True)
        assert np.all(np.abs(self.y.cpu().numpy() - want[2]) <= want[3])
        logits = self.logits.cpu().numpy()
        for s in range(S):
            token, logp = sample_ref(logits[s], self.us[s], self.ts[s], 0, self.ps[s])
            assert int(self.token[s]) == token and abs(float(self.logp[s]) - logp) <= 2.0 ** -18


def test_the_stages_of_a_step_eager_and_captured():
    st = Step()
    st.inputs(1)
    st.run()
    st.check()
    st.kv_len.add_(1)
    st.inputs(2)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        st.run()
    graph.replay()
    st.check()
    tokens = st.token.clone()
    st.kv_len.add_(1)  # the next step of the same graph
    st.inputs(3)
    graph.replay()
    st.check()
    st.kv_len.sub_(1)  # and the one before again: the cache takes the same tokens at the same places
    st.inputs(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(st.token, tokens)


@pytest.mark.parametrize("kw", [dict(experts=4), dict(temperature=0.8, top_p=0.9), dict(experts=3, temperature=1.1)])
def test_the_example_with_experts_and_drawn_tokens(kw):
    # as the example's own test: the step by step and the one-pass log probabilities of the same tokens; a text whose
    # experts' logits lie close may take another one in the two passes, so only most tokens are held to agree
    sizes = dict(hidden=256, q_heads=4, kv_heads=1, head_dim=128, mlp=256, vocab=1000)
    tokens, logps, apart, ms, entropy = decode_q8_cache.run(layers=2, steps=40, prompt_lens=(1, 50, 37, 16), **sizes, **kw)
    assert tokens.shape == (40, 4) and tokens.min() >= 0 and tokens.max() < 1000 and ms > 0
    assert torch.all(torch.isfinite(logps)) and torch.all(logps < 0)
    assert apart.abs().median().item() < 0.25


def test_calls_on_two_streams_at_once():
    r = np.random.default_rng(77)
    ex = Experts(78, 512, 256, 16, 4, True)
    layer = ex.layer(torch, mnb, 4, True)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    rope = mnb.Rope(64, dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)))

    class Lane:
        def __init__(self, tokens):
            self.x, self.y = dev(r.standard_normal((tokens, 512)).astype(np.float16)), None
            self.pos = torch.arange(tokens, dtype=torch.int32, device="cuda") * 1000
            self.turned, self.y = torch.empty(tokens, 8, 64, dtype=torch.float16, device="cuda"), torch.empty_like(self.x)
            self.ws = mnb.moe_workspace(layer, tokens)
            self.logits = dev((r.standard_normal((tokens, 40003)) * 2).astype(np.float16))
            self.u, self.p = (dev(r.uniform(0, 1, tokens).astype(np.float32)) for _ in range(2))
            self.token = torch.empty(tokens, dtype=torch.int64, device="cuda")

        def run(self):
            mnb.mnb_qk_rope(rope, self.pos, self.x.view(-1, 8, 64), Q_out=self.turned)
            mnb.mnb_moe(layer, self.turned.view(-1, 512), self.y, ws=self.ws)
            mnb.mnb_sample(self.logits, self.u, self.token, top_p=self.p)
            return self.turned, self.y, self.token

    lanes = [Lane(3), Lane(16)]
    torch.cuda.synchronize()
    want = [[t.clone() for t in lane.run()] for lane in lanes]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lanes]
    for _ in range(20):
        for lane, s in zip(lanes, streams):
            for t in (lane.turned, lane.y):
                t.zero_()
        torch.cuda.synchronize()
        for lane, s in zip(lanes, streams):
            with torch.cuda.stream(s):
                lane.run()
        torch.cuda.synchronize()
        for lane, w in zip(lanes, want):
            assert all(torch.equal(a, b) for a, b in zip((lane.turned, lane.y, lane.token), w))
