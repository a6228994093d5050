"""Cases of the 8-bit key/value cache, the attention that reads it and the token log
probabilities, and what one pass of each computes.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or,
where ``own`` is true, by the library's calls of ``block_quantized_matmul_matmulnbits_gb300.mnb``.

The cache: uint8 codes [pages, kv_heads, page, head_dim] for keys and for values, one FP32 scale
for each block of 16 tokens of a page and head; a code q stands for (q - 128) * scale.  A batch of
sequences names its pages in ``table`` [seqs, max_pages]; sequence s holds ``kv_len[s]`` tokens,
the last ``q_start[s + 1] - q_start[s]`` of which are the tokens of this call.
"""
import math
import random

import torch

own = False

BLOCK = 16  # tokens that share a scale
KINDS = ("kv_write", "kv_read", "attn", "logprobs")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token of one sequence enters the cache of a small model's layer (K = 576: 3 heads of 64)
        dict(name="kv_write_one_token", op="kv_write", seqs=1, new=1, ctx=100, kv_heads=3, head_dim=64, page=16),
        # one decode step of a server's batch: 127 sequences of uneven length and an idle slot
        dict(name="kv_write_batch_step", op="kv_write", seqs=128, new=1, ctx=4000, kv_heads=8, head_dim=128, page=64),
        # uneven prompts appended behind cached prefixes that end inside a block
        dict(name="kv_write_prompts", op="kv_write", seqs=4, new=6001, ctx=777, kv_heads=8, head_dim=128, page=32),
        # a short prefix taken back in FP16
        dict(name="kv_read_short", op="kv_read", seqs=3, new=700, ctx=0, kv_heads=2, head_dim=64, page=16),
        # long uneven prefixes taken back in FP16, to move or recompute them
        dict(name="kv_read_long", op="kv_read", seqs=12, new=16384, ctx=0, kv_heads=8, head_dim=128, page=64),
        # one generated token of a small model (9 query heads on 3): the latency of a call
        dict(name="attn_one_token", op="attn", seqs=1, new=1, ctx=576, q_heads=9, kv_heads=3, head_dim=64, page=16,
             window=0),
        # one decode step of a server's batch: 63 uneven sequences and an idle slot
        dict(name="attn_batch_step", op="attn", seqs=64, new=1, ctx=8191, q_heads=32, kv_heads=8, head_dim=128,
             page=64, window=0),
        # one decode step over long contexts: few rows, a long axis
        dict(name="attn_long_step", op="attn", seqs=3, new=1, ctx=131070, q_heads=32, kv_heads=8, head_dim=128,
             page=128, window=0),
        # five drafted tokens a sequence are checked at once (14 query heads on 2)
        dict(name="attn_five_tokens", op="attn", seqs=16, new=5, ctx=4001, q_heads=14, kv_heads=2, head_dim=64,
             page=32, window=0),
        # prompts of uneven length behind cached prefixes: a contraction
        dict(name="attn_prompts", op="attn", seqs=2, new=4096, ctx=4096, q_heads=32, kv_heads=8, head_dim=128,
             page=64, window=0),
        # one sampled token of a small model's vocabulary, with five alternatives
        dict(name="logprobs_one_token", op="logprobs", rows=1, vocab=49152, top=5),
        # a prompt scored over a large vocabulary, with twenty alternatives a token
        dict(name="logprobs_prompt", op="logprobs", rows=512, vocab=151936, top=20),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.9e15)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def heads():
        group = rng.choice((1, 2, 3, 4, 5, 7, 8))
        kv = rng.choice((1, 2, 3, 4, 8))
        return dict(q_heads=group * kv, kv_heads=kv, head_dim=rng.choice((64, 128)))

    while True:
        op = rng.choice(KINDS)
        if op == "logprobs":
            case = dict(op=op, rows=log(1, 512), vocab=log(2000, 152000), top=rng.randint(0, 20))
        elif op == "attn":
            step = rng.random()
            if step < 0.5:  # decode
                case = dict(op=op, seqs=log(1, 128), new=1, ctx=log(16, 131070))
            elif step < 0.7:  # a few tokens a sequence
                case = dict(op=op, seqs=log(1, 32), new=rng.randint(2, 9), ctx=log(16, 16000))
            else:  # prompts
                case = dict(op=op, seqs=rng.randint(1, 4), new=log(33, 4096), ctx=log(1, 8192))
            case.update(heads(), page=rng.choice((16, 32, 64, 128)), window=rng.choice((0, 0, 0, log(64, 4096))))
        else:
            h = heads()
            case = dict(op=op, kv_heads=h["kv_heads"], head_dim=h["head_dim"], page=rng.choice((16, 32, 64, 128)))
            if op == "kv_read":
                case.update(seqs=log(1, 12), new=log(32, 16384), ctx=0)
            elif rng.random() < 0.5:
                case.update(seqs=log(1, 256), new=1, ctx=log(1, 4000))
            else:
                case.update(seqs=log(1, 4), new=log(2, 6001), ctx=log(1, 4000))
        same = [c for c in listed() if c["op"] == op]
        if _cost(case) <= max(_cost(c) for c in same) and _padded(case) <= max(_padded(c) for c in same):
            return case


def _padded(case):
    """Sequences as long as the longest one: what the plain form holds."""
    if case["op"] == "logprobs":
        return case["rows"] * case["vocab"]
    return case["seqs"] * (case["ctx"] + case["new"]) * case["kv_heads"] * case["head_dim"]


def _lengths(case):
    """(new, before) of each sequence, from the case alone: the first one as long as the case says, the
    others uneven, and with four sequences or more the last one idle."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    uneven = lambda most: max(1, int(round(most ** rng.uniform(0.6, 1.0))))  # noqa: E731
    S = case["seqs"]
    new = [case["new"]] + [uneven(case["new"]) for _ in range(S - 1)]
    old = [case["ctx"]] + [uneven(case["ctx"]) if case["ctx"] else 0 for _ in range(S - 1)]
    if S >= 4:
        new[-1] = old[-1] = 0
    return new, old


def _keys_seen(n, before, window):
    """Keys that the n tokens behind `before` others attend to, added up, and the distinct ones."""
    if not window:
        return n * before + n * (n + 1) // 2, (before + n if n else 0)
    full = min(n, max(0, window - before - 1))  # tokens that see everything before them
    seen = full * before + full * (full + 1) // 2 + (n - full) * window
    return seen, (min(before + n, n + window - 1) if n else 0)


def work(case):
    if case["op"] == "logprobs":
        R, V, k = case["rows"], case["vocab"], case["top"]
        return dict(bytes=2 * R * V + 8 * R + 8 * R + 8 * R * k, flops=5 * R * V)
    new, old = _lengths(case)
    H, D = case["kv_heads"], case["head_dim"]
    T = sum(new)
    token = H * (2 * D + 8 / BLOCK)  # codes and scales of one token's keys and values
    if case["op"] == "kv_read":
        return dict(bytes=T * token + T * H * D * 4, flops=2 * T * H * D * 2)
    if case["op"] == "kv_write":  # read the tokens and the touched blocks' cached ones, write codes; then read them back
        back = sum(n + b % BLOCK for n, b in zip(new, old) if n)
        return dict(bytes=T * H * D * 4 + T * token + back * token + back * H * D * 4, flops=6 * T * H * D * 2)
    seen = [_keys_seen(n, b, case["window"]) for n, b in zip(new, old)]
    return dict(bytes=4 * T * case["q_heads"] * D + sum(d for _, d in seen) * token,
                flops=4 * D * case["q_heads"] * sum(s for s, _ in seen))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 11)
    st = dict(case)
    if case["op"] == "logprobs":
        # logits of a trained head: a wide bulk and a few likely tokens a row
        R, V = case["rows"], case["vocab"]
        x = torch.randn(R, V, device=dev, generator=g, dtype=torch.float16) * 2.5
        likely = torch.randint(0, V, (R, 40), device=dev, generator=g)
        x.scatter_add_(1, likely, torch.rand(R, 40, device=dev, generator=g).half() * 14)
        st.update(logits=x, target=likely[:, 0].contiguous(), scale=1 / 0.8)
        return st
    new, old = _lengths(case)
    S, P, H, D = case["seqs"], case["page"], case["kv_heads"], case["head_dim"]
    lens = [n + b for n, b in zip(new, old)]
    need = [-(-n // P) for n in lens]
    pages = sum(need) + 1  # the last page belongs to no sequence
    order = torch.randperm(pages - 1, device=dev, generator=g).to(torch.int32)
    table = torch.full((S, max(max(need), 1)), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n

    def codes():
        c = torch.empty(pages, H, P, D, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (H * P * D))
        for a in range(0, pages, step):
            part = c[a:a + step]
            part.copy_((torch.randn(part.shape, device=dev, generator=g, dtype=torch.float16) * 34).round_()
                       .clamp_(-127, 127).add_(128))
        return c

    start = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    scales = lambda: torch.rand(pages, H, P // BLOCK, device=dev, generator=g) * 0.02 + 0.02  # noqa: E731
    T = sum(new)
    st.update(table=table, kv_len=torch.tensor(lens, dtype=torch.int32, device=dev), q_start=start, tokens=T,
              max_new=max(new), max_len=max(lens), k_codes=codes(), v_codes=codes(), k_scales=scales(),
              v_scales=scales())
    if case["op"] == "attn":
        st["q"] = torch.randn(T, case["q_heads"], D, device=dev, generator=g, dtype=torch.float16)
        st["scale"] = D ** -0.5
    if case["op"] == "kv_write":
        # keys with a few strong channels; what was cached stays in its blocks
        st["k"] = torch.randn(T, H, D, device=dev, generator=g, dtype=torch.float16)
        st["k"][:, :, ::32] *= 3
        st["v"] = torch.randn(T, H, D, device=dev, generator=g, dtype=torch.float16)
        # the tokens of every block that the write touches, to read them back
        back = [n + b % BLOCK if n else 0 for n, b in zip(new, old)]
        st["back_start"] = torch.tensor([0] + back, device=dev).cumsum(0).to(torch.int32)
        st["back"], st["max_back"] = sum(back), max(back)
    return st


# ------------------------------------------------------------------ plain forms

def _plain_write_one(st, x, codes, scales, page, inner, fresh, kept, tok):
    """Quantises the tokens of x into the blocks (page, inner): [S, NB] blocks, `fresh` and `kept` [S, NB, 16]."""
    pages, H, P, D = codes.shape
    blocks = codes.view(pages, H, P // BLOCK, BLOCK, D)
    was = blocks[page, :, inner]                                     # [S, NB, H, 16, D]
    s_was = scales[page, :, inner]                                   # [S, NB, H]
    v = x[tok].permute(0, 1, 3, 2, 4).float()
    is_new = fresh[:, :, None, :, None]
    s = torch.where(is_new, v.abs(), torch.zeros_like(v)).amax((-1, -2)) / 127
    has_old = kept.any(-1)[:, :, None]
    s = torch.where(has_old, torch.maximum(s, s_was), s)
    s = torch.where(fresh.any(-1)[:, :, None], s, s_was)
    good = (s > 0) & (s < math.inf)
    one = torch.ones_like(s)
    inv = (1 / torch.where(good, s, one))[..., None, None]
    ratio = (s_was / torch.where(good, s, one))[..., None, None]
    good = good[..., None, None]
    zero = torch.zeros_like(v)
    q = torch.where(good, (v * inv).round().clamp(-127, 127), zero) + 128
    again = torch.where(good, ((was.float() - 128) * ratio).round().clamp(-127, 127), zero) + 128
    again = torch.where(kept[:, :, None, :, None], again, was.float())
    blocks[page, :, inner] = torch.where(is_new, q, again).to(torch.uint8)
    scales[page, :, inner] = s


def _plain_write(st):
    P, S = st["page"], st["seqs"]
    dev = st["table"].device
    n = (st["q_start"][1:] - st["q_start"][:-1])[:, None]
    kv = st["kv_len"][:, None]
    first = kv - n
    b = first // BLOCK + torch.arange((st["max_new"] + BLOCK - 2) // BLOCK + 1, device=dev)
    valid = (b * BLOCK < kv) & (n > 0)
    page = torch.gather(st["table"], 1, (b * BLOCK // P).clamp(max=st["table"].shape[1] - 1).long()).long()
    page = torch.where(valid, page, -1)                               # the page that belongs to no sequence
    inner = torch.where(valid, b * BLOCK % P // BLOCK, 0).long()
    pos = b[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)
    fresh = valid[:, :, None] & (pos >= first[:, :, None]) & (pos < kv[:, :, None])
    kept = valid[:, :, None] & (pos < first[:, :, None])
    tok = (st["q_start"][:-1, None, None] + pos - first[:, :, None]).clamp(0, st["tokens"] - 1).long()
    for name in ("k", "v"):
        _plain_write_one(st, st[name], st[name + "_codes"], st[name + "_scales"], page, inner, fresh, kept, tok)


def _places(st, start, T):
    """Sequence, position, page and row in the page of each of T tokens."""
    t = torch.arange(T, dtype=torch.int32, device=start.device)
    seq = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pos = st["kv_len"][seq] - start[seq + 1] + t
    return seq, pos, st["table"][seq, (pos // st["page"]).long()].long(), (pos % st["page"]).long()


def _plain_read(st, start, T):
    seq, pos, page, row = _places(st, start, T)
    return [((st[c + "_codes"][page, :, row].float() - 128) * st[c + "_scales"][page, :, row // BLOCK][..., None]).half()
            for c in ("k", "v")]


def _plain_attn(st):
    S, H, D, P, N, L = st["seqs"], st["kv_heads"], st["head_dim"], st["page"], st["max_new"], st["max_len"]
    G = st["q_heads"] // H
    dev = st["q"].device
    at = torch.arange(L, device=dev)
    page = st["table"][:, at // P].long()                             # [S, L]; -1 is the page of no sequence
    row = (at % P)[None]

    def dequantised(c):                                               # [S, H, L, D]
        x = st[c + "_codes"][page, :, row].float().sub_(128)
        return x.mul_(st[c + "_scales"][page, :, row // BLOCK][..., None]).transpose(1, 2)

    n = st["q_start"][1:] - st["q_start"][:-1]
    i = torch.arange(N, device=dev)
    tok = (st["q_start"][:-1, None] + i).clamp(max=max(st["tokens"] - 1, 0)).long()
    q = st["q"][tok].float().view(S, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * N, D)
    qpos = (st["kv_len"] - n)[:, None] + i                            # [S, N]
    sees = at[None, None, :] <= qpos[:, :, None]
    if st["window"]:
        sees &= at[None, None, :] > qpos[:, :, None] - st["window"]
    s = torch.matmul(q, dequantised("k").transpose(2, 3)).mul_(st["scale"]).view(S, H, G, N, L)
    s.masked_fill_(~sees[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, H, G * N, L), dequantised("v")).view(S, H, G, N, D)
    o = (o / torch.where(den == 0, 1.0, den)).permute(0, 3, 1, 2, 4).reshape(S, N, H * G, D)
    t = torch.arange(st["tokens"], dtype=torch.int32, device=dev)
    seq = torch.searchsorted(st["q_start"][1:].contiguous(), t, right=True)
    return o[seq, (t - st["q_start"][seq]).long()].half()


def _plain_logprobs(st):
    x = st["logits"].float() * st["scale"]
    top = x.amax(-1, keepdim=True)
    y = x - top
    e = y.exp()
    z = e.sum(-1, keepdim=True)
    logp = y - z.log()
    entropy = z.log()[:, 0] - (e * torch.where(e > 0, y, 0.0)).sum(-1) / z[:, 0]
    best, ids = torch.sort(logp, dim=-1, descending=True, stable=True)
    k = st["top"]
    return dict(logprob=logp.gather(1, st["target"][:, None])[:, 0], entropy=entropy,
                top_ids=ids[:, :k].to(torch.int32), top_logprobs=best[:, :k].contiguous())


# ------------------------------------------------------------------ the library's calls

def _own_state(st):
    """What a program makes once and keeps: the cache's and the batches' handles, outputs, workspaces."""
    from block_quantized_matmul_matmulnbits_gb300 import mnb
    half, dev = torch.float16, torch.device("cuda")
    if st["op"] == "logprobs":
        R, k = st["rows"], st["top"]
        return dict(mnb=mnb, logprob=torch.empty(R, device=dev), entropy=torch.empty(R, device=dev),
                    top_ids=torch.empty(R, k, dtype=torch.int32, device=dev),
                    top_logprobs=torch.empty(R, k, device=dev))
    cache = mnb.KVCache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"])
    batch = mnb.KVBatch(st["table"], st["kv_len"], st["q_start"], st["tokens"], st["max_new"], st["max_len"])
    kept = dict(mnb=mnb, cache=cache, batch=batch)
    if st["op"] == "attn":
        kept.update(out=torch.empty_like(st["q"]), ws=mnb.attn_workspace(cache, batch, st["q_heads"], st["window"]))
    else:
        T, start, most = ((st["back"], st["back_start"], st["max_back"]) if st["op"] == "kv_write" else
                          (st["tokens"], st["q_start"], st["max_new"]))
        kept["back"] = mnb.KVBatch(st["table"], st["kv_len"], start, T, most, st["max_len"])
        kept["k"], kept["v"] = (torch.empty(T, st["kv_heads"], st["head_dim"], dtype=half, device=dev)
                                for _ in range(2))
    return kept


def _own(st):
    h = st.get("kept")
    if h is None:
        h = st["kept"] = _own_state(st)
    mnb = h["mnb"]
    if st["op"] == "logprobs":
        mnb.mnb_logprobs(st["logits"], st["target"], h["logprob"], h["entropy"], h["top_ids"], h["top_logprobs"],
                         scale=st["scale"])
        return {name: h[name] for name in ("logprob", "entropy", "top_ids", "top_logprobs")}
    if st["op"] == "attn":
        mnb.mnb_attn(h["cache"], h["batch"], st["q"], h["out"], scale=st["scale"], window=st["window"], ws=h["ws"])
        return h["out"]
    if st["op"] == "kv_write":
        mnb.mnb_kv_write(h["cache"], h["batch"], st["k"], st["v"])
    mnb.mnb_kv_read(h["cache"], h["back"], h["k"], h["v"])
    if st["op"] == "kv_read":
        return dict(k=h["k"], v=h["v"])
    return dict(k=h["k"], v=h["v"], k_scales=st["k_scales"], v_scales=st["v_scales"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "attn":
        return _plain_attn(state)
    if op == "kv_read":
        k, v = _plain_read(state, state["q_start"], state["tokens"])
        return dict(k=k, v=v)
    _plain_write(state)  # what the write changed comes back as the values that its codes stand for
    k, v = _plain_read(state, state["back_start"], state["back"])
    return dict(k=k, v=v, k_scales=state["k_scales"], v_scales=state["v_scales"])


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        R, k = case["rows"], case["top"]
        logprob, entropy, tops = [], [], []
        for r in range(R):
            x = st["logits"][r].double() * st["scale"]
            lse = torch.logsumexp(x, 0)
            p = torch.softmax(x, 0)
            logprob.append(x[st["target"][r]] - lse)
            entropy.append(-(p * torch.log_softmax(x, 0)).sum())
            tops.append(torch.sort(x, descending=True).values[:k] - lse)
        return dict(logprob=torch.stack(logprob), entropy=torch.stack(entropy), top_ids=None,
                    top_logprobs=torch.stack(tops))
    P, H, D = case["page"], case["kv_heads"], case["head_dim"]
    lens, starts = st["kv_len"].tolist(), st["q_start"].tolist()

    def cached(name, s):
        """[tokens, H, D] of sequence s: codes less 128, and each token's scale [tokens, H]."""
        use = st["table"][s, :-(-lens[s] // P)].long()
        c = st[name + "_codes"][use].permute(0, 2, 1, 3).reshape(-1, H, D)[:lens[s]]
        f = st[name + "_scales"][use].permute(0, 2, 1).reshape(-1, H).repeat_interleave(BLOCK, 0)[:lens[s]]
        return c.double() - 128, f.double()

    if case["op"] == "kv_read":
        got = {"k": [], "v": []}
        for s in range(case["seqs"]):
            for name in got:
                c, f = cached(name, s)
                got[name].append(c * f[..., None])
        return {name: torch.cat(v) for name, v in got.items()}
    if case["op"] == "kv_write":
        got = dict(k=[], v=[], k_scales=st["k_scales"].double(), v_scales=st["v_scales"].double())
        for s in range(case["seqs"]):
            n = starts[s + 1] - starts[s]
            if not n:
                continue
            before = lens[s] - n
            for name in ("k", "v"):
                c, f = cached(name, s)
                x = st[name][starts[s]:starts[s + 1]].double()
                lo = before // BLOCK * BLOCK
                blocks = -(-(lens[s] - lo) // BLOCK)
                pad = torch.zeros(blocks * BLOCK, H, D, dtype=torch.float64, device=x.device)
                pad[before - lo:before - lo + n] = x
                s_new = pad.view(blocks, BLOCK, H, D).abs().amax((1, 3)) / 127
                if before > lo:
                    s_new[0] = torch.maximum(s_new[0], f[lo])
                each = s_new.repeat_interleave(BLOCK, 0)[:, :, None]
                q = torch.round(pad / each).clamp(-127, 127)
                if before > lo:
                    q[:before - lo] = torch.round(c[lo:before] * (f[lo] / s_new[0])[None, :, None])
                got[name].append((q * each)[:lens[s] - lo])
                at = torch.arange(lo, lens[s], BLOCK, device=x.device)
                got[name + "_scales"][st["table"][s, at // P].long(), :, at % P // BLOCK] = s_new
        got["k"], got["v"] = torch.cat(got["k"]), torch.cat(got["v"])
        return got
    G = case["q_heads"] // H
    out = torch.zeros(st["tokens"], case["q_heads"], D, dtype=torch.float64, device=st["q"].device)
    for s in range(case["seqs"]):
        n = starts[s + 1] - starts[s]
        if not n:
            continue
        kc, kf = cached("k", s)
        vc, vf = cached("v", s)
        i = torch.arange(lens[s] - n, lens[s], device=kc.device)[:, None]
        j = torch.arange(lens[s], device=kc.device)[None]
        hidden = j > i
        if case["window"]:
            hidden |= j <= i - case["window"]
        for h in range(H):
            k, v = kc[:, h] * kf[:, h, None], vc[:, h] * vf[:, h, None]
            for g in range(G):
                q = st["q"][starts[s]:starts[s + 1], h * G + g].double()
                a = (q @ k.T) * st["scale"]
                a[hidden] = -math.inf
                out[starts[s]:starts[s + 1], h * G + g] = torch.softmax(a, 1) @ v
    return out
