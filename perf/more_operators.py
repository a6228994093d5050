"""Cases of the position rotation with its norms, of mixture-of-experts layers with block-quantized weights and
of token sampling, and what one pass of each computes.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, in 64 where 32 lose what
matters) or, where ``own`` is true, by the library's calls of ``block_quantized_matmul_matmulnbits_gb300.mnb``.

qk_rope   a call's query and key heads, each divided by its root mean square and multiplied by a weight vector
          (where the model has one), the first rotary_dim values of a head turned by their token's position
moe       router logits x . r_e in 64 bits, the top_k largest experts (equal ones by rising number) with softmax
          weights over those (``normalize``) or over all experts; the sum of their gated MLPs
          down_e . (silu(gate_e . x) * (up_e . x)), weights (q - zp) * scale in blocks of 32
sample    the tokens by falling logit (equal ones by rising number) with probabilities from logit / temperature; the
          first top_k, of these the fewest whose probability reaches top_p, of these those of at least min_p times
          the largest; the first of them at which the cumulative probability passes u
"""
import math
import random

import torch

own = False

BLOCK = 32  # weights that share a scale
KINDS = ("qk_rope", "moe", "sample")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token of a small model (9 query heads on 3 of 64, no norms)
        dict(name="rope_one_token", op="qk_rope", seqs=1, new=1, ctx=576, q_heads=9, kv_heads=3, head_dim=64,
             rotary=64, interleaved=False, norm=False),
        # one decode step of a server's batch: 127 uneven sequences and an idle slot, norms of each head
        dict(name="rope_batch_step", op="qk_rope", seqs=128, new=1, ctx=8191, q_heads=32, kv_heads=8, head_dim=128,
             rotary=128, interleaved=False, norm=True),
        # uneven prompts far behind long cached prefixes: the angles of far positions
        dict(name="rope_prompts", op="qk_rope", seqs=4, new=8192, ctx=1000003, q_heads=32, kv_heads=8, head_dim=128,
             rotary=128, interleaved=False, norm=True),
        # prompts of a model that turns a quarter of each head, neighbours paired
        dict(name="rope_partial", op="qk_rope", seqs=3, new=2047, ctx=100, q_heads=14, kv_heads=2, head_dim=128,
             rotary=32, interleaved=True, norm=False),
        # one token of a small model's layer
        dict(name="moe_one_token_small", op="moe", tokens=1, hidden=576, inter=768, experts=8, top_k=2, bits=4, zp=False,
             normalize=True),
        # one token of a layer of many small experts, explicit zero points
        dict(name="moe_one_token", op="moe", tokens=1, hidden=2048, inter=1024, experts=64, top_k=8, bits=4, zp=True,
             normalize=True),
        # one decode step of a small batch over the same layer: most experts are read
        dict(name="moe_batch_step", op="moe", tokens=16, hidden=2048, inter=1024, experts=64, top_k=8, bits=4, zp=True,
             normalize=True),
        # a few tokens of a layer of few large experts in 8 bits
        dict(name="moe_large_experts", op="moe", tokens=5, hidden=4096, inter=14336, experts=8, top_k=2, bits=8,
             zp=False, normalize=False),
        # one token of a small model's vocabulary, the usual settings of a chat
        dict(name="sample_one_token", op="sample", rows=1, vocab=49152, kind="mixed"),
        # one decode step of a server's batch, every request with settings of its own
        dict(name="sample_batch_step", op="sample", rows=128, vocab=151936, kind="mixed"),
        # many rows without any limit: the whole vocabulary can be drawn
        dict(name="sample_unlimited", op="sample", rows=300, vocab=50257, kind="none"),
        # many continuations of prompts at once, a nucleus of each
        dict(name="sample_nucleus", op="sample", rows=512, vocab=151936, kind="top_p"),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.5e12, w["flops"] / 1.9e15)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(KINDS)
        if op == "sample":
            case = dict(op=op, rows=log(1, 512), vocab=log(2000, 152000),
                        kind=rng.choice(("mixed", "mixed", "none", "top_k", "top_p", "min_p", "greedy")))
        elif op == "moe":
            experts = rng.choice((4, 8, 16, 32, 60, 64, 128))
            case = dict(op=op, tokens=log(1, 16), hidden=32 * log(8, 160), inter=32 * log(8, 448), experts=experts,
                        top_k=rng.randint(1, min(8, experts)), bits=rng.choice((4, 4, 8)), zp=rng.random() < 0.5,
                        normalize=rng.random() < 0.7)
            if 3 * case["hidden"] * case["inter"] * experts * case["bits"] // 8 > 3 << 30:  # weights of one layer
                continue
        else:
            group, kv = rng.choice((1, 2, 3, 4, 5, 7, 8)), rng.choice((1, 2, 3, 4, 8))
            dim = rng.choice((64, 128))
            case = dict(op=op, q_heads=group * kv, kv_heads=kv, head_dim=dim,
                        rotary=rng.choice((dim, dim, dim // 2, dim // 4)), interleaved=rng.random() < 0.3,
                        norm=rng.random() < 0.6)
            if rng.random() < 0.5:  # decode
                case.update(seqs=log(1, 256), new=1, ctx=log(1, 1000000))
            else:
                case.update(seqs=rng.randint(1, 4), new=log(2, 8192), ctx=log(1, 1000000))
        if _cost(case) <= max(_cost(c) for c in listed() if c["op"] == op):
            return case


def _lengths(case):
    """(new, before) of each sequence, from the case alone: the first one as long as the case says, the others
    uneven, and with four sequences or more the last one idle."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    uneven = lambda most: max(1, int(round(most ** rng.uniform(0.6, 1.0))))  # noqa: E731
    S = case["seqs"]
    new = [case["new"]] + [uneven(case["new"]) for _ in range(S - 1)]
    old = [case["ctx"]] + [uneven(case["ctx"]) for _ in range(S - 1)]
    if S >= 4:
        new[-1] = old[-1] = 0
    return new, old


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return dict(bytes=2 * n + case["rows"] * 32, flops=4 * n)
    if case["op"] == "moe":
        T, K, I, E, k = (case[x] for x in ("tokens", "hidden", "inter", "experts", "top_k"))
        used = E * (1 - (1 - k / E) ** T)  # experts that some token takes, on average
        weight = case["bits"] / 8 + (3 if case["zp"] else 2) / BLOCK
        return dict(bytes=int(used * 3 * K * I * weight) + 2 * E * K + 4 * T * K + 8 * T * k,
                    flops=2 * T * (3 * K * I * k + E * K))
    T = sum(_lengths(case)[0])
    heads = case["q_heads"] + case["kv_heads"]
    return dict(bytes=4 * T * heads * case["head_dim"] + 4 * (T + case["rotary"] // 2),
                flops=7 * T * heads * case["head_dim"])


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7907 + 13)
    st = dict(case)
    if case["op"] == "sample":
        # logits of a trained head: a wide bulk and a few likely tokens a row
        R, V, kind = case["rows"], case["vocab"], case["kind"]
        x = torch.randn(R, V, device=dev, generator=g, dtype=torch.float16) * 2.5
        likely = torch.randint(0, V, (R, 40), device=dev, generator=g)
        x.scatter_add_(1, likely, torch.rand(R, 40, device=dev, generator=g).half() * 14)
        uniform = lambda lo, hi: torch.rand(R, device=dev, generator=g) * (hi - lo) + lo  # noqa: E731
        one_of = lambda *v: torch.tensor(v, device=dev)[  # noqa: E731
            torch.randint(0, len(v), (R,), device=dev, generator=g)]
        temperature, top_k, top_p, min_p = uniform(0.6, 1.2), None, None, None
        if kind in ("mixed", "top_k"):
            top_k = one_of(0, 20, 50, 200) if kind == "mixed" else one_of(1, 20, 40, 100, 1000)
            top_k = top_k.to(torch.int32)
        if kind in ("mixed", "top_p"):
            top_p = one_of(1.0, 0.8, 0.9, 0.95) if kind == "mixed" else uniform(0.7, 0.98)
        if kind in ("mixed", "min_p"):
            min_p = one_of(0.0, 0.0, 0.02, 0.05) if kind == "mixed" else uniform(0.01, 0.1)
        if kind == "greedy":
            temperature = torch.zeros(R, device=dev)
        st.update(logits=x, u=torch.rand(R, device=dev, generator=g), temperature=temperature, top_k=top_k,
                  top_p=top_p, min_p=min_p)
        return st
    if case["op"] == "moe":
        T, K, I, E, bits = (case[x] for x in ("tokens", "hidden", "inter", "experts", "bits"))

        def weight(n, k):
            # codes, scales that make outputs of unit deviation, zero points about the middle
            codes = torch.randint(0, 256, (E, n, k // BLOCK, BLOCK * bits // 8), device=dev, generator=g,
                                  dtype=torch.uint8)
            spread = (2 ** bits) / 12 ** 0.5 * k ** 0.5
            scales = (torch.rand(E, n, k // BLOCK, device=dev, generator=g) * 0.6 + 0.7).div_(spread).half()
            mid = 2 ** (bits - 1)
            zp = None
            if case["zp"]:
                zp = torch.randint(mid - mid // 4, mid + mid // 4 + 1, (E, n, k // BLOCK), device=dev, generator=g)
                zp = zp.to(torch.uint8)
            return codes, scales, zp

        st.update(x=torch.randn(T, K, device=dev, generator=g, dtype=torch.float16),
                  router=torch.randn(E, K, device=dev, generator=g, dtype=torch.float16) * (1.5 / K ** 0.5),
                  up=weight(2 * I, K), down=weight(K, I))
        return st
    new, old = _lengths(case)
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    T = sum(new)
    # queries, keys and values of a token side by side, as one projection gives them
    qkv = torch.randn(T, (Hq + 2 * Hk) * D, device=dev, generator=g, dtype=torch.float16)
    gain = lambda: (torch.rand(D, device=dev, generator=g) + 0.5).half() if case["norm"] else None  # noqa: E731
    half = case["rotary"] // 2
    freq = (1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    st.update(qkv=qkv, tokens=T, q_gain=gain(), k_gain=gain(), freq=freq, eps=1e-6,
              kv_len=i32([n + b for n, b in zip(new, old)]), q_start=i32([0] + new).cumsum(0).to(torch.int32),
              max_new=max(new), max_len=max(n + b for n, b in zip(new, old)))
    return st


# ------------------------------------------------------------------ plain forms

def _plain_rope(st):
    Hq, Hk, D, half = st["q_heads"], st["kv_heads"], st["head_dim"], st["rotary"] // 2
    t = torch.arange(st["tokens"], dtype=torch.int32, device=st["qkv"].device)
    seq = torch.searchsorted(st["q_start"][1:].contiguous(), t, right=True)
    pos = st["kv_len"][seq] - st["q_start"][seq + 1] + t
    angle = pos.double()[:, None] * st["freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x * (x.square().mean(-1, keepdim=True) + st["eps"]).rsqrt() * gain.float()
        a, b = ((x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if st["interleaved"] else
                (x[..., :half], x[..., half:2 * half]))
        first, second = a * cos - b * sin, b * cos + a * sin
        if st["interleaved"]:
            head = torch.stack((first, second), -1).flatten(-2)
        else:
            head = torch.cat((first, second), -1)
        return torch.cat((head, x[..., 2 * half:]), -1).half()

    q, k = st["qkv"][:, :Hq * D].unflatten(1, (Hq, D)), st["qkv"][:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    return dict(q=turned(q, st["q_gain"]), k=turned(k, st["k_gain"]))


def _weights(st, which, e):
    """Expert e's weights (q - zp) * scale in 32 bits, [rows, columns]."""
    codes, scales, zp = st[which]
    c = codes[e]
    if st["bits"] == 4:
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    mid = 2.0 ** (st["bits"] - 1)
    w = (c.float() - (mid if zp is None else zp[e].float()[..., None])) * scales[e].float()[..., None]
    return w.flatten(1)


def _plain_moe(st):
    x, k, I = st["x"], st["top_k"], st["inter"]
    logits = x.double() @ st["router"].double().T  # in 64 bits: which expert comes first decides the output
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    top = best[:, :1]
    e = (best - top).exp()
    den = e.sum(-1, keepdim=True) if st["normalize"] else (logits - top).exp().sum(-1, keepdim=True)
    weights = (e / den).float()
    y = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    for ex in torch.unique(ids).tolist():
        tok, slot = torch.nonzero(ids == ex, as_tuple=True)
        gu = x[tok].float() @ _weights(st, "up", ex).T
        gate, up = gu[:, :I], gu[:, I:]
        h = gate / (1 + (-gate).exp()) * up
        y.index_add_(0, tok, (h @ _weights(st, "down", ex).T) * weights[tok, slot][:, None])
    return dict(y=y.half(), ids=ids.to(torch.int32), weights=weights)


def _plain_sample(st):
    x = st["logits"].float() + 0.0  # -0 and +0 are equal
    R, V = x.shape
    dev = x.device
    T = st["temperature"].double()
    greedy = T <= 0
    srt, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    w = srt.double().sub_(srt[:, :1].double()).div_(torch.where(greedy, 1.0, T)[:, None]).exp_()
    n = torch.full((R,), V, dtype=torch.int64, device=dev)
    if st.get("top_k") is not None:
        k = st["top_k"].long()
        n = torch.where(k > 0, torch.minimum(k, n), n)
    n = torch.where(greedy, 1, n)
    cum = w.cumsum(-1)
    total = cum.gather(1, n[:, None] - 1)[:, 0]
    if st.get("top_p") is not None:
        p = st["top_p"].double()
        fewest = (cum < (p * total)[:, None]).sum(-1) + 1
        n = torch.where(p < 1, torch.minimum(n, fewest), n)
    if st.get("min_p") is not None:
        n = torch.minimum(n, (w >= st["min_p"].double()[:, None]).sum(-1).clamp(min=1))
    total = cum.gather(1, n[:, None] - 1)[:, 0]
    at = (cum <= (st["u"].double() * total)[:, None]).sum(-1)
    at = torch.minimum(at, n - 1)[:, None]
    return dict(token=ids.gather(1, at)[:, 0], logprob=(w.gather(1, at)[:, 0] / total).log().float())


# ------------------------------------------------------------------ the library's calls

def _own_state(st):
    """What a program makes once and keeps: the descriptors, outputs and workspaces."""
    from block_quantized_matmul_matmulnbits_gb300 import mnb
    dev, half = torch.device("cuda"), torch.float16
    if st["op"] == "sample":
        R = st["rows"]
        return dict(mnb=mnb, token=torch.empty(R, dtype=torch.int64, device=dev), logprob=torch.empty(R, device=dev))
    if st["op"] == "moe":
        (uw, us, uz), (dw, ds, dz) = st["up"], st["down"]
        layer = mnb.MoE(st["router"], uw, us, dw, ds, top_k=st["top_k"], bits=st["bits"], up_zp=uz, down_zp=dz,
                        normalize=st["normalize"])
        T, k = st["tokens"], st["top_k"]
        return dict(mnb=mnb, layer=layer, y=torch.empty(T, st["hidden"], dtype=half, device=dev),
                    ids=torch.empty(T, k, dtype=torch.int32, device=dev), weights=torch.empty(T, k, device=dev),
                    ws=mnb.moe_workspace(layer, T))
    Hq, Hk, D, T = st["q_heads"], st["kv_heads"], st["head_dim"], st["tokens"]
    rope = mnb.Rope(D, st["freq"], interleaved=st["interleaved"], q_weight=st["q_gain"], k_weight=st["k_gain"],
                    eps=st["eps"])
    table = torch.zeros(st["seqs"], 0, dtype=torch.int32, device=dev)
    batch = mnb.KVBatch(table, st["kv_len"], st["q_start"], T, st["max_new"], st["max_len"])
    return dict(mnb=mnb, rope=rope, batch=batch, q=torch.empty(T, Hq, D, dtype=half, device=dev),
                k=torch.empty(T, Hk, D, dtype=half, device=dev))


def _own(st):
    h = st.get("kept")
    if h is None:
        h = st["kept"] = _own_state(st)
    mnb = h["mnb"]
    if st["op"] == "sample":
        mnb.mnb_sample(st["logits"], st["u"], h["token"], h["logprob"], temperature=st["temperature"],
                       top_k=st.get("top_k"), top_p=st.get("top_p"), min_p=st.get("min_p"))
        return dict(token=h["token"], logprob=h["logprob"])
    if st["op"] == "moe":
        mnb.mnb_moe(h["layer"], st["x"], h["y"], ids=h["ids"], weights=h["weights"], ws=h["ws"])
        return dict(y=h["y"], ids=h["ids"], weights=h["weights"])
    q, k = st["q_heads"] * st["head_dim"], st["kv_heads"] * st["head_dim"]
    mnb.mnb_qk_rope(h["rope"], h["batch"], st["qkv"][:, :q], st["qkv"][:, q:q + k], h["q"], h["k"])
    return dict(q=h["q"], k=h["k"])


def run(state):
    if own:
        return _own(state)
    return {"qk_rope": _plain_rope, "moe": _plain_moe, "sample": _plain_sample}[state["op"]](state)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _exact_rope(case, st):
    """Pairs of values as complex numbers times e^(i position frequency), a sequence at a time."""
    Hq, Hk, D, R = case["q_heads"], case["kv_heads"], case["head_dim"], case["rotary"]
    lens, starts = st["kv_len"].tolist(), st["q_start"].tolist()
    got = dict(q=[], k=[])
    for s in range(case["seqs"]):
        a, b = starts[s], starts[s + 1]
        pos = torch.arange(lens[s] - (b - a), lens[s], device=st["qkv"].device, dtype=torch.float64)
        for name, lo, heads in (("q", 0, Hq), ("k", Hq * D, Hk)):
            x = st["qkv"][a:b, lo:lo + heads * D].double().reshape(b - a, heads, D)
            if case["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + st["eps"]) * st[name + "_gain"].double()
            order = torch.arange(R, device=x.device)
            order = order.view(-1, 2) if case["interleaved"] else order.view(2, -1).T  # pair i: its two places
            phase = pos[:, None] * st["freq"].double()
            z = torch.complex(x[..., order[:, 0]], x[..., order[:, 1]]) * torch.polar(torch.ones_like(phase),
                                                                                      phase)[:, None]
            x[..., order[:, 0]], x[..., order[:, 1]] = z.real, z.imag
            got[name].append(x)
    return {name: torch.cat(v) for name, v in got.items()}


def _exact_moe(case, st):
    """Token by token, each expert's weights expanded code by code."""
    T, K, I, k, bits = (case[n] for n in ("tokens", "hidden", "inter", "top_k", "bits"))
    x = st["x"].double()
    y = torch.zeros(T, K, dtype=torch.float64, device=x.device)
    ids = torch.zeros(T, k, dtype=torch.int32, device=x.device)
    weights = torch.zeros(T, k, dtype=torch.float64, device=x.device)
    logits = (x[:, None] * st["router"].double()).sum(-1)
    for t, row in enumerate(logits.tolist()):
        first = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        over = first if case["normalize"] else range(len(row))
        z = sum(math.exp(row[e] - row[first[0]]) for e in over)
        ids[t] = torch.tensor(first)
        weights[t] = torch.tensor([math.exp(row[e] - row[first[0]]) / z for e in first], dtype=torch.float64)

    def times(which, e, v):
        """v [n, columns] times the transposed weights, 2048 rows of them at a time."""
        codes, scales, zp = st[which]
        out = []
        for a in range(0, codes.shape[1], 2048):
            c = codes[e, a:a + 2048].reshape(-1, v.shape[1] * bits // 8).long()
            if bits == 4:
                c = (c[..., None] >> torch.tensor([0, 4], device=c.device) & 15).reshape(c.shape[0], -1)
            z = float(1 << bits - 1) if zp is None else zp[e, a:a + 2048].double().repeat_interleave(BLOCK, 1)
            w = (c.double() - z) * scales[e, a:a + 2048].double().repeat_interleave(BLOCK, 1)
            out.append(v @ w.T)
        return torch.cat(out, 1)

    for e in sorted(set(ids.flatten().tolist())):
        hit = ids == e
        tok = hit.any(1).nonzero()[:, 0]
        gu = times("up", e, x[tok])
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        y[tok] += times("down", e, h) * (weights * hit).sum(1)[tok, None]
    return dict(y=y, ids=ids, weights=weights)


def _exact_sample(case, st):
    """A row at a time, by the distinct values of its logits and how often each occurs."""
    token, logprob = [], []
    at = lambda name, r, off: off if st.get(name) is None else st[name][r].item()  # noqa: E731
    for r in range(case["rows"]):
        row = st["logits"][r].double()
        value, count = torch.unique(row, return_counts=True)
        value, count = value.flip(0), count.flip(0).double()
        T, k = at("temperature", r, 1.0), at("top_k", r, 0)
        if T <= 0:
            T, k = 1.0, 1
        w = torch.exp((value - value[0]) / T)
        end = count.cumsum(0)  # places of the order that the value and those before it take
        if k > 0:
            count = torch.minimum(count, (k - (end - count)).clamp(min=0))
        mass = (count * w).cumsum(0)
        p, m, u = at("top_p", r, 1.0), at("min_p", r, 0.0), st["u"][r].item()
        if p < 1:
            need = p * mass[-1] - (mass - count * w)  # what each value's tokens have to bring
            count = torch.minimum(count, torch.ceil(need / w).clamp(min=0))
            count[0] = count[0].clamp(min=1)
        if m > 0:
            count = torch.where((w >= m) | (w == 1), count, 0.0)
        mass = (count * w).cumsum(0)
        target = u * mass[-1]
        i = min(int((mass <= target).sum()), int((count > 0).sum()) - 1)
        j = int(((target - (mass[i] - count[i] * w[i])) / w[i]).floor().clamp(0, count[i] - 1))
        token.append((row == value[i]).nonzero()[j, 0])
        logprob.append(torch.log(w[i] / mass[-1]))
    return dict(token=torch.stack(token), logprob=torch.stack(logprob))


def exact(case, seed):
    st = prepare(case, seed)
    return {"qk_rope": _exact_rope, "moe": _exact_moe, "sample": _exact_sample}[case["op"]](case, st)
