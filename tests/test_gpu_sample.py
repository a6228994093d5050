"""mnb_sample against the definition in 64 bits: the same token, its log probability to FP32's rounding and 2^-18
(the part of a row that is summed in FP32)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from step_helpers import sample_ref  # noqa: E402

from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu


def dev(a, t):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()


def run(x, u, temperature=None, top_k=None, top_p=None, min_p=None, xd=None, stream=None):
    rows = x.shape[0]
    token = torch.full((rows,), -7, dtype=torch.int64, device="cuda")
    lp = torch.full((rows,), 7.0, device="cuda")
    mnb.mnb_sample(torch.from_numpy(x).cuda() if xd is None else xd, dev(u, np.float32), token, lp,
                   dev(temperature, np.float32), dev(top_k, np.int32), dev(top_p, np.float32), dev(min_p, np.float32),
                   stream=stream)
    torch.cuda.synchronize()
    return token.cpu().numpy(), lp.cpu().numpy()


def check(x, u, temperature=None, top_k=None, top_p=None, min_p=None, xd=None):
    token, lp = run(x, u, temperature, top_k, top_p, min_p, xd)
    f = lambda a, r, off: off if a is None else np.float32(a[r])  # noqa: E731
    for r in range(len(x)):
        want = sample_ref(x[r], np.float32(u[r]), f(temperature, r, 1.0), 0 if top_k is None else top_k[r],
                          f(top_p, r, 1.0), f(min_p, r, 0.0))
        assert token[r] == want[0], (r, token[r], want)
        if np.isfinite(want[1]):
            assert abs(lp[r] - want[1]) <= 2.0 ** -18 + 2.0 ** -23 * abs(want[1]), (r, lp[r], want)
        else:
            assert np.isnan(lp[r]) if np.isnan(want[1]) else lp[r] == want[1], (r, lp[r], want)


def logits(seed, rows, vocab, spread=2.5, likely=40):
    r = np.random.default_rng(seed)
    x = (r.standard_normal((rows, vocab)) * spread).astype(np.float32)
    for i in range(rows):
        at = r.integers(0, vocab, likely)
        x[i, at] += r.uniform(0, 14, likely).astype(np.float32)
    return r, x.astype(np.float16)


def settings(r, kind, rows):
    t = r.uniform(0.5, 1.3, rows)
    d = dict(temperature=t, top_k=r.choice([0, 1, 3, 50, 700], rows), top_p=r.choice([0.0, 0.5, 0.9, 0.99, 1.0], rows),
             min_p=r.choice([0.0, 0.01, 0.2], rows))
    return {"mixed": d, "none": {}, "temperature": dict(temperature=t), "greedy": dict(temperature=np.zeros(rows)),
            "top_k": dict(top_k=d["top_k"]), "top_p": dict(top_p=d["top_p"], temperature=t),
            "min_p": dict(min_p=d["min_p"])}[kind]


@pytest.mark.parametrize("kind", ["mixed", "none", "temperature", "greedy", "top_k", "top_p", "min_p"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 3), (5, 8), (7, 33), (40, 255), (3, 2049), (9, 4999), (1, 49152),
                                        (4, 50257), (330, 1003), (2, 151936)])
def test_the_definition(rows, vocab, kind):
    r, x = logits(rows * 31 + vocab, rows, vocab)
    check(x, r.uniform(0, 1, rows), **settings(r, kind, rows))


@pytest.mark.parametrize("kind", ["mixed", "none", "top_p", "min_p"])
@pytest.mark.parametrize("spread", [0.0, 0.02, 0.3, 1.0, 9.0])
def test_flat_and_wide_rows(spread, kind):
    # little or nothing stands out: places far down the order, equal logits, values around zero on both sides
    r, x = logits(int(spread * 100) + 5, 6, 6007, spread, 1 if spread < 1 else 20)
    check(x, r.uniform(0, 1, 6), **settings(r, kind, 6))


@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, np.nan, 0.5, 2.0 ** -24])
def test_the_ends_of_u(u):
    r, x = logits(77, 5, 3001)
    for kind in ("none", "top_k", "top_p"):
        check(x, np.full(5, u), **settings(r, kind, 5))


def test_settings_out_of_their_range():
    r, x = logits(78, 8, 1000)
    u = r.uniform(0, 1, 8)
    check(x, u, top_k=[-1, 0, 1000, 2000, 2 ** 31 - 1, -2 ** 31, 999, 1])
    check(x, u, temperature=[-1.0, np.nan, np.inf, 1e-30, 1e-40, 1e30, 3e38, 0.0])
    token, _ = run(x, u, top_p=[np.nan, np.inf, -1.0, 2.0, 1.0, 0.0, -np.inf, 1e-30])
    full, _ = run(x, u)
    best = x.argmax(1)
    assert [token[i] for i in (0, 1, 3, 4)] == [full[i] for i in (0, 1, 3, 4)]
    assert [token[i] for i in (2, 5, 6, 7)] == [best[i] for i in (2, 5, 6, 7)]
    token, _ = run(x, u, min_p=[np.nan, np.inf, -1.0, 2.0, 1.0, 0.0, -np.inf, 1.5])
    assert [token[i] for i in (0, 2, 5, 6)] == [full[i] for i in (0, 2, 5, 6)]
    assert [token[i] for i in (1, 3, 4, 7)] == [best[i] for i in (1, 3, 4, 7)]


def test_masked_tokens_and_bad_rows():
    r, x = logits(79, 12, 2003)
    x[0, ::2] = -np.inf
    x[1, :] = -np.inf
    x[2, :] = -np.inf
    x[2, 1700] = -65504
    x[3, 5] = np.nan
    x[4, 2002] = np.inf
    x[5, :] = np.nan
    x[6, :] = -np.inf
    x[6, [3, 2002]] = 1.0
    x[7, :] = 0.0
    x[7, ::3] = -0.0
    x[8, :] = -65504
    x[9, 11], x[9, 12] = 65504, 65504
    x[10, 0] = np.inf
    x[10, 1] = np.nan
    x[11, 1:] = -np.inf
    for kind in ("none", "mixed", "top_p", "greedy", "min_p"):
        check(x, r.uniform(0, 1, 12), **settings(r, kind, 12))


def test_runs_of_equal_logits_far_apart():
    # the drawn value is shared by tokens at both ends of the row, in every CTA and warp
    x = np.full((6, 40001), -3.0, np.float16)
    x[:, ::7] = 2.0
    x[1, :] = 1.0
    u = np.array([0.0, 0.999999, 0.25, 0.5, 0.75, 0.97])
    check(x, u)
    check(x, u, top_k=[1, 3, 1000, 4000, 5715, 5800])
    check(x, u, top_p=[0.1, 0.2, 0.3, 0.9, 0.95, 0.99])


def test_min_p_whose_place_lies_far_down():
    # the last kept logit lies more orders below the largest than the first histogram holds
    r = np.random.default_rng(83)
    two = np.where(r.random((40, 77)) < 0.5, 1.0, -1.0).astype(np.float16)
    ties = np.round(r.standard_normal((40, 4999)) * 2).astype(np.float16)
    flat = (r.standard_normal((40, 20011)) * 0.5).astype(np.float16)
    for x in (two, ties, flat):
        for m in (0.5, 0.1, 0.001, 1e-6):
            u, t = r.uniform(0, 1, 40), r.uniform(0.4, 3, 40)
            check(x, u, t, min_p=np.full(40, m))
            check(x, u, t, min_p=np.full(40, m), top_p=np.full(40, 0.99))
            check(x, u, t, min_p=np.full(40, m), top_k=np.full(40, 3000))


@pytest.mark.parametrize("vocab", [700, 20011, 90001])
def test_limits_and_draws_in_lower_windows(vocab):
    # flat rows: the limit, the drawn token or both lie one window or more below the first, some rows end in the second
    r = np.random.default_rng(vocab)
    for x in (r.standard_normal((24, vocab)) * 2.5, r.standard_normal((24, vocab)) * 0.4, r.uniform(0, 12, (24, vocab)),
              np.abs(r.standard_normal((24, vocab))) * 2.0 ** -r.integers(0, 12, (24, vocab))):
        x = x.astype(np.float16)
        u = r.uniform(0, 1, 24)
        u[:4] = 0.999, 0.99999, 0.0, 1.0
        t = r.uniform(0.7, 4, 24)
        check(x, u, t)
        check(x, u, t, top_p=r.uniform(0.9, 1, 24))
        check(x, u, t, top_p=r.uniform(0, 1, 24), min_p=r.choice([0.0, 1e-4], 24))


def test_odd_strides_and_another_stream():
    r, x = logits(80, 6, 1003)
    u = r.uniform(0, 1, 6)
    for stride in (1003, 1004, 1007, 1024):
        wide = torch.full((6, stride), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, :1003] = torch.from_numpy(x).cuda()
        check(x, u, top_p=np.full(6, 0.9), xd=wide[:, :1003])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, b in zip(run(x, u, stream=side), run(x, u)):
        np.testing.assert_array_equal(a, b)


def test_a_large_vocabulary():
    r, x = logits(81, 2, (1 << 20) + 13, 1.0)
    check(x, r.uniform(0, 1, 2))
    check(x, r.uniform(0, 1, 2), top_p=[0.9, 0.5])
    check(x, r.uniform(0, 1, 2), top_k=[5000, 100000])


def test_a_replayed_graph_takes_new_settings():
    r, x = logits(82, 4, 5003)
    xd, u = torch.from_numpy(x).cuda(), torch.zeros(4, device="cuda")
    t, k = torch.ones(4, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    token, lp = torch.empty(4, dtype=torch.int64, device="cuda"), torch.empty(4, device="cuda")
    mnb.mnb_sample(xd, u, token, lp, t, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.mnb_sample(xd, u, token, lp, t, k)
    for seed in range(3):
        r, x = logits(seed, 4, 5003)
        us, ts, ks = r.uniform(0, 1, 4).astype(np.float32), r.uniform(0, 2, 4).astype(np.float32), [0, 5, 50, 1]
        xd.copy_(torch.from_numpy(x)), u.copy_(dev(us, np.float32)), t.copy_(dev(ts, np.float32))
        k.copy_(dev(ks, np.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert token.tolist() == [sample_ref(x[i], us[i], ts[i], ks[i])[0] for i in range(4)]


def test_offsets_past_32_bits():
    r, x = logits(84, 3, 1000)
    stride = (1 << 30) + 5
    flat = torch.empty(2 * stride + 1000, dtype=torch.float16, device="cuda")
    rows = flat.as_strided((3, 1000), (stride, 1))
    rows.copy_(torch.from_numpy(x))
    check(x, r.uniform(0, 1, 3), top_p=[0.9, 1.0, 0.5], xd=rows)
