"""mnb_qk_rope against the definition in 64 bits (tolerances: step_helpers.rope_ref)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from step_helpers import rope_ref  # noqa: E402

from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu


def freqs(half, base=10000.0):
    return (base ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def half(r, *shape):
    return r.standard_normal(shape).astype(np.float16)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def near(got, want):
    ref, tol = want
    bad = np.abs(got.cpu().numpy().astype(np.float64).reshape(ref.shape) - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], bad.sum())


def batch_of(lens, news, table_pages=0):
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) + l - n for l, n in zip(lens, news)]).astype(np.int64)
    b = mnb.KVBatch(torch.zeros(len(lens), table_pages, dtype=torch.int32, device="cuda"), dev(np.int32(lens)), dev(start),
                    int(start[-1]), max(news), max(lens))
    return b, pos


SHAPES = [(1, 1, 64, 64, False), (9, 3, 64, 64, False), (32, 8, 128, 128, False), (5, 1, 128, 32, False),
          (14, 2, 128, 64, True), (3, 0, 64, 16, True), (0, 2, 128, 128, True), (4, 4, 64, 0, False), (1, 7, 128, 96, False),
          (40, 40, 64, 48, True), (17, 1, 128, 16, False)]


@pytest.mark.parametrize("norms", ["none", "both", "q", "k"])
@pytest.mark.parametrize("qh,kh,D,R,inter", SHAPES)
def test_the_definition(qh, kh, D, R, inter, norms):
    r = np.random.default_rng(qh * 100 + kh * 10 + R)
    lens, news = [5, 0, 70003, 1, 33], [5, 0, 3, 1, 1]
    b, pos = batch_of(lens, news)
    T = len(pos)
    f = freqs(R // 2)
    gq, gk = (half(r, D) + np.float16(1) if n in norms or norms == "both" else None for n in "qk")
    Q, K = half(r, T, qh, D), half(r, T, kh, D)
    rope = mnb.Rope(D, dev(f) if R else None, inter, dev(gq), dev(gk), eps=1e-5)
    q, k = dev(Q) if qh else None, dev(K) if kh else None
    qo, ko = (None if x is None else torch.full_like(x, 7.0) for x in (q, k))
    mnb.mnb_qk_rope(rope, b, q, k, qo, ko)
    for x, o, g in ((Q, qo, gq), (K, ko, gk)):
        if o is not None:
            near(o, rope_ref(x, pos, f, inter, g, 1e-5))
    # in place, from given positions
    mnb.mnb_qk_rope(rope, dev(pos.astype(np.int32)), q, k)
    for x, o in ((q, qo), (k, ko)):
        assert x is None or torch.equal(x.view(torch.int16), o.view(torch.int16))


@pytest.mark.parametrize("inter", [False, True])
def test_slices_of_a_fused_row(inter):
    r = np.random.default_rng(3)
    qh, kh, D, T = 6, 2, 64, 37
    row = dev(half(r, T, (qh + 2 * kh) * D + 8))
    was = row.clone()
    f = freqs(D // 2, 500.0)
    pos = r.integers(0, 1 << 20, T).astype(np.int32)
    rope = mnb.Rope(D, dev(f), inter)
    q, k = row[:, :qh * D], row[:, qh * D:(qh + kh) * D]
    mnb.mnb_qk_rope(rope, dev(pos), q, k)
    want = was.cpu().numpy()
    near(q, rope_ref(want[:, :qh * D].reshape(T, qh, D), pos, f, inter))
    near(k, rope_ref(want[:, qh * D:(qh + kh) * D].reshape(T, kh, D), pos, f, inter))
    assert torch.equal(row[:, (qh + kh) * D:], was[:, (qh + kh) * D:])


def test_far_positions_and_large_frequencies():
    r = np.random.default_rng(4)
    pos = np.array([0, 1, 131071, 1 << 24, (1 << 24) + 1, (1 << 31) - 4097, (1 << 31) - 1], np.int32)
    f = np.array([1.0, 0.999, 6.2831855, 100.7, 1e-3, 1e-8, -0.3, 0.0], np.float32)
    Q = half(r, len(pos), 2, 64)
    q = dev(Q)
    mnb.mnb_qk_rope(mnb.Rope(64, dev(f)), dev(pos), q)
    near(q, rope_ref(Q, pos, f))


def test_rows_without_a_position_are_left_alone():
    r = np.random.default_rng(5)
    f, D = freqs(32), 64
    rope = mnb.Rope(D, dev(f))
    Q = half(r, 9, 2, D)
    pos = np.array([3, -1, 8, -(1 << 31), 0, 5, -7, 2, 1], np.int32)
    q = dev(Q)
    mnb.mnb_qk_rope(rope, dev(pos), q)
    left = pos < 0
    assert np.array_equal(q.cpu().numpy()[left], Q[left])
    near(q[torch.from_numpy(~left).cuda()], rope_ref(Q[~left], pos[~left], f))
    # a batch whose sequences own fewer rows than the call has, and one with tokens before position 0
    b, _ = batch_of([4, 2, 6], [2, 4, 3])
    b.q_start.copy_(torch.tensor([0, 2, 6, 7], dtype=torch.int32))
    where = np.array([2, 3, -2, -1, 0, 1, 5, -1, -1])
    q = dev(Q)
    mnb.mnb_qk_rope(rope, b, q)
    left = where < 0
    assert np.array_equal(q.cpu().numpy()[left], Q[left])
    near(q[torch.from_numpy(~left).cuda()], rope_ref(Q[~left], where[~left], f))


def test_values_that_are_not_finite_stay_in_their_pair():
    D, f = 64, freqs(16)
    x = np.ones((2, 1, D), np.float16)
    x[0, 0, 3], x[0, 0, 40], x[1, 0, 63] = np.inf, np.nan, -np.inf  # a pair (3, 19), two places that are not turned
    q = dev(x)
    mnb.mnb_qk_rope(mnb.Rope(D, dev(f)), torch.tensor([7, 9], dtype=torch.int32, device="cuda"), q)
    bad = ~np.isfinite(q.cpu().numpy()[:, 0])
    assert set(np.flatnonzero(bad[0])) == {3, 19, 40} and set(np.flatnonzero(bad[1])) == {63}


def test_a_captured_call_on_another_stream_takes_new_lengths():
    r = np.random.default_rng(6)
    f, D = freqs(64), 128
    b, pos = batch_of([10, 200, 3], [1, 1, 1])
    Q = half(r, 3, 4, D)
    q, out = dev(Q), torch.empty(3, 4, D, dtype=torch.float16, device="cuda")
    rope = mnb.Rope(D, dev(f), q_weight=torch.ones(D, dtype=torch.float16, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mnb.mnb_qk_rope(rope, b, q, None, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mnb.mnb_qk_rope(rope, b, q, None, out)
    for step in (0, 1, 5000):
        b.kv_len.copy_(torch.tensor([10 + step, 200 + step, 3 + step], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        near(out, rope_ref(Q, pos + step, f, False, np.ones(D, np.float16)))


def test_many_tokens_and_many_sequences():
    r = np.random.default_rng(7)
    news = list(r.integers(0, 30, 300))
    lens = [int(n + r.integers(0, 1000)) if n else 0 for n in news]
    b, pos = batch_of(lens, [int(n) for n in news])
    D, f = 64, freqs(32)
    Q = half(r, len(pos), 3, D)
    q = dev(Q)
    mnb.mnb_qk_rope(mnb.Rope(D, dev(f), True), b, q)
    near(q, rope_ref(Q, pos, f, True))


@pytest.mark.parametrize("tokens,stride", [(5, (1 << 29) + 8), (4001, (1 << 20) + 8)])
def test_offsets_past_32_bits(tokens, stride):
    # one token a CTA and several
    r = np.random.default_rng(tokens)
    Q, K = half(r, tokens, 3, 64), half(r, tokens, 1, 64)
    flat = torch.empty((tokens - 1) * stride + 256, dtype=torch.float16, device="cuda")
    q, k = flat.as_strided((tokens, 3, 64), (stride, 64, 1)), flat[192:].as_strided((tokens, 1, 64), (stride, 64, 1))
    q.copy_(torch.from_numpy(Q)), k.copy_(torch.from_numpy(K))
    pos, f, gain = np.arange(tokens) * 7, freqs(32), half(r, 64) + np.float16(1)
    mnb.mnb_qk_rope(mnb.Rope(64, dev(f), q_weight=dev(gain)), dev(np.int32(pos)), q, k)
    for x, o, g in ((Q, q, gain), (K, k, None)):
        near(o.contiguous(), rope_ref(x, pos, f, False, g))
