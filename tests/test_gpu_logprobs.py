"""mnb_logprobs against the definition in 64 bits.

Tolerances: a thread adds at most 392 terms one after the other and a cluster 2048 threads in a tree, each
rounding 2^-24 of the sum; 2^x is within 2^-22; the exponent's own rounding is 2^-24 of the largest |x|.
log Z takes these as they are, the entropy times the terms' own size (its own value and the reference's
distance, at most 4 ln 2)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 410 * 2.0 ** -24 + 2.0 ** -21


def run(x, target=None, k=0, scale=1.0, stream=None):
    rows = x.shape[0]
    lp, h = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    ids = torch.full((rows, k), -7, dtype=torch.int32, device="cuda")
    tops = torch.full((rows, k), 7.0, device="cuda")
    t = None if target is None else torch.from_numpy(np.asarray(target, np.int64)).cuda()
    mnb.mnb_logprobs(x, t, None if t is None else lp, h, ids if k else None, tops if k else None, scale=scale,
                     stream=stream)
    torch.cuda.synchronize()
    return lp.cpu().numpy(), h.cpu().numpy(), ids.cpu().numpy(), tops.cpu().numpy()


def check(x16, target, k, scale=1.0, xd=None):
    lp, h, ids, tops = run(torch.from_numpy(x16).cuda() if xd is None else xd, target, k, scale)
    for r, row in enumerate(x16):
        x = row.astype(np.float64) * scale
        best = np.lexsort((np.arange(len(x)), -x))[:k]
        np.testing.assert_array_equal(ids[r], best)
        m = x.max()
        if m == -np.inf:
            assert h[r] == 0 and np.all(tops[r] == -np.inf)
            continue
        lse = m + np.log(np.exp(x - m).sum())
        p = np.exp(x - lse)
        ent = -(p[p > 0] * (x[p > 0] - lse)).sum()
        size = np.abs(x[np.isfinite(x)]).max() + abs(lse)
        tol = EPS + 2.0 ** -22 * size
        assert abs(h[r] - ent) <= tol * (4 + ent), (r, h[r], ent)
        for got, want in list(zip(tops[r], x[best] - lse)) + [(lp[r], x[target[r]] - lse)]:
            assert got == want if np.isinf(want) else abs(got - want) <= tol, (r, got, want)


SIZES = [(1, 1, 1), (3, 2, 2), (2, 7, 3), (5, 8, 8), (4, 9, 0), (2, 33, 32), (3, 255, 5), (200, 2049, 20),
         (1, 49152, 5), (3, 50257, 20), (40, 20000, 1), (2, 151936, 32), (1, 163841, 7), (1, 786432, 20),
         (330, 4999, 4)]


@pytest.mark.parametrize("rows,vocab,k", SIZES)
def test_the_definition(rows, vocab, k):
    r = np.random.default_rng(rows * 7 + vocab)
    x = (r.standard_normal((rows, vocab)) * 3).astype(np.float16)
    check(x, r.integers(0, vocab, rows), k, scale=1.0 if vocab % 2 else 1 / 0.7)


def test_odd_strides_and_another_stream():
    r = np.random.default_rng(1)
    x = (r.standard_normal((6, 1003)) * 2).astype(np.float16)
    for stride in (1003, 1004, 1007, 1024):
        wide = torch.full((6, stride), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, :1003] = torch.from_numpy(x).cuda()
        check(x, [0, 1, 2, 1002, 500, 7], 9, xd=wide[:, :1003])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = run(wide[:, :1003], [3] * 6, 4, stream=side), run(wide[:, :1003], [3] * 6, 4)
    for p, q in zip(a, b):
        np.testing.assert_array_equal(p, q)


def test_ties_go_to_the_lowest_id():
    x = np.zeros((4, 30000), np.float16)
    x[0, ::2] = -0.0                       # equal to +0
    x[1] = 3.0
    x[2, 29990:] = 1.0
    x[3, 5::9] = 2.0                       # more equal ones than a list holds
    check(x, [0, 1, 29999, 5], 32)


def test_peaked_and_wide_rows():
    r = np.random.default_rng(2)
    x = (r.standard_normal((5, 40000))).astype(np.float16)
    x[0, 39999] = 60.0
    x[1, 17] = 20.0
    x[2] *= np.float16(200)
    x[3] = np.sort(x[3])
    x[4] = -60000.0
    x[4, 31234] = 60000.0
    check(x, [39999, 17, 3, 39999, 31234], 6)


def test_masked_tokens_and_empty_rows():
    r = np.random.default_rng(3)
    x = r.standard_normal((5, 9000)).astype(np.float16)
    x[0, :8000] = -np.inf
    x[1, 3:] = -np.inf                     # three tokens left, ten asked for
    x[2] = -np.inf
    x[3, ::2] = -np.inf
    lp, h, ids, tops = run(torch.from_numpy(x).cuda(), [3, 0, 4, 0, 5], 10)
    assert lp[2] == -np.inf and lp[0] == -np.inf and lp[3] == -np.inf
    check(x, [8001, 4, 4, 1, 5], 10)


@pytest.mark.parametrize("scale", [1.0, 1e-5, 8.0])
def test_lowest_values_beside_masked_tokens(scale):
    # FP16's lowest value is a logit, -infinity is none, whatever the scale
    x = np.full((4, 9001), -np.inf, np.float16)
    x[0, ::3] = -65504
    x[1, :10] = -65504
    x[1, 10:20] = -65472
    x[2] = -65504
    x[3, ::2] = -65504
    x[3, 7] = 1.0
    check(x, [3, 11, 9000, 7], 12, scale=scale)


def test_non_finite_rows_and_targets_of_no_token():
    r = np.random.default_rng(4)
    x = r.standard_normal((5, 3001)).astype(np.float16)
    x[1, 2999] = np.nan
    x[2, 5] = np.inf
    x[3] = np.nan
    lp, h, ids, tops = run(torch.from_numpy(x).cuda(), [-1, 0, 5, 1, 3001], 8)
    for row in (1, 2, 3):
        assert np.isnan(lp[row]) and np.isnan(h[row]) and np.all(np.isnan(tops[row]))
    assert np.all((ids >= 0) & (ids < 3001))
    assert lp[0] == 0 and lp[4] == 0 and np.all(np.isfinite(h[[0, 4]]))


def test_without_target_or_alternatives():
    x = torch.randn(3, 5000, device="cuda").half()
    lp, h, ids, tops = run(x)
    assert np.all(lp == 7) and np.all(np.isfinite(h))
    _, h2, ids, _ = run(x, [1, 2, 3], 32)
    np.testing.assert_array_equal(h, h2)
    for r in range(3):
        assert len(set(ids[r])) == 32
