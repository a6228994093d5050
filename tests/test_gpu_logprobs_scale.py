"""mnb_logprobs with scales from the largest binary32 takes down to a hundredth: the definition in 64 bits on
differences of logits, whose size does not matter then.  And what the sums lose where one token is likely."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from test_gpu_logprobs import EPS, run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.01, 1.0, 100.0, 177.0, 178.0, 1e3, 2e4, 1e6, 1e12, 1e30, 2e38])
def test_scales_of_any_size(scale):
    # a temperature near zero: differences of logits are what counts, however large scale times a logit is
    r = np.random.default_rng(9)
    x = (r.standard_normal((6, 5003)) * 3).astype(np.float16)
    x[1] = np.clip(x[1].astype(np.float32) * 5e3, -65504, 65504)
    x[2, 7:9] = 65504
    x[3] = np.float16(2.0 ** -24) * r.integers(0, 9, 5003)
    x[4, ::3] = -np.inf
    x[5] = -65504
    lp, h, ids, tops = run(torch.from_numpy(x).cuda(), [3, 4, 7, 6, 1, 0], 5, scale=scale)
    for i, row in enumerate(x):
        best = np.lexsort((np.arange(5003), -row.astype(np.float64)))[:5]
        np.testing.assert_array_equal(ids[i], best)
        y = (row.astype(np.float64) - row.max()) * np.float64(np.float32(scale))
        logz = np.log(np.exp(y).sum())
        p = np.exp(y - logz)
        ent = -(p[p > 0] * (y[p > 0] - logz)).sum()
        assert abs(h[i] - ent) <= EPS * (8 + ent) + 2.0 ** -20, (i, h[i], ent)
        for got, at in list(zip(tops[i], best)) + [(lp[i], [3, 4, 7, 6, 1, 0][i])]:
            want = y[at] - logz
            if want < -2.3e38:  # below binary32 in units of log2, or a token that cannot be drawn
                assert got < -2.3e38, (i, got, want)
            else:
                assert abs(got - want) <= EPS + 2.0 ** -22 * abs(want), (i, got, want)


def test_the_entropy_of_rows_with_one_likely_token():
    # log Z and the mean of y are about zero then: what is left are the roundings of a sum near 1, at most 12 a thread
    # and 11 of the joins, 2^-23 / sqrt(12) each
    r = np.random.default_rng(10)
    x = (r.standard_normal((40, 49152)) * 2).astype(np.float16)
    x[np.arange(40), r.integers(0, 49152, 40)] = r.uniform(16, 19, 40).astype(np.float16)
    h = run(torch.from_numpy(x).cuda(), scale=1.0)[1].astype(np.float64)
    y = x.astype(np.float64)
    y -= np.log(np.exp(y).sum(1))[:, None]
    want = -(np.exp(y) * y).sum(1)
    assert np.sqrt(((h - want) ** 2).mean()) <= 23 ** 0.5 * 2.0 ** -23 / 12 ** 0.5
