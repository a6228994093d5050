"""mnb_moe against the definition in 64 bits (tolerances: step_helpers.Experts.ref)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from step_helpers import Experts  # noqa: E402

from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu


def run(layer, X, stream=None):
    M = len(X)
    x = torch.from_numpy(X).cuda()
    y = torch.full((M, layer.hidden), 9.0, dtype=torch.float16, device="cuda")
    ids = torch.full((M, layer.top_k), -5, dtype=torch.int32, device="cuda")
    w = torch.full((M, layer.top_k), 9.0, device="cuda")
    mnb.mnb_moe(layer, x, y, ids, w, mnb.moe_workspace(layer, M), stream=stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy(), y.cpu().numpy().astype(np.float64)


def check(ex, layer, X, normalize=True):
    ids, w, y = run(layer, X)
    want = ex.ref(X, layer.top_k, normalize)
    np.testing.assert_array_equal(ids, want[0])
    # exponentials 2^-22, a sum of at most 256 in FP32, a division
    assert np.all(np.abs(w - want[1]) <= (2.0 ** -21 + 16 * 2.0 ** -24) * want[1])
    bad = np.abs(y - want[2]) > want[3]
    assert not bad.any(), (np.argwhere(bad)[:4], bad.sum())


SIZES = [(1, 32, 32, 1, 1, 4, False, True), (1, 64, 96, 4, 2, 8, True, True), (2, 32, 160, 3, 3, 4, "any", False),
         (3, 160, 64, 5, 3, 8, False, True), (16, 576, 256, 8, 2, 4, True, True), (16, 256, 128, 2, 2, 4, False, True),
         (16, 288, 96, 2, 1, 8, "any", False), (16, 128, 64, 256, 16, 4, True, False), (9, 1056, 544, 6, 2, 4, False, True),
         (7, 2080, 352, 7, 7, 8, True, True), (5, 4096, 128, 3, 1, 4, True, True), (13, 96, 2048, 40, 8, 4, False, True),
         (1, 5120, 32, 2, 2, 4, False, False)]


@pytest.mark.parametrize("M,K,I,E,k,bits,zp,normalize", SIZES)
def test_the_definition(M, K, I, E, k, bits, zp, normalize):
    ex = Experts(M * 1000 + K + I, K, I, E, bits, zp)
    X = ex.rng.standard_normal((M, K)).astype(np.float16)
    check(ex, ex.layer(torch, mnb, k, normalize), X, normalize)


@pytest.mark.parametrize("size", [2.0 ** -9, 64.0])
def test_inputs_of_other_sizes(size):
    # the products silu(gate) up lie around size^2: FP16 would lose small ones and overflow with large ones
    ex = Experts(11, 256, 192, 4, 4, True, size)
    X = (ex.rng.standard_normal((6, 256)) * size).astype(np.float16)
    if size < 1:
        codes, scales, z = ex.down
        ex.down = codes, np.float16(scales * np.float16(2.0 ** 9)), z
    else:
        codes, scales, z = ex.down
        ex.down = codes, np.float16(scales * np.float16(2.0 ** -6)), z
    check(ex, ex.layer(torch, mnb, 2, True), X)


def test_equal_logits_go_to_the_lower_expert():
    ex = Experts(12, 64, 32, 40, 4, False)
    ex.router[5:40] = ex.router[4]
    X = ex.rng.standard_normal((8, 64)).astype(np.float16)
    check(ex, ex.layer(torch, mnb, 6, True), X)
    X[:] = 0  # every logit is 0
    ids, w, y = run(ex.layer(torch, mnb, 6, False), X)
    assert np.array_equal(ids, np.tile(np.arange(6), (8, 1))) and np.allclose(w, 1 / 40, rtol=1e-6) and not y.any()


def test_logits_that_differ_beyond_fp32():
    # terms of 2^22 that cancel: what is left decides, and is lost in a 24-bit sum
    ex = Experts(13, 64, 32, 3, 4, False)
    ex.router[:] = 0
    X = np.zeros((1, 64), np.float16)
    X[0, :4] = [2048, 2048, 2048, 1]
    ex.router[0, :4] = [2048, -2048, 0, 2.0 ** -9]
    ex.router[1, :4] = [2048, 0, -2048, 2.0 ** -8]
    ex.router[2, :4] = [0, 2048, -2048, 2.0 ** -10]
    ids, w, y = run(ex.layer(torch, mnb, 3, True), X)
    assert ids.tolist() == [[1, 0, 2]]


@pytest.mark.parametrize("bits", [4, 8])
def test_tokens_do_not_touch_each_other(bits):
    ex = Experts(14, 96, 64, 4, bits, True)
    X = ex.rng.standard_normal((5, 96)).astype(np.float16)
    layer = ex.layer(torch, mnb, 2, True)
    X[1, 7] = np.nan
    X[3, 0] = np.inf
    ids, w, y = run(layer, X)
    assert ids.min() >= 0 and ids.max() < 4
    assert not np.isfinite(y[1]).any() and not np.isfinite(y[3]).all()
    ref = ex.ref(X[[0, 2, 4]], 2, True)
    assert np.array_equal(ids[[0, 2, 4]], ref[0]) and np.all(np.abs(y[[0, 2, 4]] - ref[2]) <= ref[3])


def test_repeats_give_the_same_bits_and_streams_and_graphs_work():
    ex = Experts(15, 512, 256, 16, 4, True)
    X = ex.rng.standard_normal((11, 512)).astype(np.float16)
    layer = ex.layer(torch, mnb, 4, True)
    first = run(layer, X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (run(layer, X), run(layer, X, stream=side)):
        for a, b in zip(first, got):
            np.testing.assert_array_equal(a, b)
    x, y = torch.from_numpy(X).cuda(), torch.empty(11, 512, dtype=torch.float16, device="cuda")
    ws = mnb.moe_workspace(layer, 11)
    ws.fill_(255)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.mnb_moe(layer, x, y, ws=ws)
    for seed in (1, 2):
        X = np.random.default_rng(seed).standard_normal((11, 512)).astype(np.float16)
        x.copy_(torch.from_numpy(X))
        graph.replay()
        torch.cuda.synchronize()
        ref = ex.ref(X, 4, True)
        assert np.all(np.abs(y.cpu().numpy() - ref[2]) <= ref[3])


def test_offsets_past_32_bits():
    K, I, E, where = 4096, 2048, 256, [3, 255]
    ex = Experts(16, K, I, 2, 8, True)
    small = ex.layer(torch, mnb, 2, True)

    def spread(t):
        big = torch.zeros(E, *t.shape[1:], dtype=t.dtype, device="cuda")
        big[where] = t
        return big

    router, *weights = small.kept
    router, weights = spread(router), [spread(t) for t in weights]
    rest = torch.ones(E, dtype=torch.bool)
    rest[where] = False
    router[rest.cuda()] = -0.1  # far below, of positive inputs
    uw, us, uz, dw, ds, dz = weights
    layer = mnb.MoE(router, uw, us, dw, ds, top_k=2, bits=8, up_zp=uz, down_zp=dz, normalize=True)
    X = np.abs(ex.rng.standard_normal((3, K))).astype(np.float16)
    ids, w, y = run(layer, X)
    want = ex.ref(X, 2, True)
    assert np.array_equal(ids, np.array(where)[want[0]])
    assert np.all(np.abs(y - want[2]) <= want[3])
