"""mnb_attn against the definition in 64 bits (lm_helpers.attn_ref, which says where its tolerance comes from)."""
import numpy as np
import pytest

from lm_helpers import Case, attn_ref

torch = pytest.importorskip("torch")
from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu


def run(c, q, scale, window=0, out=None, stream=None, **hints):
    cache, batch = c.upload(torch, mnb, **hints)
    qd = torch.from_numpy(q).cuda()
    out = torch.full_like(qd, 7.0) if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = mnb.attn_workspace(cache, batch, q.shape[1], window)
    if ws is not None:
        ws.fill_(255)  # NaN: what a call does not write, it does not read
    torch.cuda.synchronize()
    mnb.mnb_attn(cache, batch, qd, out, scale=scale, window=window, lse=lse, ws=ws, stream=stream)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)


def queries(c, heads, seed=0):
    r = np.random.default_rng(seed + 5)
    return r.standard_normal((c.T, heads, c.D)).astype(np.float16)


def check(c, heads, window=0, scale=None, seed=0, **kw):
    q = queries(c, heads, seed)
    scale = c.D ** -0.5 if scale is None else scale
    want, want_lse, tol = attn_ref(c, q, scale, window)
    out, lse = run(c, q, scale, window, **kw)
    assert np.all(np.isfinite(out))
    worst = np.max(np.abs(out - want) / tol)
    assert worst <= 1, f"worst error is {worst:.3g} of its tolerance"
    empty = np.isinf(want_lse)
    assert np.all(lse[empty] == -np.inf) and np.all(out[empty] == 0)
    assert np.all(np.abs(lse - want_lse)[~empty] <= 2e-4 + 1e-6 * np.abs(want_lse[~empty]))
    return out


CASES = [  # lens, news, kv heads, group, dim, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [1], 3, 3, 64, 16, 0),
    ([577], [1], 3, 3, 64, 16, 0),
    ([15, 16, 17, 0], [1, 1, 1, 1], 2, 8, 128, 16, 0),     # the last one is a token without a position
    ([63, 64, 65, 0], [1, 1, 1, 0], 2, 7, 64, 32, 0),      # the last one is an idle slot
    ([300, 9, 128], [1, 1, 1], 2, 4, 128, 64, 0),
    ([1500], [1], 1, 16, 128, 256, 0),
    ([200], [1], 1, 32, 64, 128, 0),                       # more heads on a kv head than a tile has rows
    ([5], [5], 1, 1, 128, 16, 0),
    ([40, 3], [5, 3], 2, 7, 64, 32, 0),
    ([37, 70, 0, 16], [37, 9, 0, 16], 2, 3, 64, 16, 0),
    ([130], [130], 1, 2, 128, 16, 0),
    ([300], [129], 1, 5, 64, 64, 0),
    ([260, 33], [140, 33], 2, 8, 128, 32, 0),
    ([3, 40], [8, 2], 1, 2, 64, 16, 0),                    # five tokens before position 0
    ([500], [1], 2, 2, 128, 16, 1),
    ([500], [1], 2, 2, 64, 16, 7),
    ([500, 20], [1, 1], 1, 4, 128, 32, 100),
    ([300], [140], 1, 3, 64, 16, 33),
    ([300, 60], [150, 60], 1, 8, 128, 16, 16),
    ([90], [90], 2, 1, 64, 32, 5000),
    ([40] * 70, [1] * 70, 1, 2, 64, 16, 0),
    ([6, 30] * 300, [3, 0] * 300, 1, 8, 64, 16, 0),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention_is_the_definition(i):
    lens, news, H, G, D, P, window = CASES[i]
    check(Case(i, lens, news, H, D, P), H * G, window, seed=i)


@pytest.mark.parametrize("news", [[1, 1], [3, 60]])
def test_value_scales_of_any_size(news):
    # a tiny scale beside a huge one, blocks of zeros, every sequence dominated by one block
    c = Case(30, [90, 150], news, 2, 64, 16, v_spread=True)
    for p in (0, 3):
        c.scales[1][p], c.codes[1][p] = 0, 128
    check(c, 6)


@pytest.mark.parametrize("news", [[1], [40]])
def test_large_scores(news):
    c = Case(31, [200], news, 1, 128, 16)
    check(c, 4, scale=3.0)


@pytest.mark.parametrize("news,window", [([1, 1], 20), ([45, 30], 20), ([45, 30], 0)])
def test_hidden_blocks_may_hold_anything(news, window):
    # NaN and infinite scales in blocks past the end and out of the window, and in pages of no sequence
    lens = [120, 77]
    c = Case(32, lens, news, 2, 64, 32)
    shown = [x.copy() for x in c.scales]
    used = np.zeros((c.pages, c.P // 16), bool)
    for s, (n, length) in enumerate(zip(news, lens)):
        first = max(0, length - n - window + 1) if window else 0
        for b in range(first // 16, -(-length // 16)):
            used[c.table[s, b * 16 // c.P], b * 16 % c.P // 16] = True
    for w in (0, 1):
        for bad, share in ((np.nan, 0), (np.inf, 1)):
            hide = ~used & (np.arange(c.pages)[:, None] % 2 == share)
            c.scales[w][np.broadcast_to(hide[:, None], c.scales[w].shape)] = bad
    q = queries(c, 6)
    out, lse = run(c, q, 0.125, window)
    c.scales = shown
    want, want_lse, tol = attn_ref(c, q, 0.125, window)
    assert np.all(np.abs(out - want) <= tol) and np.all(np.isfinite(lse))


def test_rows_masked_from_a_bad_block_stay_finite():
    # causal rows before a block with a NaN scale are finite, the rows that see it are NaN
    c = Case(33, [64], [64], 1, 64, 16)
    c.scales[1][c.table[0, 2], 0, 0] = np.nan
    out, _ = run(c, queries(c, 2), 0.125)
    assert np.all(np.isfinite(out[:32])) and np.all(np.isnan(out[32:]))


@pytest.mark.parametrize("news", [[1, 1], [50, 40]])
def test_pages_outside_the_cache_are_hidden(news):
    c = Case(34, [100, 60], news, 2, 128, 16)
    c.table[0, 1], c.table[1, 0], c.table[0, 6] = -5, c.pages, 2 ** 31 - 1
    check(c, 4)


def test_no_pages_at_all():
    c = Case(35, [30], [2], 1, 64, 16)
    c.table[:] = -1
    assert np.all(check(c, 2) == 0)


@pytest.mark.parametrize("lens,news", [([3000], [1]), ([2500, 2200], [1, 2]), ([1400], [40])])
def test_wrong_length_bounds_cost_time_only(lens, news):
    c = Case(36, lens, news, 1, 64, 64)
    for max_len in (1, 100, 100000):
        check(c, 2, max_len=max_len)
    check(c, 2, max_new=64)


def test_strided_rows_another_stream_and_repeats():
    c = Case(37, [900, 333], [1, 3], 2, 64, 32)
    q = queries(c, 6)
    cache, batch = c.upload(torch, mnb)
    fused = torch.zeros(c.T, 10 * 64, dtype=torch.float16, device="cuda")
    fused[:, :384] = torch.from_numpy(q).cuda().view(c.T, -1)
    wide = torch.zeros(c.T, 512, dtype=torch.float16, device="cuda")
    ws = mnb.attn_workspace(cache, batch, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mnb.mnb_attn(cache, batch, fused[:, :384], wide[:, :384], ws=ws, stream=side)
    side.synchronize()
    want, _, tol = attn_ref(c, q, 64 ** -0.5)
    got = wide[:, :384].float().cpu().numpy().reshape(want.shape)
    assert np.all(np.abs(got - want) <= tol) and torch.all(wide[:, 384:] == 0)
    again = torch.empty_like(wide[:, :384])
    mnb.mnb_attn(cache, batch, fused[:, :384], again, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(again, wide[:, :384])


def test_graph_replay_with_other_lengths():
    c = Case(38, [400, 250], [1, 1], 2, 128, 64)
    q = queries(c, 4)
    cache, batch = c.upload(torch, mnb)
    qd = torch.from_numpy(q).cuda()
    out, ws = torch.empty_like(qd), mnb.attn_workspace(cache, batch, 4)
    mnb.mnb_attn(cache, batch, qd, out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.mnb_attn(cache, batch, qd, out, ws=ws)
    for lens in ([400, 250], [17, 64], [0, 399]):
        c.lens = lens
        batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        if lens[1] > 250:  # longer than the table's own pages: give it some of the other sequence's
            c.table[1] = c.table[0]
            batch.page_table.copy_(torch.from_numpy(c.table))
        graph.replay()
        torch.cuda.synchronize()
        want, _, tol = attn_ref(c, q, 128 ** -0.5)
        assert np.all(np.abs(out.float().cpu().numpy() - want) <= tol)


def test_offsets_past_32_bits():
    H, D, P = 8, 128, 256
    pages = (1 << 32) // (H * P * D) + 4
    big = [torch.empty(pages, H, P, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.empty(pages, H, P // 16, device="cuda") for _ in range(2)]
    c = Case(39, [300], [2], H, D, P, spare=0)
    where = torch.tensor([pages - 1, pages - 4], device="cuda")
    at = torch.from_numpy(c.table[0, :2].astype(np.int64)).cuda()
    for w in (0, 1):
        big[w][where] = torch.from_numpy(c.codes[w]).cuda()[at]
        sc[w][where] = torch.from_numpy(c.scales[w]).cuda()[at]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = mnb.KVCache(*big, *sc)
    q = queries(c, 8)
    want, _, tol = attn_ref(c, q, 128 ** -0.5)
    batch = mnb.KVBatch(where.to(torch.int32).view(1, 2), i32(300), i32(0, 2), 2, 2, 300)
    qd = torch.from_numpy(q).cuda()
    out = torch.empty_like(qd)
    mnb.mnb_attn(cache, batch, qd, out, ws=mnb.attn_workspace(cache, batch, 8))
    torch.cuda.synchronize()
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("dim,window", [(64, 0), (128, 0), (128, 50)])
@pytest.mark.parametrize("max_len", [None, 60000])
def test_prompts_among_single_tokens(dim, window, max_len):
    # rows of both kernels in one call: a prompt, one over and one at the split kernel's 48 rows, single
    # tokens, an idle slot; a large length bound cuts the keys into many chunks
    c = Case(40, [310, 80, 97, 40, 0, 700], [170, 13, 12, 1, 0, 1], 2, dim, 32)
    check(c, 8, window, max_len=max_len)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news", [[1], [9], [200]])
def test_scores_that_rise_along_the_keys(dim, news):
    # the reference of the sum has to move again and again, in the end by more than binary32's range of 2^x
    c = Case(41, [700], news, 1, dim, 16)
    r = np.random.default_rng(41)
    grow = np.linspace(0.0, 0.2, c.table.shape[1])
    for b, p in enumerate(c.table[0]):
        if p >= 0:
            c.codes[0][p] = r.integers(200, 256, c.codes[0][p].shape, dtype=np.uint8)
            c.scales[0][p] = grow[b]
    q = np.abs(queries(c, 2))
    want, want_lse, tol = attn_ref(c, q, 0.3)
    out, lse = run(c, q, 0.3)
    assert np.all(np.abs(out - want) <= tol)
    assert np.all(np.abs(lse - want_lse) <= 2e-4 + 1e-6 * np.abs(want_lse))


@pytest.mark.parametrize("news", [[4], [60]])
def test_a_bad_query_row_stays_alone(news):
    c = Case(42, [150], news, 1, 64, 16)
    q = queries(c, 3)
    want, _, tol = attn_ref(c, q, 0.125)
    q[1, 0, 5], q[2, 2, 7] = np.nan, np.inf
    out, _ = run(c, q, 0.125)
    good = np.ones(q.shape[:2], bool)
    good[1, 0] = good[2, 2] = False
    assert np.all((np.abs(out - want) <= tol)[good]) and np.all(np.isnan(out[1, 0]))


@pytest.mark.parametrize("seqs,max_len", [(90, 2000), (90, 6000), (256, 5000), (257, 5000)])
def test_many_single_tokens_with_long_bounds(seqs, max_len):
    # tokens of many sequences, which the kernel takes longest first: equal lengths, idle slots and empty ones
    r = np.random.default_rng(seqs)
    lens = [int(x) for x in r.choice([0, 1, 16, 40, 150, 300], seqs)]
    news = [int(n > 0 and x > 0.1) for n, x in zip(lens, r.random(seqs))]
    news[5], lens[5] = 1, 0  # a token without a position
    c = Case(44, lens, news, 8, 64, 16)
    check(c, 8, max_len=max_len)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_len", [None, 40000])
def test_rows_between_the_kernels(dim, max_len):
    # 49 to 128 rows a sequence: a short bound goes to the split kernel in tiles of 16 rows, a long one to the
    # prompt kernel, with more chunks than the sequences have keys for
    check(Case(45, [400, 33, 16, 210], [16, 9, 16, 1], 2, dim, 32), 16, max_len=max_len)
    check(Case(46, [301], [7], 2, dim, 16), 14, window=60, max_len=max_len)
