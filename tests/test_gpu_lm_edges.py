"""Calls at the edges of the cache, attention and log probabilities: lengths past the page table, positions next to
2^31, windows of any size, scales of either sign and infinite ones,
scores of any size, single rows of any stride."""
import numpy as np
import pytest

from lm_helpers import Case, attn_ref_rows, past_the_table, write_ref
from test_gpu_attn import queries, run
from test_gpu_kv_cache import read_ref, run_write, tokens

torch = pytest.importorskip("torch")
from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu


def agree(c, heads, scale, window=0, q=None, **kw):
    """mnb_attn against the definition; returns what it gave."""
    q = queries(c, heads) if q is None else q
    want, want_lse, tol = attn_ref_rows(c, q, scale, window)
    out, lse = run(c, q, scale, window, **kw)
    assert np.all(np.isfinite(out))
    worst = np.max(np.abs(out - want) / tol)
    assert worst <= 1, f"worst error is {worst:.3g} of its tolerance"
    empty = np.isinf(want_lse)
    assert np.all(lse[empty] == -np.inf) and np.all(out[empty] == 0)
    assert np.all(np.abs(lse[~empty] - want_lse[~empty]) <= 2e-4 + 1e-6 * np.abs(want_lse[~empty]))
    return out, lse


# ---- lengths past the table: the positions keep their numbers, those without a page are missing

PAST = [  # positions past the table by sequence, new tokens
    ([1], [1]),
    ([2], [5]),
    ([16, -3, 0], [16, 1, 9]),
    ([5, -40, 33], [1, 7, 40]),
    ([500, 1], [3, 300]),          # no new token of the first has a page
]


@pytest.mark.parametrize("over,news", PAST)
def test_tokens_past_the_table_are_not_written(over, news):
    c = Case(60, [128] * len(over), news, 2, 64, 16)
    short = past_the_table(c, over)
    k, v = tokens(c, 6)
    want = write_ref(c, k, v)
    c.table = short
    got = run_write(c, k, v)
    for w in (0, 1):
        np.testing.assert_array_equal(got[0][w], want[0][w])
        np.testing.assert_array_equal(got[1][w], want[1][w])


@pytest.mark.parametrize("over,news", PAST)
def test_tokens_past_the_table_are_not_read(over, news):
    c = Case(61, [128] * len(over), news, 2, 128, 32)
    short = past_the_table(c, over)
    want = read_ref(c, 9)
    c.table = short
    cache, batch = c.upload(torch, mnb)
    k, v = (torch.full((c.T, c.H, c.D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    mnb.mnb_kv_read(cache, batch, k, v)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(v.cpu().numpy(), want[1])


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("over,news", PAST + [([1, 60], [300, 300])])
def test_attention_of_tokens_past_the_table(over, news, dim, window):
    c = Case(62, [256] * len(over), news, 1, dim, 32)
    short = past_the_table(c, over)
    q = queries(c, 3)
    want = attn_ref_rows(c, q, 0.1, window)
    c.table = short
    out, lse = run(c, q, 0.1, window)
    assert np.all(np.abs(out - want[0]) <= want[2])
    empty = np.isinf(want[1])
    assert np.all(lse[empty] == -np.inf)
    assert np.all(np.abs(lse - want[1])[~empty] <= 2e-4 + 1e-6 * np.abs(want[1][~empty]))


def test_a_decode_step_replayed_past_the_table():
    c = Case(63, [62], [1], 2, 64, 32)
    c.table = c.table[:, :2].copy()
    cache, batch = c.upload(torch, mnb)
    g = torch.Generator("cuda").manual_seed(63)
    k, v = (torch.randn(1, 2, 64, device="cuda", generator=g).half() for _ in range(2))
    q = torch.randn(1, 4, 64, device="cuda", generator=g).half()
    out = torch.empty_like(q)
    ws = mnb.attn_workspace(cache, batch, 4)
    step = lambda: (batch.kv_len.add_(1), mnb.mnb_kv_write(cache, batch, k, v),  # noqa: E731
                    mnb.mnb_attn(cache, batch, q, out, ws=ws))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()  # position 63, the table's last
    torch.cuda.synchronize()
    held = [t.clone() for t in (cache.K, cache.V, cache.K_scales, cache.V_scales)]
    full = out.clone()
    for _ in range(3):
        k.mul_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, (cache.K, cache.V, cache.K_scales, cache.V_scales)):
            assert torch.equal(a, b)
        assert torch.equal(out, full)  # the same 64 keys


# ---- positions next to 2^31: one page, over and over

FULL = 2 ** 31 - 4096  # positions that exist


def repeated_page(kv_len, tokens, max_new):
    c = Case(68, [256], [1], 1, 64, 256, spare=0)
    c.table[:] = 0
    cache, _ = c.upload(torch, mnb)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(1, 2 ** 23, dtype=torch.int32, device="cuda")
    return c, cache, mnb.KVBatch(table, i32(kv_len), i32(0, tokens), tokens, max_new, 2 ** 31 - 1)


@pytest.mark.parametrize("n", [1, 150])
def test_attention_next_to_the_last_position(n):
    # every key of the page counts 2^23 - 16 times (for the later tokens too, whose positions do not exist): the page's own
    # result.  A warp adds 2^31 / 456 / 4 / 16 products one after the other, a CTA of the prompt kernel 2^31 / 152 / 16
    kv_len = 2 ** 31 - 1
    c, cache, batch = repeated_page(kv_len, n, n)
    q = np.random.default_rng(68).standard_normal((n, 1, 64)).astype(np.float16)
    qd = torch.from_numpy(q).cuda()
    out, lse = torch.empty_like(qd), torch.empty(n, 1, device="cuda")
    mnb.mnb_attn(cache, batch, qd, out, lse=lse, ws=mnb.attn_workspace(cache, batch, 1))
    torch.cuda.synchronize()
    c.news, c.q_start = [n], np.array([0, n])
    c.lens = [256 + n]  # every token sees the whole page, and none of what follows it
    c.table = np.array([[0, -1, -1]], np.int32)
    want, want_lse, tol = attn_ref_rows(c, q, 0.125)
    adds = 2 ** 31 / (456 * 64 if n == 1 else 152 * 16)
    v = np.abs((c.codes[1][0, 0].astype(float) - 128) * c.scales[1][0, 0].repeat(16)[:, None]).max()
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol + adds * 2.0 ** -23 * v)
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse - np.log(2 ** 23 - 16)) <= 2e-4 + adds * 2.0 ** -23)


def test_writing_and_reading_next_to_the_last_position():
    c, cache, batch = repeated_page(FULL + 2, 5, 5)
    held = cache.K.clone()
    k = torch.randn(5, 1, 64, device="cuda").half()
    mnb.mnb_kv_write(cache, batch, k, k)
    back = [torch.full_like(k, 9.0) for _ in range(2)]
    mnb.mnb_kv_read(cache, batch, *back)
    torch.cuda.synchronize()
    step = cache.K_scales[0, 0, 15].item()
    assert (back[0][:3] - k[:3]).abs().max().item() <= 0.51 * step + 2e-3 and torch.all(back[0][3:] == 9)
    assert torch.equal(cache.K[:, :, :240], held[:, :, :240])


# ---- windows

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,news", [([3], [8]), ([100], [200]), ([40], [41])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60])
def test_the_largest_windows(dim, lens, news, window):
    c = Case(66, lens, news, 1, dim, 16)
    agree(c, 2, 0.125, window)


# ---- scales

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news,window", [([5], 0), ([100], 0), ([200], 0), ([200], 50), ([1], 0)])
@pytest.mark.parametrize("scale", [-0.125, 0.0, -2.0])
def test_scales_of_either_sign(dim, news, window, scale):
    c = Case(64, [230], news, 1, dim, 32)
    agree(c, 2, scale, window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news", [[1], [5], [100], [200]])
@pytest.mark.parametrize("which,max_len", [(0, None), (1, None), (0, 20000), (1, 20000)])
def test_an_infinite_key_or_value_is_seen(dim, news, which, max_len):
    # FP16's infinity among the keys or values: its block's scale is infinite, and whoever sees it gets NaN
    c = Case(65, [230], news, 2, dim, 16)
    b = 224 // 16 - (6 if news == [200] else 1)
    p = c.table[0, b]
    c.scales[which][p], c.codes[which][p] = np.inf, 128
    out, lse = run(c, queries(c, 8), dim ** -0.5, max_len=max_len)
    pos = 230 - news[0] + np.arange(news[0])
    assert np.all(np.isnan(out[pos >= b * 16])) and np.all(np.isnan(lse[pos >= b * 16]))
    assert np.all(np.isfinite(out[pos < b * 16]))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news", [[1], [5], [150]])
@pytest.mark.parametrize("size", [1e4, 6e4])
def test_scores_of_any_size(dim, news, size):
    # keys and queries at the end of FP16's range: nearly every row has one key that no rounding of the scores brings
    # down to the next one, and its value is the result
    c = Case(67, [150], news, 1, dim, 16)
    c.scales[0][:] *= np.float32(1e4)
    q = np.clip(queries(c, 2).astype(np.float64) * size, -65504, 65504).astype(np.float16)
    want, want_lse, _ = attn_ref_rows(c, q, 1.0)
    out, lse = run(c, q, 1.0)
    assert np.all(np.isfinite(out))
    assert np.all(np.abs(lse - want_lse) <= 1e-6 * np.abs(want_lse).max())
    k, v = ([c.value(w, 0, j)[0] for j in range(150)] for w in (0, 1))
    clear = 0
    for t in range(c.T):
        seen = 150 - c.T + t + 1
        for h in range(2):
            x = np.array(k[:seen]) @ q[t, h].astype(np.float64)
            step = 2.0 ** -24 * (dim + 8) * (np.abs(k[:seen]) @ np.abs(q[t, h].astype(np.float64))).max()
            best = int(x.argmax())
            if np.sort(x)[-2:-1].max(initial=-np.inf) < x[best] - 4 * step - 40:
                clear += 1
                assert np.all(np.abs(out[t, h] - v[best]) <= 2.0 ** -10 * np.abs(v[best]))
    assert clear >= 0.9 * 2 * c.T


# ---- single rows

def test_a_single_row_has_no_stride():
    # a row of a matrix whose rows are not 16 bytes apart, keys and values from different ones
    c = Case(69, [40], [1], 2, 64, 16)
    k, v = tokens(c, 7)
    want = write_ref(c, k, v)
    q = queries(c, 4)
    cache, batch = c.upload(torch, mnb)
    wide = lambda a, n: torch.zeros(1, n, dtype=torch.float16, device="cuda")[:, :a.size].copy_(  # noqa: E731
        torch.from_numpy(a).cuda().view(1, -1))
    mnb.mnb_kv_write(cache, batch, wide(k, 131), wide(v, 133))
    c.codes, c.scales = want
    back = [torch.zeros(1, n, dtype=torch.float16, device="cuda")[:, :128] for n in (141, 143)]
    mnb.mnb_kv_read(cache, batch, *back)
    out = torch.zeros(1, 259, dtype=torch.float16, device="cuda")[:, :256]
    mnb.mnb_attn(cache, batch, wide(q, 261), out)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(cache.K.cpu().numpy(), want[0][0])
    np.testing.assert_array_equal(cache.V.cpu().numpy(), want[0][1])
    for w in (0, 1):
        np.testing.assert_array_equal(back[w].cpu().numpy().reshape(1, 2, 64), read_ref(c)[w])
    want_out, _, tol = attn_ref_rows(c, q, 0.125)
    assert np.all(np.abs(out.float().cpu().numpy().reshape(1, 4, 64) - want_out) <= tol)
