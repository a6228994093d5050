"""The prompt kernel of mnb_attn with one row tile a CTA and with two, whole and in chunks: parity with the definition,
and what a tile may meet (rising scores, bad scales, bad query rows, missing pages).  The plans of the cases are
pinned in test_lm_edges_host.py."""
import numpy as np
import pytest

import prompt_cases
from lm_helpers import Case, attn_ref_rows
from test_gpu_attn import queries, run
from test_gpu_lm_edges import agree

torch = pytest.importorskip("torch")
from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu

both_dims = pytest.mark.parametrize("dim", [64, 128])
tiles = pytest.mark.parametrize("name", ["two tiles, whole", "two tiles, chunks", "one tile, whole", "one tile, chunks"])


def make(name, dim, seed):
    p = prompt_cases.BY_NAME[name]
    return p, Case(seed, p.lens, p.news, p.kv_heads, dim, 32)


@both_dims
@pytest.mark.parametrize("name", prompt_cases.BY_NAME)
def test_prompts_are_the_definition(name, dim):
    p, c = make(name, dim, 80)
    agree(c, p.kv_heads * p.group, dim ** -0.5, p.window)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = mnb.mnb_attn_plan(c.cache, c.batch, p.kv_heads * p.group, p.window)
    assert sms != 152 or (plan["prompt_rows"], plan["splits"] > 1) == (p.rows, p.chunks), plan


@both_dims
@tiles
def test_rising_scores(name, dim):
    # the reference moves with every tile of keys, in the end by more than binary32's range of 2^x
    p, c = make(name, dim, 81)
    r = np.random.default_rng(81)
    last = -(-p.lens[0] // 32)
    for b in range(last):
        page = c.table[0, b]
        c.codes[0][page] = r.integers(200, 256, c.codes[0][page].shape, dtype=np.uint8)
        c.scales[0][page] = 0.2 * b / last
    agree(c, p.kv_heads * p.group, 0.3, q=np.abs(queries(c, p.kv_heads * p.group)))


@both_dims
@tiles
@pytest.mark.parametrize("which,bad", [(0, np.nan), (0, np.inf), (1, np.nan), (1, np.inf)])
def test_a_bad_block_is_seen_by_the_rows_behind_it(name, dim, which, bad):
    p, c = make(name, dim, 82)
    heads = p.kv_heads * p.group
    first = p.lens[0] - p.news[0]
    b = (first + p.news[0] // 2) // 16
    q = queries(c, heads)
    want, _, tol = attn_ref_rows(c, q, dim ** -0.5)
    page, blk = c.table[0, b // 2], b % 2
    c.scales[which][page, :, blk] = bad
    if bad == np.inf:
        c.codes[which][page, :, 16 * blk:16 * blk + 16] = 128
    out, lse = run(c, q, dim ** -0.5)
    before = first + np.arange(p.news[0]) < 16 * b
    assert np.all((np.abs(out - want) <= tol)[before])
    assert np.all(np.isnan(out[~before])) and np.all(np.isnan(lse[~before]))


@both_dims
@tiles
def test_bad_query_rows_stay_alone(name, dim):
    p, c = make(name, dim, 83)
    heads = p.kv_heads * p.group
    q = queries(c, heads)
    want, _, tol = attn_ref_rows(c, q, dim ** -0.5)
    good = np.ones(q.shape[:2], bool)
    for t, h, value in ((1, 0, np.nan), (2, heads - 1, np.inf), (p.news[0] - 1, 1, -np.inf), (p.news[0] // 2, 0, np.nan)):
        q[t, h, 5], good[t, h] = value, False
    out, _ = run(c, q, dim ** -0.5)
    assert np.all((np.abs(out - want) <= tol)[good]) and np.all(np.isnan(out[1, 0]))


@both_dims
@tiles
def test_missing_pages_between_others(name, dim):
    # page numbers outside the cache: in a tile of keys that every row sees wholly, and in one on the diagonal
    p, c = make(name, dim, 84)
    last = (p.lens[0] - 1) // 32
    c.table[0, 1], c.table[0, 2], c.table[0, last - 1] = -5, c.pages, 2 ** 31 - 1
    agree(c, p.kv_heads * p.group, dim ** -0.5)


@both_dims
@pytest.mark.parametrize("name", ["two tiles, window", "two tiles, chunks and window", "one tile, window"])
def test_blocks_outside_the_windows_may_hold_anything(name, dim):
    p, c = make(name, dim, 85)
    heads = p.kv_heads * p.group
    q = queries(c, heads)
    want, _, tol = attn_ref_rows(c, q, dim ** -0.5, p.window)
    used = np.zeros((c.pages, 2), bool)
    for b in range(max(0, p.lens[0] - p.news[0] - p.window + 1) // 16, -(-p.lens[0] // 16)):
        used[c.table[0, b // 2], b % 2] = True
    for w in (0, 1):
        for bad, share in ((np.nan, 0), (np.inf, 1)):
            hide = ~used & (np.arange(c.pages)[:, None] % 2 == share)
            c.scales[w][np.broadcast_to(hide[:, None], c.scales[w].shape)] = bad
    out, lse = run(c, q, dim ** -0.5, p.window)
    assert np.all(np.abs(out - want) <= tol) and np.all(np.isfinite(lse))


@both_dims
@pytest.mark.parametrize("name", ["two tiles, whole", "two tiles, chunks", "one tile, whole"])
def test_value_scales_over_many_orders(name, dim):
    p = prompt_cases.BY_NAME[name]
    c = Case(86, p.lens, p.news, p.kv_heads, dim, 32, v_spread=True)
    for page in (0, 3):
        c.scales[1][page], c.codes[1][page] = 0, 128
    agree(c, p.kv_heads * p.group, dim ** -0.5)


@both_dims
@pytest.mark.parametrize("name", ["two tiles, whole", "two tiles, window", "one tile, whole"])
@pytest.mark.parametrize("scale", [-0.125, 0.0])
def test_scales_that_are_not_positive(name, dim, scale):
    p, c = make(name, dim, 87)
    agree(c, p.kv_heads * p.group, scale, p.window)


def test_strided_rows_on_another_stream():
    p, c = make("two tiles, ragged", 64, 88)
    width = p.kv_heads * p.group * 64
    q = queries(c, p.kv_heads * p.group)
    want, _, tol = attn_ref_rows(c, q, 0.125)
    cache, batch = c.upload(torch, mnb)
    fused = torch.full((c.T, width + 1024), float("nan"), dtype=torch.float16, device="cuda")
    fused[:, 512:512 + width] = torch.from_numpy(q).cuda().view(c.T, -1)
    wide = torch.full((c.T, width + 64), 3.0, dtype=torch.float16, device="cuda")
    ws = mnb.attn_workspace(cache, batch, p.kv_heads * p.group)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mnb.mnb_attn(cache, batch, fused[:, 512:512 + width], wide[:, 64:], ws=ws, stream=side)
    side.synchronize()
    got = wide[:, 64:].float().cpu().numpy().reshape(want.shape)
    assert np.all(np.abs(got - want) <= tol) and torch.all(wide[:, :64] == 3)
