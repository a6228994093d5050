"""mnb_kv_write and mnb_kv_read against their definition, step by step in binary32: codes, scales and
values have to be equal."""
import numpy as np
import pytest

from lm_helpers import Case, write_ref

torch = pytest.importorskip("torch")
from block_quantized_matmul_matmulnbits_gb300 import mnb  # noqa: E402

pytestmark = pytest.mark.gpu


def tokens(c, seed=0, scale=1.0):
    r = np.random.default_rng(seed + 77)
    return [(r.standard_normal((c.T, c.H, c.D)) * scale).astype(np.float16) for _ in range(2)]


def run_write(c, k, v, stream=None):
    cache, batch = c.upload(torch, mnb)
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    torch.cuda.synchronize()
    mnb.mnb_kv_write(cache, batch, kd, vd, stream=stream)
    torch.cuda.synchronize()
    return [cache.K.cpu().numpy(), cache.V.cpu().numpy()], [cache.K_scales.cpu().numpy(), cache.V_scales.cpu().numpy()]


def check_write(c, k, v, **kw):
    codes, scales = run_write(c, k, v, **kw)
    want_codes, want_scales = write_ref(c, k, v)
    for w in (0, 1):
        np.testing.assert_array_equal(scales[w], want_scales[w])
        np.testing.assert_array_equal(codes[w], want_codes[w])


SHAPES = [  # lens, news, heads, dim, page
    ([1], [1], 1, 64, 16),
    ([16], [16], 3, 64, 16),
    ([17], [1], 3, 64, 16),
    ([100], [1], 8, 128, 64),
    ([31, 0, 5, 64], [3, 0, 5, 1], 2, 128, 32),
    ([333, 47, 16], [300, 47, 2], 2, 64, 128),
    ([700], [18], 1, 128, 256),
    ([15, 31, 48, 1] * 20, [1] * 80, 2, 64, 16),
    ([9, 25] * 600, [2, 0] * 600, 1, 64, 16),      # more sequences than one round of the search
    ([40, 3], [40, 8], 2, 64, 16),                 # five tokens before position 0 are left out
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_write_is_the_definition(i):
    lens, news, H, D, P = SHAPES[i]
    c = Case(i, lens, news, H, D, P)
    check_write(c, *tokens(c, i))


def test_growing_and_kept_scales():
    # small tokens keep the block's scale, large ones make the older codes follow
    for scale in (1e-3, 30.0):
        c = Case(3, [37, 90], [3, 1], 4, 128, 32)
        check_write(c, *tokens(c, 1, scale))


def test_zeros_subnormals_and_non_finite():
    c = Case(4, [20, 33, 64], [20, 33, 40], 2, 64, 16)
    k, v = tokens(c, 2)
    k[:16] = 0
    v[:] *= np.float16(2.0 ** -24)   # FP16 subnormals
    k[25, 1, 5] = np.nan
    k[60, 0, 3] = np.inf
    check_write(c, k, v)


def test_writing_again_changes_nothing():
    c = Case(5, [45, 20], [9, 20], 2, 128, 16)
    k, v = tokens(c, 3, 20.0)
    cache, batch = c.upload(torch, mnb)
    kd, vd = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    mnb.mnb_kv_write(cache, batch, kd, vd)
    first = [t.clone() for t in (cache.K, cache.V, cache.K_scales, cache.V_scales)]
    mnb.mnb_kv_write(cache, batch, kd, vd)
    torch.cuda.synchronize()
    for a, b in zip(first, (cache.K, cache.V, cache.K_scales, cache.V_scales)):
        assert torch.equal(a, b)


def test_one_token_at_a_time():
    # growing the sequence token by token: each step is the definition on the cache before it
    c = Case(6, [1], [1], 2, 64, 16, spare=4)
    c.table[:, :2] = [[0, 1]]
    r = np.random.default_rng(8)
    for length in range(1, 21):
        c.lens, c.news = [length], [1]
        k, v = ((r.standard_normal((1, 2, 64)) * length).astype(np.float16) for _ in range(2))
        codes, scales = run_write(c, k, v)
        want = write_ref(c, k, v)
        for w in (0, 1):
            np.testing.assert_array_equal(codes[w], want[0][w])
            np.testing.assert_array_equal(scales[w], want[1][w])
        c.codes, c.scales = codes, scales


def test_pages_outside_the_cache_are_skipped():
    c = Case(7, [40, 40], [40, 3], 2, 64, 16)
    c.table[0, 1] = -1
    c.table[1, 2] = c.pages
    check_write(c, *tokens(c, 4))


def test_strided_rows_and_another_stream():
    c = Case(8, [50, 7], [30, 7], 2, 64, 16)
    k, v = tokens(c, 5)
    cache, batch = c.upload(torch, mnb)
    fused = torch.zeros(c.T, 5 * 64 + 2 * 2 * 64, dtype=torch.float16, device="cuda")
    fused[:, 320:448] = torch.from_numpy(k).cuda().view(c.T, -1)
    fused[:, 448:] = torch.from_numpy(v).cuda().view(c.T, -1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mnb.mnb_kv_write(cache, batch, fused[:, 320:448], fused[:, 448:], stream=side)
    back = torch.zeros_like(fused)
    side.wait_stream(torch.cuda.current_stream())
    mnb.mnb_kv_read(cache, batch, back[:, 320:448], back[:, 448:], stream=side)
    side.synchronize()
    codes, scales = write_ref(c, k, v)
    np.testing.assert_array_equal(cache.K.cpu().numpy(), codes[0])
    np.testing.assert_array_equal(cache.V.cpu().numpy(), codes[1])
    assert torch.all(back[:, :320] == 0)
    c.codes, c.scales = codes, scales
    want = read_ref(c)
    np.testing.assert_array_equal(back[:, 320:448].cpu().numpy().reshape(want[0].shape), want[0])
    np.testing.assert_array_equal(back[:, 448:].cpu().numpy().reshape(want[1].shape), want[1])


def read_ref(c, fill=0):
    got = [np.full((c.T, c.H, c.D), fill, np.float16) for _ in range(2)]
    for s, (n, length) in enumerate(zip(c.news, c.lens)):
        for i in range(n):
            pos = length - n + i
            for w in (0, 1):
                x = c.value(w, s, pos) if pos >= 0 else None
                if x is not None:  # (q - 128) * scale fits 64 bits exactly: one rounding to binary32, one to FP16
                    got[w][c.q_start[s] + i] = x.astype(np.float32).astype(np.float16)
    return got


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_read_is_the_definition(i):
    lens, news, H, D, P = SHAPES[i]
    c = Case(50 + i, lens, news, H, D, P)
    if i == 5:
        c.table[1, 0] = 10 ** 6
    cache, batch = c.upload(torch, mnb)
    k, v = (torch.full((c.T, H, D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    mnb.mnb_kv_read(cache, batch, k, v)
    torch.cuda.synchronize()
    want = read_ref(c, 9)
    np.testing.assert_array_equal(k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(v.cpu().numpy(), want[1])


def test_offsets_past_32_bits():
    # the sequence's pages lie past 2^32 code bytes
    H, D, P = 8, 128, 256
    pages = (1 << 32) // (H * P * D) + 4
    cache = mnb.KVCache(*(torch.empty(pages, H, P, D, dtype=torch.uint8, device="cuda") for _ in range(2)),
                        *(torch.empty(pages, H, P // 16, device="cuda") for _ in range(2)))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = mnb.KVBatch(i32(pages - 1, pages - 3).view(1, 2), i32(300), i32(0, 300), 300, 300, 300)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(300, H, D, device="cuda", generator=g, dtype=torch.float16)
    k, v = torch.empty_like(x), torch.empty_like(x)
    mnb.mnb_kv_write(cache, batch, x, -x)
    mnb.mnb_kv_read(cache, batch, k, v)
    assert torch.equal(k, -v)
    # half a step of the block's scale, and the FP16 rounding
    step = torch.nn.functional.pad(x.abs().float(), (0, 0, 0, 0, 0, 4)).view(19, 16, H, D).amax((1, 3)) / 127
    step = step.repeat_interleave(16, 0)[:300, :, None]
    assert torch.all((k.float() - x.float()).abs() <= 0.5001 * step + x.abs().float() * 2.0 ** -10)
