"""Refusals of the cache, attention and log-probability calls, without a GPU: made-up addresses that are
never followed, in a child process that sees no GPU (a call that passes its checks then returns
MNB_ERR_NO_DEVICE)."""
import ctypes

import pytest

from test_abi_host import run_without_gpu

from block_quantized_matmul_matmulnbits_gb300 import build as mnb_build
from block_quantized_matmul_matmulnbits_gb300 import mnb

A = 0x1000


@pytest.fixture(scope="module", autouse=True)
def built():
    mnb_build.build()
    yield


def cache(**kw):
    d = dict(num_pages=8, page_size=16, kv_heads=2, head_dim=64, reserved=0, K=A, V=A, K_scales=A, V_scales=A)
    return mnb.MnbKvCache(*{**d, **kw}.values())


def batch(**kw):
    d = dict(seqs=2, max_pages=4, tokens=5, max_new=4, max_len=60, page_table=A, kv_len=A, q_start=A)
    return mnb.MnbKvBatch(*{**d, **kw}.values())


def kv(fn, c=None, b=None, K=A, V=A, stride=128):
    ref = lambda x: None if x == 0 else ctypes.byref(x)  # noqa: E731
    return getattr(mnb.lib(), fn)(ref(cache() if c is None else c), ref(batch() if b is None else b), K, V, stride,
                                  None)


def attn(c=None, b=None, Q=A, q_stride=256, q_heads=4, window=0, out=A, out_stride=256, lse=None, ws=A, ws_bytes=0):
    return mnb.lib().mnb_attn(ctypes.byref(c or cache()), ctypes.byref(b or batch()), Q, q_stride, q_heads, 0.1,
                              window, out, out_stride, lse, ws, ws_bytes, None)


def logprobs(logits=A, rows=2, vocab=100, stride=100, scale=1.0, target=A, top=3, logprob=A, entropy=A, ids=A, tops=A):
    return mnb.lib().mnb_logprobs(logits, rows, vocab, stride, scale, target, top, logprob, entropy, ids, tops, None)


def child_shared_checks():
    E = mnb
    bad = [(dict(c=0), E.MNB_ERR_ARG), (dict(b=0), E.MNB_ERR_ARG)]
    for kw, code in ((dict(num_pages=-1), E.MNB_ERR_ARG), (dict(kv_heads=0), E.MNB_ERR_ARG),
                     (dict(reserved=1), E.MNB_ERR_ARG), (dict(K=None), E.MNB_ERR_ARG), (dict(V=None), E.MNB_ERR_ARG),
                     (dict(K_scales=None), E.MNB_ERR_ARG), (dict(V_scales=None), E.MNB_ERR_ARG),
                     (dict(page_size=8), E.MNB_ERR_UNSUPPORTED), (dict(page_size=48), E.MNB_ERR_UNSUPPORTED),
                     (dict(page_size=512), E.MNB_ERR_UNSUPPORTED), (dict(head_dim=96), E.MNB_ERR_UNSUPPORTED),
                     (dict(kv_heads=1 << 17), E.MNB_ERR_UNSUPPORTED), (dict(num_pages=1 << 40), E.MNB_ERR_UNSUPPORTED),
                     (dict(K=A + 8), E.MNB_ERR_ALIGN), (dict(V_scales=A + 4), E.MNB_ERR_ALIGN)):
        bad.append((dict(c=cache(**kw)), code))
    for kw, code in ((dict(seqs=-1), E.MNB_ERR_ARG), (dict(tokens=-1), E.MNB_ERR_ARG), (dict(max_new=-1), E.MNB_ERR_ARG),
                     (dict(max_len=-1), E.MNB_ERR_ARG), (dict(max_pages=-1), E.MNB_ERR_ARG),
                     (dict(page_table=None), E.MNB_ERR_ARG), (dict(kv_len=None), E.MNB_ERR_ARG),
                     (dict(q_start=None), E.MNB_ERR_ARG), (dict(tokens=1 << 40), E.MNB_ERR_UNSUPPORTED),
                     (dict(kv_len=A + 2), E.MNB_ERR_ALIGN)):
        bad.append((dict(b=batch(**kw)), code))
    for fn in ("mnb_kv_write", "mnb_kv_read"):
        for kw, code in bad:
            assert kv(fn, **kw) == code, (fn, kw, code)
        assert kv(fn, K=None) == kv(fn, V=None) == E.MNB_ERR_ARG
        assert kv(fn, stride=127) == E.MNB_ERR_ARG and kv(fn, stride=129) == E.MNB_ERR_ALIGN
        assert kv(fn, K=A + 2) == E.MNB_ERR_ALIGN
        for kw in (dict(b=batch(seqs=0)), dict(b=batch(tokens=0)), dict(b=batch(max_pages=0)),
                   dict(c=cache(num_pages=0))):
            assert kv(fn, **kw) == E.MNB_OK  # nothing to do
        assert kv(fn) == E.MNB_ERR_NO_DEVICE
    for kw, code in bad[2:]:
        assert attn(**kw) == code, (kw, code)
    L = mnb.lib()
    assert L.mnb_attn(None, ctypes.byref(batch()), A, 256, 4, 0.1, 0, A, 256, None, A, 0, None) == E.MNB_ERR_ARG
    assert L.mnb_attn_workspace(None, ctypes.byref(batch()), 4, 0, 152) == E.MNB_ERR_ARG


def child_attn_checks():
    E = mnb
    assert attn(q_heads=0) == attn(window=-1) == attn(q_stride=255) == attn(out_stride=128) == E.MNB_ERR_ARG
    assert attn(Q=None) == attn(out=None) == attn(ws_bytes=-1) == E.MNB_ERR_ARG
    assert attn(q_heads=3) == E.MNB_ERR_UNSUPPORTED
    assert attn(q_stride=260) == attn(out_stride=260) == E.MNB_ERR_ALIGN
    assert attn(Q=A + 2) == attn(out=A + 2) == attn(lse=A + 1) == attn(ws=A + 4) == E.MNB_ERR_ALIGN
    assert attn(b=batch(tokens=0), Q=None) == attn(b=batch(seqs=0)) == E.MNB_OK
    assert attn() == E.MNB_ERR_NO_DEVICE
    # without pages the tensors of the cache may be missing: the rows see nothing
    assert attn(c=cache(num_pages=0, K=None, V=None), b=batch(page_table=None)) == E.MNB_ERR_NO_DEVICE
    ws = lambda **kw: mnb.lib().mnb_attn_workspace(ctypes.byref(cache()), ctypes.byref(batch(**kw)), 4, 0, 152)  # noqa: E731
    assert ws() == 0 and ws(tokens=0) == 0
    assert ws(seqs=1, tokens=1, max_new=1, max_len=100000, max_pages=7000) > 0


def child_logprobs_checks():
    E = mnb
    for kw in (dict(rows=-1), dict(vocab=0), dict(stride=99), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(top=-1), dict(top=101), dict(logits=None),
               dict(logprob=None), dict(ids=None), dict(tops=None)):
        assert logprobs(**kw) == E.MNB_ERR_ARG, kw
    for kw in (dict(vocab=(1 << 24) + 1, stride=1 << 25), dict(top=33), dict(rows=1 << 40)):
        assert logprobs(**kw) == E.MNB_ERR_UNSUPPORTED, kw
    for kw in (dict(logits=A + 2), dict(target=A + 4), dict(logprob=A + 2), dict(ids=A + 1), dict(tops=A + 2),
               dict(entropy=A + 2)):
        assert logprobs(**kw) == E.MNB_ERR_ALIGN, kw
    assert logprobs(rows=0, logits=None) == E.MNB_OK
    assert logprobs() == E.MNB_ERR_NO_DEVICE
    assert logprobs(target=None, logprob=None, entropy=None, top=0, ids=None, tops=None) == E.MNB_ERR_NO_DEVICE


@pytest.mark.parametrize("fn", [child_shared_checks, child_attn_checks, child_logprobs_checks])
def test_refusals(fn):
    run_without_gpu(fn)


def test_the_binding_checks_its_tensors():
    torch = pytest.importorskip("torch")
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k, s = u8(4, 2, 32, 64), torch.zeros(4, 2, 2)
    c = mnb.KVCache(k, k.clone(), s, s.clone())
    for bad in ((k, u8(4, 2, 32, 128), s, s), (k, k, torch.zeros(4, 2, 1), s), (k, k, s.double(), s),
                (k.float(), k, s, s), (k.transpose(0, 1), k.transpose(0, 1), s, s)):
        with pytest.raises(ValueError):
            mnb.KVCache(*bad)
    b = mnb.KVBatch(i32(2, 3), i32(2), i32(3), 4, 2, 50)
    for bad in ((i32(3, 3), i32(2), i32(3)), (i32(2, 3), i32(2), i32(2)), (i32(2, 3).long(), i32(2), i32(3)),
                (i32(2, 6)[:, ::2], i32(2), i32(3))):
        with pytest.raises(ValueError):
            mnb.KVBatch(*bad, 4, 2, 50)
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    for K, V in ((h(4, 2, 32), h(4, 2, 64)), (h(3, 2, 64), h(3, 2, 64)), (h(4, 2, 64).bfloat16(), h(4, 2, 64)),
                 (h(4, 4, 64)[:, ::2], h(4, 2, 64)), (h(4, 256)[:, :128], h(4, 2, 64))):
        for fn in (mnb.mnb_kv_write, mnb.mnb_kv_read):
            with pytest.raises(ValueError):
                fn(c, b, K, V, stream=0)
    with pytest.raises(ValueError):
        mnb.mnb_attn(c, b, h(4, 4, 64), h(4, 4, 64), lse=torch.zeros(4, 2), stream=0)
    with pytest.raises(ValueError):
        mnb.mnb_logprobs(torch.zeros(2, 5), stream=0)


@pytest.mark.parametrize("bad", [dict(target="int32"), dict(logprob="float16"), dict(entropy="rows"),
                                 dict(top_ids="strided"), dict(top_logprobs="k")])
def test_the_binding_checks_what_log_probabilities_go_into(bad):
    torch = pytest.importorskip("torch")
    given = dict(target=torch.zeros(3, dtype=torch.int64), logprob=torch.zeros(3), entropy=torch.zeros(3),
                 top_ids=torch.zeros(3, 2, dtype=torch.int32), top_logprobs=torch.zeros(3, 2))
    wrong = dict(int32=torch.zeros(3, dtype=torch.int32), float16=torch.zeros(3, dtype=torch.float16),
                 rows=torch.zeros(2), strided=torch.zeros(3, 4, dtype=torch.int32)[:, ::2], k=torch.zeros(3, 1))
    name, how = next(iter(bad.items()))
    with pytest.raises(ValueError):
        mnb.mnb_logprobs(torch.zeros(3, 9, dtype=torch.float16), **{**given, name: wrong[how]}, stream=0)
