"""Refusals of the rotation, mixture-of-experts and sampling calls, without a GPU: made-up addresses that are never
followed, in a child process that sees no GPU (a call that passes its checks then returns MNB_ERR_NO_DEVICE)."""
import ctypes

import numpy as np
import pytest

from step_helpers import rope_ref, sample_ref
from test_abi_host import run_without_gpu
from test_lm_ops_host import batch

from block_quantized_matmul_matmulnbits_gb300 import build as mnb_build
from block_quantized_matmul_matmulnbits_gb300 import mnb

A = 0x1000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    mnb_build.build()
    yield


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope(r=0, b=None, positions=A, tokens=5, Q=A, qs=256, qh=4, K=A, ks=128, kh=2, Qo=A, qos=256, Ko=A, kos=128, **kw):
    d = dict(head_dim=64, rotary_dim=64, interleaved=0, eps=1e-6, inv_freq=A, q_weight=A, k_weight=None)
    d = mnb.MnbRope(*{**d, **kw}.values()) if r == 0 else r
    return mnb.lib().mnb_qk_rope(ref(d), ref(b), positions, tokens, Q, qs, qh, K, ks, kh, Qo, qos, Ko, kos, None)


def moe(layer=0, X=A, M=3, Y=2 * A, ids=A, weights=A, ws=A, ws_bytes=1 << 30, **kw):
    d = dict(hidden=64, inter=96, experts=4, top_k=2, bits=4, flags=1, router=A, up_Wq=A, up_scales=A, up_zp=None,
             down_Wq=A, down_scales=A, down_zp=A)
    d = mnb.MnbMoeLayer(*{**d, **kw}.values()) if layer == 0 else layer
    return mnb.lib().mnb_moe(ref(d), X, M, Y, ids, weights, ws, ws_bytes, None)


def sample(logits=A, rows=2, vocab=100, stride=100, u=A, t=A, k=A, p=A, m=A, token=A, lp=A):
    return mnb.lib().mnb_sample(logits, rows, vocab, stride, u, t, k, p, m, token, lp, None)


def child_rope_checks():
    E = mnb
    for kw in (dict(r=None), dict(tokens=-1), dict(qh=-1), dict(kh=-1), dict(rotary_dim=-16), dict(rotary_dim=80),
               dict(interleaved=2), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(b=batch(tokens=4)),
               dict(b=batch(tokens=5, seqs=-1)), dict(qs=248), dict(qos=248), dict(qs=512), dict(kos=512), dict(ks=120), dict(kos=120), dict(Q=None),
               dict(Qo=None), dict(K=None), dict(Ko=None), dict(inv_freq=None), dict(positions=None),
               dict(b=batch(tokens=5, kv_len=None)), dict(b=batch(tokens=5, q_start=None))):
        assert rope(**kw) == E.MNB_ERR_ARG, kw
    for kw in (dict(head_dim=96), dict(head_dim=0), dict(rotary_dim=24), dict(tokens=1 << 31), dict(qh=65535)):
        assert rope(**kw) == E.MNB_ERR_UNSUPPORTED, kw
    for kw in (dict(qs=260), dict(qos=260), dict(ks=132), dict(kos=132), dict(Q=A + 8), dict(Qo=A + 2), dict(K=A + 4),
               dict(Ko=A + 8), dict(q_weight=A + 8), dict(k_weight=A + 2), dict(inv_freq=A + 2), dict(positions=A + 2),
               dict(b=batch(tokens=5, kv_len=A + 2)), dict(b=batch(tokens=5, q_start=A + 1))):
        assert rope(**kw) == E.MNB_ERR_ALIGN, kw
    for kw in (dict(tokens=0, Q=None), dict(qh=0, kh=0, Q=None), dict(b=batch(tokens=5, seqs=0))):
        assert rope(**kw) == E.MNB_OK, kw
    for kw in (dict(), dict(b=batch(tokens=5, page_table=None, max_pages=0), positions=None), dict(kh=0, K=None, Ko=None),
               dict(qh=0, Q=None, Qo=None), dict(rotary_dim=0, inv_freq=None), dict(qh=65534, qs=1 << 23, qos=1 << 23), dict(qs=512, Qo=2 * A),
               dict(tokens=1, qs=512, b=batch(tokens=1)), dict(qs=512, qos=512)):
        assert rope(**kw) == E.MNB_ERR_NO_DEVICE, kw


def child_moe_checks():
    E = mnb
    for kw in (dict(layer=None), dict(M=-1), dict(hidden=0), dict(inter=-32), dict(experts=0), dict(top_k=0),
               dict(top_k=5), dict(flags=2), dict(X=None), dict(Y=None), dict(X=A, Y=A), dict(router=None),
               dict(up_Wq=None), dict(up_scales=None), dict(down_Wq=None), dict(down_scales=None), dict(ws=None),
               dict(ws_bytes=-1), dict(ws_bytes=100)):
        assert moe(**kw) == E.MNB_ERR_ARG, kw
    for kw in (dict(hidden=48), dict(inter=16), dict(hidden=1 << 16), dict(inter=1 << 17), dict(experts=257),
               dict(experts=256, top_k=17), dict(bits=2), dict(bits=5), dict(M=17)):
        assert moe(**kw) == E.MNB_ERR_UNSUPPORTED, kw
    for kw in (dict(X=A + 8), dict(Y=A + 2), dict(router=A + 4), dict(up_Wq=A + 8), dict(up_scales=A + 2),
               dict(down_Wq=A + 8), dict(down_scales=A + 2), dict(up_zp=A + 1), dict(down_zp=A + 2), dict(ids=A + 2),
               dict(weights=A + 1), dict(ws=A + 8)):
        assert moe(**kw) == E.MNB_ERR_ALIGN, kw
    assert moe(M=0, X=None, Y=None, ws=None, ws_bytes=0) == E.MNB_OK
    assert moe() == moe(ids=None, weights=None, flags=0, bits=8) == E.MNB_ERR_NO_DEVICE
    layer = mnb.MnbMoeLayer(64, 96, 4, 2, 4, 1)
    size = lambda M: mnb.lib().mnb_moe_workspace(ctypes.byref(layer), M)  # noqa: E731
    assert 0 <= size(0) < size(1) <= size(16) and size(17) == E.MNB_ERR_UNSUPPORTED and size(-1) == E.MNB_ERR_ARG
    assert mnb.lib().mnb_moe_workspace(None, 1) == E.MNB_ERR_ARG
    assert moe(ws_bytes=size(3)) == E.MNB_ERR_NO_DEVICE and moe(ws_bytes=size(3) - 1) == E.MNB_ERR_ARG


def child_sample_checks():
    E = mnb
    for kw in (dict(rows=-1), dict(vocab=0), dict(stride=99), dict(logits=None), dict(u=None), dict(token=None)):
        assert sample(**kw) == E.MNB_ERR_ARG, kw
    for kw in (dict(vocab=(1 << 24) + 1, stride=1 << 25), dict(rows=1 << 40)):
        assert sample(**kw) == E.MNB_ERR_UNSUPPORTED, kw
    for kw in (dict(logits=A + 2), dict(u=A + 2), dict(t=A + 1), dict(k=A + 2), dict(p=A + 2), dict(m=A + 3),
               dict(token=A + 4), dict(lp=A + 2)):
        assert sample(**kw) == E.MNB_ERR_ALIGN, kw
    assert sample(rows=0, logits=None) == E.MNB_OK
    assert sample() == sample(t=None, k=None, p=None, m=None, lp=None) == E.MNB_ERR_NO_DEVICE


@pytest.mark.parametrize("fn", [child_rope_checks, child_moe_checks, child_sample_checks])
def test_refusals(fn):
    run_without_gpu(fn)


def test_the_binding_checks_its_tensors():
    torch = pytest.importorskip("torch")
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for bad in (dict(inv_freq=torch.zeros(4).double()), dict(inv_freq=torch.zeros(2, 2)), dict(q_weight=h(32)),
                dict(k_weight=torch.zeros(64)), dict(q_weight=h(128)[::2])):
        with pytest.raises(ValueError):
            mnb.Rope(64, **bad)
    with pytest.raises(mnb.MnbError):  # host tensors
        mnb.mnb_qk_rope(mnb.Rope(64), i32(3), h(3, 2, 64))
    E, K, I = 4, 64, 96
    good = dict(router=h(E, K), up_Wq=torch.zeros(E, 2 * I, 2, 16, dtype=torch.uint8), up_scales=h(E, 2 * I, 2),
                down_Wq=torch.zeros(E, K, 3, 16, dtype=torch.uint8), down_scales=h(E, K, 3), top_k=2)
    layer = mnb.MoE(**good)
    assert mnb.mnb_moe_workspace(layer, 16) > 0
    with pytest.raises(mnb.MnbError):
        mnb.mnb_moe_workspace(layer, 17)
    for bad in (dict(router=torch.zeros(E, K)), dict(up_scales=h(E, 2 * I, 3)), dict(down_scales=h(E, K, 2)), dict(bits=8),
                dict(up_zp=torch.zeros(E, 2 * I, 2)), dict(down_zp=torch.zeros(E, K, 2, dtype=torch.uint8)),
                dict(up_scales=h(E, 2 * I, 4)[..., ::2])):
        with pytest.raises(ValueError):
            mnb.MoE(**{**good, **bad})
    for X, Y, kw in ((h(3, 32), h(3, 32), {}), (h(3, 64), h(2, 64), {}), (h(3, 64), h(3, 128)[:, ::2], {}),
                     (h(3, 64), h(3, 64), dict(ids=i32(3, 1))), (h(3, 64), h(3, 64), dict(weights=h(3, 2)))):
        with pytest.raises(ValueError):
            mnb.mnb_moe(layer, X, Y, **kw)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_moe(layer, h(3, 64), h(3, 64), stream=0)
    x, u, token = h(3, 9), torch.zeros(3), torch.zeros(3, dtype=torch.int64)
    for kw in (dict(u=torch.zeros(2)), dict(token=i32(3)), dict(top_k=torch.zeros(3)), dict(top_p=torch.zeros(3).double()),
               dict(min_p=torch.zeros(6)[::2]), dict(temperature=h(3)), dict(logits=x.float()), dict(logprob=h(3))):
        d = {**dict(logits=x, u=u, token=token), **kw}
        with pytest.raises((ValueError, mnb.MnbError)):
            mnb.mnb_sample(d.pop("logits"), d.pop("u"), d.pop("token"), stream=0, **d)


def test_the_references():
    # a quarter turn, in both orders; the angle of a far position against an exact product
    x = np.arange(64, dtype=np.float16)[None, None] + np.float16(1)
    f = np.full(32, np.float32(np.pi / 2))
    out, tol = rope_ref(x, [1], f)
    assert np.allclose(out[0, 0, :32], -x[0, 0, 32:], atol=1e-4) and np.allclose(out[0, 0, 32:], x[0, 0, :32], atol=1e-4)
    out, _ = rope_ref(x, [1], f, True)
    assert np.allclose(out[0, 0, ::2], -x[0, 0, 1::2], atol=1e-4)
    one = np.zeros((1, 1, 64), np.float16)
    one[0, 0, 0] = 1
    out, _ = rope_ref(one, [1 << 20], np.full(32, np.float32(1.0)))
    assert abs(out[0, 0, 0] - np.cos(float(1 << 20))) < 1e-9
    row = np.array([1, 3, 3, 0], np.float16)
    w = np.exp([0.0, 0.0, -2.0, -3.0])  # tokens 1, 2, 0, 3: they end at 0.458, 0.915, 0.977 and 1
    for u, want in ((0.0, 1), (0.46, 2), (0.95, 0), (0.999, 3)):
        assert sample_ref(row, u)[0] == want
    assert sample_ref(row, 0.999, top_k=3)[0] == 0 and sample_ref(row, 0.999, top_p=0.5)[0] == 2
    assert abs(sample_ref(row, 0.999, min_p=0.1)[1] - np.log(w[2] / w[:3].sum())) < 1e-12
