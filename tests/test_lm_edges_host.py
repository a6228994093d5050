"""Refusals and checks of the cache, attention and log-probability calls at their edges, without a GPU."""
import ctypes

import pytest

from test_abi_host import run_without_gpu
from test_lm_ops_host import A, batch, cache, logprobs
import prompt_cases

from block_quantized_matmul_matmulnbits_gb300 import build as mnb_build
from block_quantized_matmul_matmulnbits_gb300 import mnb


@pytest.fixture(scope="module", autouse=True)
def built():
    mnb_build.build()
    yield


def attn_scaled(scale):
    return mnb.lib().mnb_attn(ctypes.byref(cache()), ctypes.byref(batch()), A, 256, 4, scale, 0, A, 256, None, A, 0,
                              None)


def child_attn_scale():
    for scale in (float("nan"), float("inf"), -float("inf"), 1e28, -3e38):
        assert attn_scaled(scale) == mnb.MNB_ERR_ARG, scale
    for scale in (0.0, -0.0, 0.125, -0.125, 1e27, -1e27, 1e-40):
        assert attn_scaled(scale) == mnb.MNB_ERR_NO_DEVICE, scale


def test_attention_refuses_scales_that_are_not_finite():
    run_without_gpu(child_attn_scale)



def child_logprobs_scale():
    for scale in (2.1e38, 3e38, 3.4e38, -0.0):
        assert logprobs(scale=scale) == mnb.MNB_ERR_ARG, scale
    for scale in (2e38, 1e-40):
        assert logprobs(scale=scale) == mnb.MNB_ERR_NO_DEVICE, scale


def test_log_probabilities_refuse_scales_past_binary32():
    run_without_gpu(child_logprobs_scale)



@pytest.mark.parametrize("name,dtype,shape", [("target", "float64", (3,)), ("target", "int32", (3, 2)),
                                              ("logprob", "int32", (3,)), ("logprob", "float16", (3, 2)),
                                              ("entropy", "int32", (3,)), ("top_ids", "float32", (3, 2)),
                                              ("top_ids", "int64", (3, 1)), ("top_logprobs", "int32", (3, 2))])
def test_the_binding_checks_types_of_the_same_size(name, dtype, shape):
    torch = pytest.importorskip("torch")
    given = dict(target=torch.zeros(3, dtype=torch.int64), logprob=torch.zeros(3), entropy=torch.zeros(3),
                 top_ids=torch.zeros(3, 2, dtype=torch.int32), top_logprobs=torch.zeros(3, 2))
    if name == "top_ids" and dtype == "int64":
        given["top_logprobs"] = torch.zeros(3, 1)
    given[name] = torch.zeros(*shape, dtype=getattr(torch, dtype))
    with pytest.raises(ValueError):
        mnb.mnb_logprobs(torch.zeros(3, 9, dtype=torch.float16), **given, stream=0)


def host_cache(torch, heads=2, dim=64):
    codes, scales = torch.zeros(4, heads, 32, dim, dtype=torch.uint8), torch.zeros(4, heads, 2)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return mnb.KVCache(codes, codes.clone(), scales, scales.clone()), mnb.KVBatch(i32(2, 3), i32(2), i32(3), 4, 2, 50)


@pytest.mark.parametrize("dtype,shape", [("int32", (4, 4)), ("float16", (4, 8)), ("float64", (4, 2))])
def test_the_binding_checks_the_type_of_the_sums(dtype, shape):
    torch = pytest.importorskip("torch")
    c, b = host_cache(torch)
    q = torch.zeros(4, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        mnb.mnb_attn(c, b, q, q.clone(), lse=torch.zeros(*shape, dtype=getattr(torch, dtype)), stream=0)



def refused(call):
    with pytest.raises(mnb.MnbError) as e:
        call()
    return e.value.code == mnb.MNB_ERR_ARG and "on the same GPU" in str(e.value)


def test_host_tensors_never_reach_a_kernel():
    torch = pytest.importorskip("torch")
    c, b = host_cache(torch)
    kv, q = torch.zeros(4, 2, 64, dtype=torch.float16), torch.zeros(4, 4, 64, dtype=torch.float16)
    for fn in (mnb.mnb_kv_write, mnb.mnb_kv_read):
        assert refused(lambda: fn(c, b, kv, kv.clone(), stream=0))
    assert refused(lambda: mnb.mnb_attn(c, b, q, q.clone(), stream=0))
    assert refused(lambda: mnb.mnb_logprobs(torch.zeros(2, 9, dtype=torch.float16), entropy=torch.zeros(2), stream=0))


@pytest.mark.gpu
def test_tensors_of_two_places_never_reach_a_kernel():
    torch = pytest.importorskip("torch")
    host, _ = host_cache(torch)
    on = lambda x: x.cuda()  # noqa: E731
    codes = [on(x) for x in (host.K, host.V, host.K_scales, host.V_scales)]
    with pytest.raises(ValueError):
        mnb.KVCache(*codes[:3], host.V_scales)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        mnb.KVBatch(i32(2, 3), i32(2), i32(3).cpu(), 4, 2, 50)
    c, b = mnb.KVCache(*codes), mnb.KVBatch(i32(2, 3), i32(2), i32(3), 4, 2, 50)
    kv, q = (torch.zeros(4, h, 64, dtype=torch.float16, device="cuda") for h in (2, 4))
    lse, ws = torch.zeros(4, 4, device="cuda"), torch.zeros(4096, dtype=torch.uint8, device="cuda")
    for fn in (mnb.mnb_kv_write, mnb.mnb_kv_read):
        assert refused(lambda: fn(c, b, kv.cpu(), kv)) and refused(lambda: fn(c, b, kv, kv.cpu()))
        assert refused(lambda: fn(host, b, kv, kv.clone()))
    for bad in (dict(Q=q.cpu()), dict(out=q.cpu()), dict(lse=lse.cpu()), dict(ws=ws.cpu()), dict(ws=ws[:1].expand(4096))):
        assert refused(lambda: mnb.mnb_attn(c, b, **{**dict(Q=q, out=q.clone(), lse=lse, ws=ws), **bad})), bad
    x, t = torch.zeros(2, 9, dtype=torch.float16, device="cuda"), torch.zeros(2, dtype=torch.int64)
    assert refused(lambda: mnb.mnb_logprobs(x, t, lse[0, :2].contiguous()))
    assert refused(lambda: mnb.mnb_logprobs(x, entropy=torch.zeros(2)))


# What tests/test_gpu_prompt_tiles.py and others rely on: which kernel, with how many row tiles and chunks, takes a case.
def plan(dim, kv_heads, group, lens, news, page=32, window=0, max_len=None, sms=152):
    c = cache(page_size=page, kv_heads=kv_heads, head_dim=dim)
    b = batch(seqs=len(lens), tokens=sum(news), max_new=max(news), max_len=max_len or max(lens))
    info = mnb.MnbAttnPlanInfo()
    rc = mnb.lib().mnb_attn_plan(ctypes.byref(c), ctypes.byref(b), kv_heads * group, window, sms, ctypes.byref(info))
    assert rc == mnb.MNB_OK
    return info.as_dict()


def test_the_plan_and_the_workspace():
    assert plan(64, 3, 3, [577], [1]) == dict(prompt_rows=0, split_rows=8, chunk=128, splits=5, cluster=1, by_length=0)
    p = plan(128, 8, 4, [131071], [1])
    assert p["split_rows"] == 8 and p["splits"] > 8 and not p["cluster"]
    b = batch(seqs=1, tokens=1, max_new=1, max_len=131071)
    c = cache(page_size=32, kv_heads=8, head_dim=128)
    assert mnb.lib().mnb_attn_workspace(ctypes.byref(c), ctypes.byref(b), 32, 0, 152) == 32 * p["splits"] * 130 * 4
    assert plan(64, 1, 1, [5], [0]) == dict.fromkeys(p, 0)  # nothing to launch
    info = mnb.MnbAttnPlanInfo()
    L = mnb.lib()
    assert L.mnb_attn_plan(None, ctypes.byref(b), 4, 0, 152, ctypes.byref(info)) == mnb.MNB_ERR_ARG
    assert L.mnb_attn_plan(ctypes.byref(c), ctypes.byref(b), 32, 0, 152, None) == mnb.MNB_ERR_ARG
    assert L.mnb_attn_plan(ctypes.byref(c), ctypes.byref(b), 12, 0, 152, ctypes.byref(info)) == mnb.MNB_ERR_UNSUPPORTED


@pytest.mark.parametrize("case", prompt_cases.CASES, ids=lambda c: c.name)
@pytest.mark.parametrize("dim", [64, 128])
def test_cases_of_the_prompt_kernel_keep_their_plan(case, dim):
    p = plan(dim, case.kv_heads, case.group, case.lens, case.news, window=case.window, max_len=case.max_len)
    assert (p["prompt_rows"], p["splits"] > 1, p["split_rows"] > 0) == (case.rows, case.chunks, case.singles), p
