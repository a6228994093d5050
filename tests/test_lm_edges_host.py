"""Refusals and checks of the cache, attention and log-probability calls at their edges, without a GPU."""
import ctypes

import pytest

from test_abi_host import run_without_gpu
from test_lm_ops_host import A, batch, cache

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
