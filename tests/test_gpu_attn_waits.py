"""Waits of the attention kernel of many rows that run out: a short limit (the diagnostic setting) makes
some wait expire at one place or another.  The kernel reports it and ends; the device answers, and the
next call is right."""

import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
from tests.test_gpu_attn_paged import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    fb.build()
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def _restore_defaults():
    yield
    fb.fp8bs_debug_config(0, 0)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_is_reported_and_the_kernel_ends(dev, D, codes):
    lengths = [(300, 3000), (40, 90), (20, 700), (500, 500)]
    q, tensors, table, cu, lens = make(lengths, 8, 2, D, codes, 16, "slots", dev, seed=D)
    cache, ws = fb.KvCache(*tensors), fb.new_attn_workspace(D)
    want = fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws).clone()
    assert fb.fp8bs_check_error(ws) == 0
    o = torch.empty_like(q)
    for limit in (1, 100, 1000, 3000, 10000, 30000):
        fb.fp8bs_debug_config(timeout_cycles=limit)
        fb.fp8bs_attn_paged(q, cache, table, cu, lens, o=o, workspace=ws)
        rc = fb.fp8bs_check_error(ws)
        assert rc == fb.FP8BS_ERR_TIMEOUT or limit > 1 and rc == 0
        fb.fp8bs_debug_config(0, 0)
        fb.fp8bs_attn_paged(q, cache, table, cu, lens, o=o, workspace=ws)
        assert fb.fp8bs_check_error(ws) == 0 and torch.equal(o, want)
