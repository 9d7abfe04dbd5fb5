"""Calls given a stream that make their buffers themselves, while the current
stream is busy with other work on the same memory."""

import numpy as np
import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
import synth
from tests import w4_reference as R
from tests.test_gpu_w4_experts import bf16_dev, dev, f64, scales_dev, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("M", [4, 20])
def test_layer_on_a_side_stream_without_buffers(dev, M, raw):  # noqa: F811
    E, Hd, I, k, fmt, group = 12, 512, 128, 3, R.MXFP4, 32
    x, wr = synth.x_bf16(M, Hd, seed=1), R.bf16(synth.w_f32(E, Hd, seed=2))
    c13, s13 = (v.reshape(E + 1, 2 * I, -1) for v in R.weight((E + 1) * 2 * I, Hd, fmt, group, 3))
    c2, s2 = (v.reshape(E + 1, Hd, -1) for v in R.weight((E + 1) * Hd, I, fmt, group, 4))
    args = [to_dev(v, dev) for v in (c13, s13, c2, s2)]
    xd, wrd = bf16_dev(x, dev), bf16_dev(wr, dev)
    ref_ids, ref_w, rel = R.route(x, wr, E, k, True, "one")
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(4):
        # freed blocks full of ones, and work that is still to come on them
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) for n in (1 << 10, 1 << 14, 1 << 17, 1 << 20)]
        torch.cuda._sleep(2_000_000)
        for t in junk:
            t.fill_(0xFE)
        del junk, t
        ids, tw = fb.fp8bs_moe_route(xd, wrd, k, shared="one", stream=stream)
        y = fb.fp8bs_moe_w4a16(xd, ids, tw, *args, fmt, group, stream=stream)
        outs.append((ids, tw, y))
    side.synchronize()  # (the current stream may still be asleep)
    for ids, tw, y in outs:
        with torch.cuda.stream(side):
            ids, tw, y = ids.cpu().numpy(), tw.cpu().numpy(), f64(y)
        assert np.array_equal(ids, ref_ids) and np.all(np.abs(tw - ref_w) <= rel * ref_w)
        ref, bound = R.moe(x, ids, tw, R.value(c13, s13, fmt, group), R.value(c2, s2, fmt, group))
        assert np.all(np.abs(y - ref) <= bound)
    torch.cuda.synchronize()
