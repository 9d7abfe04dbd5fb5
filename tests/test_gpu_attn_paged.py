"""Attention over a paged cache against 64 bits: lengths, masks, pages, layouts."""

import math

import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
from tests import attn_reference as A

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -8  # a weight's rounding at most, in the kernel that rounds it once


@pytest.fixture(scope="module")
def dev():
    fb.build()
    return torch.device("cuda", 0)


def make(lengths, Hq, Hk, D, codes, page, order, dev, seed=0, behind=0, spare=3, size=1.0):
    """q, cache tensors, table, cu, lens of sequences (new, kv)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    T = sum(n for n, _ in lengths) + behind
    q = (torch.randn((T, Hq, D), generator=g, device=dev) * size).to(torch.bfloat16)
    need = [-(-kv // page) for _, kv in lengths]
    pages = sum(need) + spare
    shape = (pages, page, Hk, D) if order == "slots" else (pages, Hk, page, D)
    rows = [torch.randn(shape, generator=g, device=dev).to(torch.bfloat16) for _ in range(2)]
    if codes:
        scale = torch.randint(117, 121, shape[:3], generator=g, device=dev).to(torch.uint8)
        tensors = [torch.randint(0, 256, shape, generator=g, device=dev).to(torch.uint8) for _ in range(2)]
        tensors = [torch.where(t & 0x7F == 0x7F, t & 0xF8, t) for t in tensors] + [scale, scale.flip(0).contiguous()]
    else:
        tensors = rows
    if order == "heads":
        tensors = [t.transpose(1, 2) for t in tensors]
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lengths), max(need + [1]) + 2), 1 << 30, dtype=torch.int32, device=dev)  # never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = torch.tensor([0] + [n for n, _ in lengths], dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
    lens = torch.tensor([kv for _, kv in lengths], dtype=torch.int32, device=dev)
    # what lies in slots that no sequence has reaches nothing
    if not codes:
        used = torch.zeros((pages, page), dtype=torch.bool, device=dev)
        for b, (_, kv) in enumerate(lengths):
            j = torch.arange(kv, device=dev)
            used[table[b].long()[j // page], j % page] = True
        for t in tensors:
            t[~used] = float("nan")
    return q, tensors, table, cu, lens


def check(lengths, q, tensors, table, o, window=0, scale=None):
    first = 0
    D = q.shape[2]
    for b, (n, kv) in enumerate(lengths):
        k, v = A.rows_of(tensors, table[b], kv)
        codes = None
        if len(tensors) == 4 and kv:
            j = torch.arange(kv)
            page, at = table[b].cpu().long()[j // tensors[0].shape[1]], j % tensors[0].shape[1]
            codes = [2.0 ** (torch.where(z == 255, 0, z).double() - 127) for z in (t.cpu()[page, at] for t in tensors[2:])]
        ref, bound = A.attend(q[first:first + n], k, v, kv, D ** -0.5 if scale is None else scale, window, WEIGHT, codes)
        A.near(o[first:first + n], ref, bound)
        first += n


LENGTHS = {
    "one key": [(1, 1)], "one token": [(1, 777)], "edges": [(1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 128), (1, 129)],
    "none": [(0, 5), (1, 0), (0, 0), (2, 3), (3, 1)], "drafts": [(4, 300), (2, 2), (7, 130)],
    "prompt": [(33, 33)], "chunk": [(70, 311), (1, 40)], "long": [(1, 3333), (1, 9)],
}


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("Hq,Hk,D,page,order", [(8, 2, 128, 16, "slots"), (5, 1, 64, 1, "heads"), (16, 2, 256, 32, "heads"),
                                                (3, 3, 128, 64, "heads"), (34, 2, 64, 8, "slots")])
@pytest.mark.parametrize("which", LENGTHS)
def test_lengths(dev, which, Hq, Hk, D, page, order, codes):
    lengths = LENGTHS[which]
    q, tensors, table, cu, lens = make(lengths, Hq, Hk, D, codes, page, order, dev, seed=len(which), behind=2)
    o = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev)
    ws = fb.new_attn_workspace(D)
    fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, o=o, workspace=ws)
    assert fb.fp8bs_check_error(ws) == 0
    check(lengths, q, tensors, table, o)
    assert bool((o[sum(n for n, _ in lengths):] == 5).all())  # rows behind the last sequence


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 200, 1 << 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_window(dev, window, D, codes):
    lengths = [(1, 500), (40, 129), (5, 5), (1, 1), (200, 333)]
    q, tensors, table, cu, lens = make(lengths, 6, 2, D, codes, 16, "slots", dev, seed=window % 97)
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=window)
    check(lengths, q, tensors, table, o, window)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("size,scale", [(30.0, None), (1.0, 3.0), (0.0, None), (1.0, 1e-6)])
def test_sharp_and_flat_scores(dev, size, scale, codes):
    lengths = [(1, 700), (100, 400)]
    q, tensors, table, cu, lens = make(lengths, 8, 2, 128, codes, 16, "slots", dev, seed=7, size=size)
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, scale=scale)
    check(lengths, q, tensors, table, o, scale=scale)


@pytest.mark.parametrize("lengths", [[(1, 700), (3, 50)], [(100, 400), (40, 40)]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_far_apart(dev, D, lengths):
    """Rows of zeros, tiny rows and large ones beside each other; queries of all sizes."""
    q, tensors, table, cu, lens = make(lengths, 8, 2, D, True, 16, "slots", dev, seed=D)
    g = torch.Generator(device=dev).manual_seed(1)
    for t in tensors[2:]:
        t.copy_(torch.randint(90, 125, t.shape, generator=g, device=dev).to(torch.uint8))
    tensors[3][torch.rand(tensors[3].shape, generator=g, device=dev) < 0.2] = 0
    tensors[1][tensors[3] == 0] = 0
    q *= torch.exp2(torch.randint(-60, 3, q.shape[:2], generator=g, device=dev).float()).unsqueeze(2).to(torch.bfloat16)
    q[0, 0] = 0
    check(lengths, q, tensors, table, fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(dev, what, D):
    lengths = [(150, 300), (4, 90), (1, 70)]
    for window in (0, 60):
        q, tensors, table, cu, lens = make(lengths, 4, 2, D, False, 16, "slots", dev, seed=3)
        for b, j in ((0, 200), (0, 299), (0, 290), (1, 88), (2, 3)):
            page, at = int(table[b, j // 16]), j % 16
            tensors[1][page, at, 1, 7] = what
        o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=window)
        check(lengths, q, tensors, table, o, window)


@pytest.mark.parametrize("codes", [False, True])
def test_keys_that_are_not_numbers_reach_only_rows_that_see_them(dev, codes):
    lengths, D = [(150, 300)], 128
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, codes, 16, "slots", dev, seed=4)
    page, at = int(table[0, 250 // 16]), 250 % 16
    if codes:
        tensors[2][page, at, 0], tensors[3][page, at, 1] = 255, 255
    else:
        tensors[0][page, at, 0, 9], tensors[1][page, at, 1] = math.nan, math.nan
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens)
    assert not bool(torch.isnan(o[:100]).any()) and bool(torch.isnan(o[100:]).all())


def test_strided_queries_outputs_and_shared_pages(dev):
    # two sequences with the same first pages; q a slice of wider rows, o every second head
    page, D, Hk, Hq = 16, 128, 2, 4
    q, tensors, table, cu, lens = make([(1, 100), (2, 100)], Hq, Hk, D, False, page, "slots", dev, seed=9)
    table[1, :4] = table[0, :4]
    wide = torch.zeros((3, Hq + 4, D), dtype=torch.bfloat16, device=dev)
    wide[:, 2:2 + Hq] = q
    o = torch.full((3, 2 * Hq, D), 3.0, dtype=torch.bfloat16, device=dev)
    fb.fp8bs_attn_paged(wide[:, 2:2 + Hq], fb.KvCache(*tensors), table, cu, lens, o=o[:, 1::2])
    check([(1, 100), (2, 100)], q, tensors, table, o[:, 1::2])
    assert bool((o[:, ::2] == 3).all())


@pytest.mark.parametrize("codes", [False, True])
def test_many_sequences_and_long_ones(dev, codes):
    lengths = [(1, (37 * b) % 211 + 1) for b in range(fb.FP8BS_ATTN_MAX_SEQS)]
    q, tensors, table, cu, lens = make(lengths, 2, 1, 64, codes, 16, "slots", dev, seed=1)
    check(lengths, q, tensors, table, fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens))
    lengths = [(1, 40000), (3, 20011)]
    q, tensors, table, cu, lens = make(lengths, 8, 1, 128, codes, 64, "heads", dev, seed=2)
    check(lengths, q, tensors, table, fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens))


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_chunks_are_right_and_the_same_every_time(dev, D, codes):
    """Many units an item, items that several blocks share, few rows and many."""
    for lengths in ([(4, 3001), (9, 5000), (3, 64)], [(130, 2777), (60, 1500)]):
        q, tensors, table, cu, lens = make(lengths, 16, 2, D, codes, 16, "slots", dev, seed=D + codes)
        cache, ws = fb.KvCache(*tensors), fb.new_attn_workspace(D)
        o = fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws)
        check(lengths, q, tensors, table, o)
        for _ in range(20):
            assert torch.equal(o, fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws))
        assert fb.fp8bs_check_error(ws) == 0


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("page", [1, 2, 64, 256, 1024])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_and_pages_of_all_sizes(dev, D, page, codes):
    """Also sequences with more new tokens than keys, and with none of either."""
    lengths = [(40, 300), (33, 33), (20, 7), (18, 0), (0, 12), (50, 1029), (1, 90)]
    for window in (0, 37):
        q, tensors, table, cu, lens = make(lengths, 12, 2, D, codes, page, "heads", dev, seed=page + D, behind=3)
        o, ws = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev), fb.new_attn_workspace(D)
        fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=window, o=o, workspace=ws)
        assert fb.fp8bs_check_error(ws) == 0
        check(lengths, q, tensors, table, o, window)
        assert bool((o[-3:] == 5).all())


@pytest.mark.parametrize("new", [1, 40])
def test_keys_and_values_side_by_side(dev, new):
    """One tensor [pages, head, slot, 2, D] and one [heads, pages, slots, D]: other orders of the axes."""
    lengths, D, page = [(new, 200), (new, 77)], 128, 16
    q, tensors, table, cu, lens = make(lengths, 8, 4, D, False, page, "slots", dev, seed=11)
    pages = tensors[0].shape[0]
    both = torch.empty((pages, 4, page, 2, D), dtype=torch.bfloat16, device=dev)
    for i in range(2):
        both[:, :, :, i] = tensors[i].transpose(1, 2)
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*[both[:, :, :, i].transpose(1, 2) for i in range(2)]), table, cu, lens)
    check(lengths, q, tensors, table, o)
    apart = [t.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for t in tensors]
    assert torch.equal(o, fb.fp8bs_attn_paged(q, fb.KvCache(*apart), table, cu, lens))


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("codes", [False, True])
def test_the_longest_sequences(dev, new, codes):
    """2^30 keys, of which a window sees a few; one more is too long."""
    D, page, cols = 64, 65536, (1 << 14) + 1
    q, tensors, _, cu, _ = make([(new, page)], 4, 1, D, codes, page, "slots", dev, seed=12, spare=0)
    table, ws = torch.zeros((1, cols), dtype=torch.int32, device=dev), fb.new_attn_workspace(D)
    cache = fb.KvCache(*tensors)

    def at(kv):
        o = fb.fp8bs_attn_paged(q, cache, table, cu, torch.tensor([kv], dtype=torch.int32, device=dev), window=300, workspace=ws)
        return fb.fp8bs_check_error(ws), o

    rc, o = at(1 << 30)
    assert rc == 0
    check([(new, page)], q, tensors, table[:, :1], o, 300)
    assert at((1 << 30) + 1)[0] == fb.FP8BS_ERR_DEVICE


def test_two_graphs_with_one_workspace(dev):
    D, ws = 128, fb.new_attn_workspace(128)
    calls = []
    for lengths in ([(1, 5000), (1, 70)], [(300, 2000), (2, 9)]):
        q, tensors, table, cu, lens = make(lengths, 8, 2, D, False, 16, "slots", dev, seed=len(calls))
        cache, o = fb.KvCache(*tensors), torch.empty_like(q)
        want = fb.fp8bs_attn_paged(q, cache, table, cu, lens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fb.fp8bs_attn_paged(q, cache, table, cu, lens, o=o, workspace=ws)
        calls.append((graph, o, want, (cache, table, cu, lens, q)))
    for i in (0, 1, 1, 0, 0, 1):
        calls[i][1].zero_()
        calls[i][0].replay()
        assert torch.equal(calls[i][1], calls[i][2])


def test_cache_past_32_bit_offsets(dev):
    page, Hk, D = 64, 8, 128
    pages = (1 << 31) // (page * Hk * D) + 9
    k = torch.empty((pages, page, Hk, D), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    ids = [pages - 1, 0, pages - 2]
    for p in ids:
        k[p], v[p] = torch.randn((page, Hk, D), device=dev), torch.randn((page, Hk, D), device=dev)
    table = torch.tensor([ids], dtype=torch.int32, device=dev)
    q = torch.randn((1, 8, D), device=dev).to(torch.bfloat16)
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device=dev), torch.tensor([150], dtype=torch.int32, device=dev)
    o = fb.fp8bs_attn_paged(q, fb.KvCache(k, v), table, cu, lens)
    small = torch.stack([k[p] for p in ids]), torch.stack([v[p] for p in ids])
    check([(1, 150)], q, small, torch.tensor([0, 1, 2], dtype=torch.int32).unsqueeze(0), o)
    # and a token appended to the last page
    slot = torch.tensor([pages * page - 1], device=dev)
    row = torch.randn((1, 3 * Hk, D), device=dev).to(torch.bfloat16)
    fb.fp8bs_qk_norm_rope_append(row[:, :Hk], row[:, Hk:2 * Hk], row[:, 2 * Hk:], slot, slot, fb.Rope(0), fb.KvCache(k, v))
    assert torch.equal(k[-1, -1], row[0, Hk:2 * Hk]) and torch.equal(v[-1, -1], row[0, 2 * Hk:])


def test_deterministic_captured_and_on_a_side_stream(dev):
    lengths = [(1, 1000), (5, 333), (1, 31)]
    D = 128
    q, tensors, table, cu, lens = make(lengths, 8, 2, D, False, 16, "slots", dev, seed=5)
    cache, ws = fb.KvCache(*tensors), fb.new_attn_workspace(D)
    want = fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws).clone()
    o = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fp8bs_attn_paged(q, cache, table, cu, lens, o=o, workspace=ws)
    for _ in range(3):
        o.zero_()
        graph.replay()
        assert torch.equal(o, want)
    # the captured call follows the lengths on the device
    lens.copy_(torch.tensor([900, 200, 31], dtype=torch.int32))
    graph.replay()
    check([(1, 900), (5, 200), (1, 31)], q, tensors, table, o)
    lens.copy_(torch.tensor([1000, 333, 31], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = fb.fp8bs_attn_paged(q, cache, table, cu, lens, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_lengths_and_pages_that_do_not_fit_are_reported(dev):
    D = 128
    q, tensors, table, cu, lens = make([(1, 100), (2, 64)], 4, 2, D, False, 16, "slots", dev, seed=6)
    cache, ws = fb.KvCache(*tensors), fb.new_attn_workspace(D)

    def status(**kw):
        a = dict(q=q, cache=cache, block_table=table, cu_q=cu, kv_len=lens, workspace=ws)
        o = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev)
        fb.fp8bs_attn_paged(**{**a, **kw}, o=o)
        return fb.fp8bs_check_error(ws), o

    assert status()[0] == 0
    bad = table.clone()
    bad[0, 1] = tensors[0].shape[0]
    rc, o = status(block_table=bad)
    assert rc == fb.FP8BS_ERR_DEVICE
    check([(2, 64)], q[1:], tensors, table[1:], o[1:])  # the other sequence has its values
    bad[0, 1] = -1
    assert status(block_table=bad)[0] == fb.FP8BS_ERR_DEVICE
    def vec(*v):
        return torch.tensor(v, dtype=torch.int32, device=dev)
    assert status(kv_len=vec(table.shape[1] * 16 + 1, 64))[0] == fb.FP8BS_ERR_DEVICE
    assert status(kv_len=vec(-1, 64))[0] == fb.FP8BS_ERR_DEVICE
    assert status(cu_q=vec(0, 1, 4))[0] == fb.FP8BS_ERR_DEVICE
    assert status(cu_q=vec(-1, 1, 3))[0] == fb.FP8BS_ERR_DEVICE
    assert status(cu_q=vec(0, 3, 1))[0] == fb.FP8BS_ERR_DEVICE
    assert status()[0] == 0


def test_append_then_attend(dev):
    """A prompt in two chunks and decoded tokens, with their rotation, against 64 bits over all of them."""
    Hq, Hk, D, page = 8, 2, 128, 16
    for codes in (False, True):
        cache = fb.new_kv_cache(12, page, Hk, D, fb.FP8BS_KV_E4M3 if codes else fb.FP8BS_KV_BF16)
        rope = fb.Rope(64, 1e4)
        g = torch.Generator(device=dev).manual_seed(8)
        gam = [(1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2)]
        table = torch.randperm(12, generator=g, device=dev).to(torch.int32).unsqueeze(0)
        done = 0
        for n in (70, 45, 1, 1, 1):
            row = torch.randn((n, (Hq + 2 * Hk) * D), generator=g, device=dev).to(torch.bfloat16).view(n, -1, D)
            pos = done + torch.arange(n, device=dev)
            slots = table[0].long()[pos // page] * page + pos % page
            q = fb.fp8bs_qk_norm_rope_append(row[:, :Hq], row[:, Hq:Hq + Hk], row[:, Hq + Hk:], pos, slots, rope, cache, *gam)
            done += n
            cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
            lens = torch.tensor([done], dtype=torch.int32, device=dev)
            o = fb.fp8bs_attn_paged(q, cache, table, cu, lens)
            check([(n, done)], q, cache.tensors, table, o)
