"""Attention over a paged cache: what a row does not see has no part in it, whatever it holds.

References are those of attn_reference.py, in 64 bits.  Bounds are a row's own: of the keys that it
sees, and of nothing else.

* A score's D products, its factors and the difference from the maximum, exp2, the sums: as in
  attn_reference.py.
* A weight's rounding: `weight` of itself, 2^-11 in fp16 (codes); 2^-8 in bf16, and 2^-16 where two
  bf16 numbers stand for it.
* Codes: q is off by 2^-39 of its largest magnitude.  A weight times its value's scale is a number of
  fp16 of which 2^7 stands for the largest, or for up to 2^14 times that (the scales of a unit's
  keys may differ by 2^14 before each has its own): below fp16's normal numbers it is off by
  2^-25 2^-7 2^14 = 2^-18 of the largest, and multiplies the value's code.
"""

import math

import pytest
import torch

import fp8_block_scale_x128_gb300 as fb
from tests import attn_reference as A
from tests.test_gpu_attn_paged import make

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    fb.build()
    return torch.device("cuda", 0)


def attend(q, k, v, scale, window, weight, units=None):
    """One sequence: q [n, Hq, D], k and v [kv, Hk, D] in 64 bits; `units`: the scales [kv, Hk] of
    codes.  Returns o and its bound: row by row, from the keys that the row sees alone."""
    q = q.double().cpu()
    n, Hq, D = q.shape
    kv, G = k.shape[0], Hq // k.shape[1]
    o, bound = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(n):
        place = kv - n + i
        lo = max(place - window + 1, 0) if window else 0
        if place < 0:
            continue
        for h in range(Hq):
            kh, vh = k[lo:place + 1, h // G], v[lo:place + 1, h // G]
            s, size = kh @ q[i, h] * scale, kh.abs() @ q[i, h].abs() * scale
            most = s.max()
            w = torch.exp(s - most)
            total = w.sum()
            fine = torch.isfinite(vh)
            vs = torch.where(fine, vh, 0.0)
            odd = torch.where(fine, 0.0, vh).sum(0)  # a value that is not finite reaches the rows that see it
            o[i, h] = w @ vs / total + odd
            off = 2.0 ** -23 * (D / 16 + 16) * size + 4 * STEP * (1.5 * (s.abs() + most.abs()) + 150) + 2.0 ** -21
            least = 0.0
            if units is not None:
                off = off + scale * 2.0 ** -39 * q[i, h].abs().max() * kh.abs().sum(1)
                unit = units[lo:place + 1, h // G]
                least = 2.0 ** -18 * w.max() * unit.max() * (vs.abs() / unit.unsqueeze(1)).sum(0) / total
            # (a score of next to no weight may be off by much)
            off = torch.exp((s - most + off).clamp(max=30.0)) - w + w * (weight + 2 * STEP * (len(s) / 16 + 16))
            off = torch.nan_to_num(off, nan=0.0)
            # (N + n) / (S + e) is off N / S by (|n| + |N / S| |e|) / (S - |e|) at most
            e = off.sum() / total
            bound[i, h] = (off @ vs.abs() / total + e * (w @ vs / total).abs()) / (1 - e).clamp(min=1e-6) + least
    return o, bound


def check(lengths, q, tensors, table, o, window=0, scale=None, weight=2.0 ** -8):
    codes = len(tensors) == 4
    first, D, page = 0, q.shape[2], tensors[0].shape[1]
    for b, (n, kv) in enumerate(lengths):
        k, v = A.rows_of(tensors, table[b], kv)
        units = None
        if codes:
            j = torch.arange(kv)
            z = tensors[3].cpu()[table[b].cpu().long()[j // page], j % page]
            units = 2.0 ** (torch.where(z == 255, 0, z).double() - 127)
        ref, bound = attend(q[first:first + n], k, v, D ** -0.5 if scale is None else scale, window,
                            2.0 ** -11 if codes else weight, units)
        A.near(o[first:first + n], ref, bound)
        first += n


def at(tensors, table, b, j):
    """The page and slot of a sequence's key j."""
    page = tensors[0].shape[1]
    return int(table[b, j // page]), j % page


# ---- values and keys that are not numbers ------------------------------------------

FEW = [(2, 40), (4, 300), (7, 130), (3, 9)]


@pytest.mark.parametrize("window", [0, 3, 40])
@pytest.mark.parametrize("what", ["row", "code", "scale"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq", [2, 4])  # tiles of 8 and of 16 rows
def test_codes_of_few_rows_that_are_not_numbers_reach_only_rows_that_see_them(dev, Hq, D, what, window):
    q, tensors, table, cu, lens = make(FEW, Hq, 2, D, True, 16, "slots", dev, seed=D + window)
    for b, (n, kv) in enumerate(FEW):
        for j in {kv - 1, kv - 2, max(kv - n - window // 2, 0) if window else kv - 1}:  # drafted tokens; one behind a window
            place = at(tensors, table, b, j)
            if what == "row":  # as an append of an infinity or a NaN writes it
                tensors[1][place][1], tensors[3][place][1] = 0x7F, 255
            elif what == "code":
                tensors[1][place][1, 5 + b], tensors[1][place][0, D - 1] = 0x7F, 0xFF
            else:
                tensors[3][place][1] = 255
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=window)
    check(FEW, q, tensors, table, o, window)


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("what", ["row", "code", "scale"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_of_many_rows_that_are_not_numbers_reach_only_rows_that_see_them(dev, D, what, window):
    lengths = [(150, 300), (40, 90), (30, 1000)]
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, True, 16, "slots", dev, seed=D + window)
    for b, (n, kv) in enumerate(lengths):
        for j in (kv - 1, kv - 20, kv - n - 2 if window else kv - 5):
            place = at(tensors, table, b, j)
            if what == "row":
                tensors[1][place][1], tensors[3][place][1] = 0x7F, 255
            elif what == "code":
                tensors[1][place][1, 5 + b], tensors[1][place][0, D - 1] = 0x7F, 0xFF
            else:
                tensors[3][place][1] = 255
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=window)
    check(lengths, q, tensors, table, o, window)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new", [4, 40])
def test_a_bad_token_appended_as_codes_leaves_those_before_it(dev, new, what):
    """The last token's value has a number that is none: the rows before it do not see it."""
    Hq, Hk, D, page = 4, 2, 128, 16
    g = torch.Generator(device=dev).manual_seed(new)
    cache = fb.new_kv_cache(4, page, Hk, D, fb.FP8BS_KV_E4M3)
    row = torch.randn((new, Hq + 2 * Hk, D), generator=g, device=dev).to(torch.bfloat16)
    row[-1, Hq + Hk + 1, 9] = what
    pos = torch.arange(new, device=dev)
    q = fb.fp8bs_qk_norm_rope_append(row[:, :Hq], row[:, Hq:Hq + Hk], row[:, Hq + Hk:], pos, pos, fb.Rope(D), cache)
    table = torch.arange(4, dtype=torch.int32, device=dev).unsqueeze(0)
    cu, lens = (torch.tensor(v, dtype=torch.int32, device=dev) for v in ([0, new], [new]))
    o = fb.fp8bs_attn_paged(q, cache, table, cu, lens)
    check([(new, new)], q, cache.tensors, table, o)
    assert bool(torch.isfinite(o[:-1]).all()) and bool(torch.isnan(o[-1, Hq // Hk:]).all())


# ---- scales of codes ---------------------------------------------------------------

@pytest.mark.parametrize("size,scale", [(1e-3, None), (1.0, 1e-6), (1.0, 1e-30), (1e-20, 1e-20)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_of_zeros_and_tiny_scores_under_a_mask(dev, D, size, scale):
    """Units whose keys are all rows of zeros, and sequences without a key, at scores of next to nothing."""
    lengths = [(20, 0), (30, 300), (40, 200), (17, 5)]
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, True, 16, "slots", dev, seed=D, size=size)
    for b, (n, kv) in enumerate(lengths):
        for j in range(256 if b == 1 else 0, kv):
            place = at(tensors, table, b, j)
            tensors[0][place], tensors[2][place] = 0, 0
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, scale=scale)
    check(lengths, q, tensors, table, o, scale=scale)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("byte", [133, 143, 155, 180])  # 2^6 .. 2^53
@pytest.mark.parametrize("lengths", [[(4, 300), (7, 130)], [(150, 300), (40, 90)]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scales_that_are_masked_change_nothing(dev, D, lengths, byte, window):
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, True, 16, "slots", dev, seed=D + byte)
    for b, (n, kv) in enumerate(lengths):
        for j in (kv - 1, kv - n - window // 2 - 2 if window else kv - 2):
            place = at(tensors, table, b, j)
            tensors[2][place][0], tensors[3][place][1] = byte, byte
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=window)
    check(lengths, q, tensors, table, o, window)


@pytest.mark.parametrize("apart", [-70, -20, 14, 15, 20, 40])
@pytest.mark.parametrize("lengths", [[(4, 300), (7, 130)], [(150, 300), (40, 90)]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_of_next_to_no_weight(dev, D, lengths, apart):
    """A key far below the others' scores: its value, or its own size, takes nothing from them."""
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, True, 16, "slots", dev, seed=D)
    q[:, :, :] = q.abs() + 0.5
    for b, (n, kv) in enumerate(lengths):
        for j in (3, kv - n - 5):
            place = at(tensors, table, b, j)
            tensors[0][place] = 0xFE  # -448: scores of some -448 sqrt(D) scale
            tensors[2][place][0], tensors[2][place][1] = 127, 127 + max(apart, 0)
            tensors[3][place][0] = 119 + apart
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens)
    check(lengths, q, tensors, table, o)


@pytest.mark.parametrize("lengths", [[(4, 300), (7, 130)], [(150, 300), (40, 90)]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_zeros_beside_others(dev, D, lengths):
    """Keys and values of zeros, with a scale byte of 0 as an append writes them, and units of nothing else."""
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, True, 16, "slots", dev, seed=D)
    g = torch.Generator(device=dev).manual_seed(2)
    for i in (0, 1):
        none = torch.rand(tensors[2 + i].shape, generator=g, device=dev) < 0.1
        for j in range(128, 256):
            if lengths[0][1] > j:
                none[at(tensors, table, 0, j)] = True
        tensors[i][none], tensors[2 + i][none] = 0, 0
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens)
    check(lengths, q, tensors, table, o)


@pytest.mark.parametrize("lengths", [[(4, 300), (7, 130)], [(150, 300), (40, 90)]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_zeros_beside_the_largest_values(dev, D, lengths):
    """A value of zeros has its weight in the sum, also beside values of 2^50."""
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, True, 16, "slots", dev, seed=D)
    g = torch.Generator(device=dev).manual_seed(3)
    tensors[3][torch.rand(tensors[3].shape, generator=g, device=dev) < 0.2] += 60
    none = torch.rand(tensors[3].shape, generator=g, device=dev) < 0.3
    tensors[1][none], tensors[3][none] = 0, 0
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens)
    check(lengths, q, tensors, table, o)


# ---- scores of minus infinity ------------------------------------------------------

@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("lengths", [[(4, 300), (1, 7), (3, 2), (2, 5000)], [(150, 300), (40, 90), (20, 7), (30, 4000)]])
def test_rows_whose_scores_are_all_minus_infinity_are_no_numbers(dev, lengths, codes):
    D = 128
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, codes, 16, "slots", dev, seed=1)
    if codes:
        tensors[0][:, :, 1, 3] = 0xB8  # -1
        q[:, 3, 3] = math.inf
    else:
        tensors[0][:, :, 1, 3] = -math.inf
        q[:, 3, 3], q[:, 2, 3] = 1.0, -1.0
    cache, ws = fb.KvCache(*tensors), fb.new_attn_workspace(D)
    o = fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws)
    first = 0
    for n, kv in lengths:
        rows = o[first:first + n].float()
        none = max(n - kv, 0)  # rows that see no key
        assert bool((rows[:none] == 0).all())
        assert bool(torch.isnan(rows[none:, 3]).all())
        assert bool(torch.isfinite(rows[none:, :2]).all())
        first += n


def test_a_score_of_minus_infinity_beside_others_is_no_weight(dev):
    for lengths in ([(4, 300), (2, 9)], [(150, 300), (40, 90)]):
        q, tensors, table, cu, lens = make(lengths, 4, 2, 128, False, 16, "slots", dev, seed=2)
        q[:, :, 3] = q[:, :, 3].abs() + 0.25
        for b, (n, kv) in enumerate(lengths):
            tensors[0][at(tensors, table, b, kv - n)][1, 3] = -math.inf
        check(lengths, q, tensors, table, fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens))


# ---- large scores -------------------------------------------------------------------

@pytest.mark.parametrize("power", [10, 14, 17, 20, 24, 27, 30, 50])
@pytest.mark.parametrize("lengths", [[(4, 300), (7, 130)], [(150, 300), (40, 90)]])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_of_any_size_leave_numbers(dev, D, codes, lengths, power):
    """A row of one key has that key's value, whatever its score; a key far below another has no part."""
    q, tensors, table, cu, lens = make(lengths, 4, 2, D, codes, 16, "slots", dev, seed=D + power)
    if codes:
        tensors[2][::2] += power  # pages in turn: units whose scales are far apart, or of one kind
    else:
        tensors[0].mul_(2.0 ** power)
    cache = fb.KvCache(*tensors)
    o = fb.fp8bs_attn_paged(q, cache, table, cu, lens, window=1)
    first = 0
    for b, (n, kv) in enumerate(lengths):
        _, v = A.rows_of(tensors, table[b], kv)
        ref = v[kv - n:].repeat_interleave(2, 1)
        # a weight's rounding, a power of two's, and a score's with its value's exponent
        A.near(o[first:first + n], ref, (2.0 ** -8 if not codes else 2.0 ** -11 + 2.0 ** -20) * ref.abs())
        first += n
    # two keys whose scores are far apart: the upper one's value
    q = q.abs() + 0.5
    for b, (n, kv) in enumerate(lengths):
        for j in range(kv):
            place = at(tensors, table, b, j)
            if codes:
                tensors[0][place], tensors[2][place] = (0x7E if j % 2 else 0xFE), 127 + power
            else:
                tensors[0][place] = 2.0 ** power * (8 if j % 2 else -8)
    o = fb.fp8bs_attn_paged(q, cache, table, cu, lens, window=2)
    first = 0
    for b, (n, kv) in enumerate(lengths):
        _, v = A.rows_of(tensors, table[b], kv)
        places = torch.arange(kv - n, kv)
        ref = v[torch.where(places % 2 == 1, places, (places - 1).clamp(min=0))].repeat_interleave(2, 1)
        A.near(o[first:first + n], ref, (2.0 ** -8 if not codes else 2.0 ** -11 + 2.0 ** -20) * ref.abs())
        first += n


# ---- the precision of weights ------------------------------------------------------

@pytest.mark.parametrize("new,codes,weight", [(1, False, 2.0 ** -16), (1, True, None), (200, True, None), (200, False, 2.0 ** -8)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_are_rounded_as_stated(dev, D, new, codes, weight):
    """Two keys a row, of opposite values: what is left is of the size of the weights' errors."""
    lengths = [(1, 2)] * 64 if new == 1 else [(new, new + 1)]
    q, tensors, table, cu, lens = make(lengths, 2, 2, D, codes, 16, "slots", dev, seed=D, size=0.05)
    for b, (n, kv) in enumerate(lengths):
        for j in range(1, kv):
            a, c = at(tensors, table, b, j), at(tensors, table, b, j - 1)
            tensors[1][a] = tensors[1][c] ^ 0x80 if codes else -tensors[1][c]
            if codes:
                tensors[3][a] = tensors[3][c]
    o = fb.fp8bs_attn_paged(q, fb.KvCache(*tensors), table, cu, lens, window=2)
    check(lengths, q, tensors, table, o, 2, weight=weight)


def test_a_thread_of_its_own(dev):
    """The first call of a host thread that has made no other."""
    import threading
    lengths = [(150, 300)]
    q, tensors, table, cu, lens = make(lengths, 4, 2, 128, False, 16, "slots", dev, seed=3)
    cache, ws, o = fb.KvCache(*tensors), fb.new_attn_workspace(128), torch.zeros_like(q)
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            fb.fp8bs_attn_paged(q, cache, table, cu, lens, o=o, workspace=ws)
            torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed
    check(lengths, q, tensors, table, o)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_items_without_masks(dev, D, codes):
    """One token a sequence of many query heads, lengths that end with a unit: nothing to look through."""
    lengths = [(1, 128 * (1 + b % 2)) for b in range(300)]
    q, tensors, table, cu, lens = make(lengths, 128, 4, D, codes, 16, "slots", dev, seed=D)
    cache, ws = fb.KvCache(*tensors), fb.new_attn_workspace(D)
    o = fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws)
    for _ in range(20):
        assert torch.equal(o, fb.fp8bs_attn_paged(q, cache, table, cu, lens, workspace=ws))
    assert fb.fp8bs_check_error(ws) == 0
    rows = [0, 1, 151, 152, 299]
    first = torch.tensor(rows, device=dev)
    check([lengths[r] for r in rows], q[first], tensors, table[first], o[first])
