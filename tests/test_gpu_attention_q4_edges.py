"""Decode attention over a Q4 KV cache (bq_attn_decode_q4) where its rounding,
its maximum and its masks can go wrong: fp16 output against fp32 output, the
same contents in caches of other sizes, scores of any size, scores that are all
-inf, value scales that are not finite where some rows do not see them,
idle slots, numbers of segments just above the grid."""
import numpy as np
import pytest

from quantised_weight_gemv_b200 import bq
from tests.gpu_helpers import DEV
from tests.kv_helpers import attention_ref, check_attention, random_cache_q4, run_attention, to_dev

pytestmark = pytest.mark.gpu


def q_bits(seed, *shape, size=1.0):
    return (np.random.default_rng(seed).standard_normal(shape) * size).astype(np.float16).view(np.uint16)


@pytest.mark.parametrize("B,Tq,Hkv,G,D,Tmax,lens", [
    # one and two row tiles a warp, both head widths; small caches and those past 2^17 positions
    (1, 1, 2, 5, 128, 256, [250]),
    (4, 1, 4, 5, 128, 16384, [16384, 300, 0, 9000]),
    (3, 4, 3, 4, 128, 16384, [16384, 100, 9001]),
    (9, 1, 8, 4, 64, 2048, [2048 - 200 * i for i in range(9)]),
    (2, 8, 4, 5, 64, 32768, [5, 20000]),
])
def test_fp16_output_is_the_fp32_output_rounded_once(B, Tq, Hkv, G, D, Tmax, lens):
    """Exactly: softmax weights, sums and merges do not depend on the output's
    type, so the two outputs differ by one rounding to nearest."""
    planes = random_cache_q4(40, B, Hkv, Tmax, D)
    q = q_bits(41, B, Tq, Hkv * G, D)
    f32 = run_attention(planes, q, lens, G, D ** -0.5, False)
    f16 = run_attention(planes, q, lens, G, D ** -0.5, True)
    assert np.array_equal(f16, f32.astype(np.float16).astype(np.float32))


@pytest.mark.parametrize("Tq", [1, 4])
def test_the_same_contents_in_a_larger_cache_give_the_same_bits(Tq):
    """A cache allocated 256 times as long, and one with idle slots behind the
    sequence."""
    Hkv, G, D, n = 2, 4, 128, 500
    part = random_cache_q4(42, 1, Hkv, 512, D)
    q = q_bits(43, 1, Tq, Hkv * G, D)
    want = run_attention(part, q, [n], G, 0.088)
    for B, Tmax in ((1, 1 << 17), (5, 1 << 15)):
        planes = []
        for p in part:
            w = np.zeros((B, Hkv, Tmax, p.shape[-1]), p.dtype)
            w[0, :, :512] = p[0]
            planes.append(w)
        qq = np.concatenate([q] + [np.zeros_like(q)] * (B - 1))
        assert np.array_equal(run_attention(planes, qq, [n] + [0] * (B - 1), G, 0.088)[:1], want)


def exact_scores(seed, B, Tq, Hkv, G, D, Tmax, dims):
    """A cache and queries whose scores are sums of two terms, exact in fp32:
    sum over (element, size) of dims of size * code[element], codes random and
    scales 1; query rows differ in sign."""
    kc, ks, vc, vs = [p.copy() for p in random_cache_q4(seed, B, Hkv, Tmax, D)]
    r = np.random.default_rng(seed + 1)
    kc[:] = 0x88                                                      # code 0
    ks[:] = 0x3c00
    q = np.zeros((B, Tq, Hkv * G, D), np.float16)
    for d, size in dims:
        byte = d // 32 * 16 + d % 16
        assert d % 32 < 16                                            # (a low nibble)
        kc[..., byte] = 0x80 | (8 + (r.integers(-8, 8, kc.shape[:3]) if size else 0))
        q[..., d] = size
    q[:, :, 1::2] *= -1
    return (kc, ks, vc, vs), q.view(np.uint16)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("dims,scale", [
    # sizes of the terms of a score, softmax scale: the largest scores are ties of
    # positions whose codes agree, others are further away than exp reaches
    ([(3, 1024.0)], 2.0 ** 14), ([(3, 1024.0)], 2.0 ** 20), ([(3, 2.0 ** -24)], 1e18), ([(3, 32768.0)], 1e18),
    ([(3, 32768.0)], -1e18), ([(3, 4096.0), (37, 2.0 ** -8)], 2.0 ** 14),
    # scores of 2^25 whose differences reach into the softmax
    ([(3, 4096.0), (37, 2.0 ** -8)], 2.0 ** 8 * 3),
    # scores too small to matter
    ([(3, 1.0)], 1e-30), ([(3, 32768.0)], 0.0),
])
@pytest.mark.parametrize("B,Tq,Hkv,G,D,Tmax,lens", [
    (2, 1, 2, 4, 128, 512, [512, 33]),
    (1, 1, 2, 3, 64, 8192, [8100]),
    (2, 4, 1, 4, 128, 1024, [1000, 3]),
    (20, 1, 8, 2, 64, 2048, [2048 - 10 * i for i in range(20)]),
])
def test_scores_of_any_size(B, Tq, Hkv, G, D, Tmax, lens, dims, scale, f16):
    """The scores are exact, so check_attention's bound holds without the
    scores' own error.  What is left of it: the exponent's argument x, an exact
    difference of scores times scale * log2(e), takes three roundings, so that a
    weight is off by 2^-22 x of itself: 2^-17 up to x = 2^5 (twice, for the sum of
    weights); further weights are below 2^-32, and n <= 2^13 of them are off by
    2^13 2^-32 2^-15 times a value below 8."""
    planes, q = exact_scores(50, B, Tq, Hkv, G, D, Tmax, dims)
    o_ref, ao, slack, floor = attention_ref(planes, q, lens, G, scale)
    got = run_attention(planes, q, lens, G, scale, f16)
    check_attention(got, (o_ref, ao, np.full_like(slack, 2 * 2.0 ** -17), floor + 2.0 ** -31), f16)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("B,Tq,Hkv,G,D,Tmax,lens", [
    (2, 1, 2, 3, 128, 64, [1, 64]),                                   # whole segments
    (1, 1, 1, 4, 64, 8192, [8000]),                                   # merged over warps and CTAs
    (2, 5, 1, 4, 128, 1024, [1000, 3]),
])
def test_scores_that_are_all_minus_infinity(B, Tq, Hkv, G, D, Tmax, lens, f16):
    """A query element of infinity against codes of one sign: every score is
    -inf, whose softmax is NaN; a row that sees no position is 0, and rows
    beside it do not change."""
    planes, q = exact_scores(52, B, Tq, Hkv, G, D, Tmax, [(3, 1.0), (37, 1.0)])
    planes[0][...] = planes[0] & 0x77 | 0x11                          # codes -7, -5, -3, -1
    o_ref, ao, slack, floor = attention_ref(planes, q, lens, G, 0.25)
    q[:, :, 0] = 0x7c00
    o = run_attention(planes, q, lens, G, 0.25, f16)
    for b in range(B):
        for i in range(Tq):
            sees = lens[b] - (Tq - 1 - i) > 0
            assert np.isnan(o[b, i, 0]).all() if sees else not o[b, i, 0].any()
    o[:, :, 0] = o_ref[:, :, 0]
    check_attention(o, (o_ref, ao, np.full_like(slack, 2 * 2.0 ** -17), floor + 2.0 ** -31), f16)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("Tq,G,D,n", [(1, 4, 128, 70), (2, 4, 128, 65), (4, 2, 64, 33), (8, 5, 128, 300), (8, 4, 64, 64),
                                      (32, 2, 128, 97), (5, 3, 128, 4100), (3, 8, 128, 40)])
def test_value_scales_that_are_not_finite_stay_with_the_rows_that_see_them(Tq, G, D, n, f16):
    """NaN and infinite value scales at the last positions: a query token that
    does not see one is as accurate as without it, one that does is NaN in that
    block's 32 elements alone."""
    Hkv, Tmax, scale = 2, -(-n // 32) * 32, D ** -0.5
    planes = [p.copy() for p in random_cache_q4(54, 1, Hkv, Tmax, D)]
    q = q_bits(55, 1, Tq, Hkv * G, D)
    bad = [(n - 1, 0, 0x7e00), (n - 1, 1, 0x7c00), (n - 2, 1, 0xfc00), (n - Tq // 2 - 1, 0, 0x7c00), (n - Tq, D // 32 - 1, 0xfe00)]
    for t, j, bits in bad:
        planes[3][:, :, t, j] = 0                                     # (the reference: without them)
    o_ref, ao, slack, floor = attention_ref(planes, q, [n], G, scale)
    for t, j, bits in bad:
        planes[3][:, :, t, j] = bits
    o = run_attention(planes, q, [n], G, scale, f16)
    for i in range(Tq):
        nan = np.zeros(D, bool)
        for t, j, _ in bad:
            nan[32 * j:32 * j + 32] |= t < n - (Tq - 1 - i)
        assert np.isnan(o[0, i][:, nan]).all()
        o[0, i][:, nan] = o_ref[0, i][:, nan]
    check_attention(o, (o_ref, ao, slack, floor), f16)


@pytest.mark.parametrize("where", ["first", "last", "apart"])
@pytest.mark.parametrize("n", [1, 8])
def test_idle_slots_beside_live_sequences(where, n):
    """1000 slots, n of them live: the live ones' rows against fp64, the others 0."""
    B, Hkv, G, D, Tmax = 1000, 2, 3, 64, 512
    at = {"first": range(n), "last": range(B - n, B), "apart": range(3, B, B // n)}[where]
    part = random_cache_q4(56, n, Hkv, Tmax, D)
    planes = []
    for p in part:
        w = np.zeros((B, *p.shape[1:]), p.dtype)
        w[list(at)] = p
        planes.append(w)
    lens, live = np.zeros(B, np.int32), [512 - 37 * i for i in range(n)]
    lens[list(at)] = live
    q = q_bits(57, B, 1, Hkv * G, D)
    o = run_attention(planes, q, lens, G, 0.125)
    check_attention(o[list(at)], attention_ref(part, q[list(at)], live, G, 0.125), True)
    o[list(at)] = 0
    assert not o.any()


def test_idle_slots_behind_the_live_ones_are_not_walked():
    """Seen by the time: 8 sequences at the front of 1000 slots take less than
    twice as long as at the back, where a walk over the idle slots behind them, a
    load after another, takes five times as long."""
    import torch
    B, Hkv, G, D, Tmax = 1000, 8, 5, 128, 4096
    planes = [torch.zeros((B, Hkv, Tmax, D // n), dtype=t, device=DEV) for n, t in ((2, torch.uint8), (32, torch.int16)) * 2]
    kv = bq.kv_cache_q4(*planes)
    q = to_dev(q_bits(58, B, Hkv * G, D))
    o = torch.zeros((B, Hkv * G, D), device=DEV)
    ws = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(D, 1, G), DEV)

    def us(first):
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        lens[first:first + 8] = Tmax
        best = float("inf")
        for _ in range(8):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            for _ in range(8):                        # (8 launches: the device, not the host's calls)
                bq.attn_decode_q4(kv, q, lens, G, 0.09, o, ws)
            e[1].record()
            torch.cuda.synchronize()
            best = min(best, e[0].elapsed_time(e[1]) * 125)
        return best

    us(0)
    front, back = us(0), us(B - 8)
    assert front < 2 * back, (front, back)


@pytest.mark.parametrize("B,Hkv,Tmax,lens", [
    # segments of 48, 33, 32 and 31 units, two cuts beside one, long ones between short ones
    (19, 8, 1536, [1536] * 19), (19, 8, 1056, [1056] * 19), (19, 8, 1024, [1024] * 19), (38, 4, 992, [992 - i for i in range(38)]),
    (24, 8, 1088, [960 + (37 * i) % 129 for i in range(24)]), (40, 4, 4096, [4096 if i % 10 == 3 else 300 + 40 * i for i in range(40)]),
])
def test_numbers_of_segments_just_above_the_grid(B, Hkv, Tmax, lens):
    planes = random_cache_q4(59, B, Hkv, Tmax, 64)
    q = q_bits(60, B, 1, Hkv, 64)
    o = run_attention(planes, q, lens, 1, 0.125, False)
    check_attention(o, attention_ref(planes, q, lens, 1, 0.125), False)


@pytest.mark.parametrize("bits", [0x7e00, 0x7c00, 0xfc00])
@pytest.mark.parametrize("Tq,G,D,n", [(2, 4, 128, 65), (8, 5, 128, 300), (4, 2, 64, 33)])
def test_key_scales_that_are_not_finite_stay_with_the_rows_that_see_them(Tq, G, D, n, bits):
    """The last token's own key scale: earlier tokens are as accurate as without
    it, the last is NaN where the scale is."""
    Hkv, Tmax, scale = 2, -(-n // 32) * 32, D ** -0.5
    planes = [p.copy() for p in random_cache_q4(61, 1, Hkv, Tmax, D)]
    q = q_bits(62, 1, Tq, Hkv * G, D)
    ref = [r[:, :-1] for r in attention_ref(planes, q, [n], G, scale)]
    planes[1][:, :, n - 1, 1] = bits
    o = run_attention(planes, q, [n], G, scale)
    check_attention(o[:, :-1], ref, True)
    if bits == 0x7e00:
        assert np.isnan(o[:, -1]).all()


def test_more_sequences_than_a_grid_has_rows():
    """70000 sequences, 150 of them with positions."""
    B, Hkv, G, D, Tmax = 70000, 1, 2, 64, 32
    r = np.random.default_rng(63)
    at = np.sort(r.choice(B, 150, replace=False))
    at[0], at[-1] = 0, B - 1
    part = random_cache_q4(64, 150, Hkv, Tmax, D)
    planes = []
    for p in part:
        w = np.zeros((B, *p.shape[1:]), p.dtype)
        w[at] = p
        planes.append(w)
    lens, live = np.zeros(B, np.int32), r.integers(1, 33, 150)
    lens[at] = live
    q = q_bits(65, B, 1, Hkv * G, D)
    o = run_attention(planes, q, lens, G, 0.125)
    check_attention(o[at], attention_ref(part, q[at], live, G, 0.125), True)
    o[at] = 0
    assert not o.any()
