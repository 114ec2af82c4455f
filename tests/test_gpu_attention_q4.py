"""Decode attention over a Q4 KV cache (bq_attn_decode_q4) against fp64, over
head widths and groupings, lengths around the 32-position work unit, several
query tokens, masks that leave rows empty, unusual scales, streams, graphs and
workspaces.  The tolerance is derived in kv_helpers.check_attention."""
import numpy as np
import pytest

from quantised_weight_gemv_b200 import bq
from tests.gpu_helpers import DEV
from tests.kv_helpers import attention_ref, check_attention, random_cache_q4, run_attention, to_dev

pytestmark = pytest.mark.gpu


def q_bits(seed, *shape, size=1.0):
    return (np.random.default_rng(seed).standard_normal(shape) * size).astype(np.float16).view(np.uint16)


CASES = [
    # B, Tq, Hkv, G, D, Tmax, lens
    (1, 1, 1, 1, 128, 32, [1]),
    (1, 1, 1, 1, 64, 32, [32]),
    (2, 1, 2, 4, 128, 64, [33, 31]),
    (3, 1, 1, 5, 128, 96, [64, 65, 2]),
    (1, 1, 4, 8, 128, 4096, [4095]),
    (1, 1, 8, 5, 128, 4096, [4096]),
    (5, 1, 3, 7, 64, 160, [160, 1, 95, 0, 17]),
    (1, 1, 2, 9, 128, 1024, [1000]),
    (2, 1, 1, 16, 64, 2048, [2048, 777]),
    (2, 2, 2, 4, 128, 256, [200, 1]),
    (1, 4, 2, 5, 128, 512, [511]),
    (3, 8, 2, 5, 128, 288, [288, 7, 130]),
    (1, 3, 1, 6, 64, 320, [300]),
    (1, 32, 1, 16, 128, 128, [100]),
    (2, 32, 2, 1, 64, 64, [40, 20]),
    (1, 7, 1, 11, 128, 9600, [9533]),
    (2, 8, 2, 6, 128, 2048, [2048, 33]),
    (1, 7, 2, 8, 64, 1024, [1023]),
    (2, 9, 1, 8, 128, 512, [500, 8]),
    (3, 3, 3, 8, 128, 800, [800, 33, 790]),
    (40, 1, 2, 2, 128, 64, [(7 * i) % 65 for i in range(40)]),
    (300, 1, 2, 1, 64, 32, [(5 * i) % 33 for i in range(300)]),
    (2, 1, 1, 4, 128, 32768, [32768, 5]),
    (6, 1, 4, 3, 128, 2048, [2048, 0, 1, 1999, 0, 640]),
    # shares: segments with CTAs of their own, short ones that are not cut, long and short mixed
    (9, 1, 2, 4, 128, 8192, [8192, 8191, 4097, 33, 8000, 7777, 6000, 1, 8192]),
    (100, 1, 3, 2, 64, 1024, [(37 * i) % 1025 for i in range(100)]),
    (70, 1, 1, 5, 128, 4096, [4096 if i % 9 == 4 else (11 * i) % 200 for i in range(70)]),
    (33, 2, 4, 3, 128, 1056, [1056 - i for i in range(33)]),
    # two row tiles a warp with one fp16 term a weight (more than 2^17 cached positions)
    (4, 4, 3, 4, 128, 16384, [16384, 100, 9001, 0]),
    (5, 3, 2, 8, 64, 16384, [2, 16383, 700, 12000, 33]),
    # segments kept whole or split where there are few units
    (1, 1, 2, 4, 128, 384, [384]),
    (1, 1, 2, 4, 128, 416, [413]),
    (3, 1, 2, 2, 64, 512, [12, 385, 512]),
    (2, 4, 1, 12, 128, 1024, [1024, 350]),
    (1, 8, 2, 8, 128, 640, [640]),
    # numbers of sequences around those a plan's lane holds, empty ones among them
    (32, 1, 2, 2, 64, 256, [(91 * i) % 257 for i in range(32)]),
    (64, 1, 2, 4, 64, 512, [(i % 5 != 0) * ((77 * i) % 513) for i in range(64)]),
    (128, 1, 1, 3, 128, 320, [(i > 60) * ((53 * i) % 321) for i in range(128)]),
    (128, 1, 1, 1, 64, 2048, [2048 if i in (3, 77, 127) else 0 for i in range(128)]),
    (129, 1, 2, 1, 64, 96, [(29 * i) % 97 for i in range(129)]),
    (130, 1, 1, 2, 64, 4096, [4000 if i in (0, 64, 129) else 0 for i in range(130)]),
]


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("B,Tq,Hkv,G,D,Tmax,lens", CASES)
def test_parity(B, Tq, Hkv, G, D, Tmax, lens, f16):
    planes = random_cache_q4(B + 10 * Tmax + G, B, Hkv, Tmax, D)
    q = q_bits(Tmax + Tq, B, Tq, Hkv * G, D)
    o = run_attention(planes, q, lens, G, D ** -0.5, f16)
    check_attention(o, attention_ref(planes, q, lens, G, D ** -0.5), f16)


def test_lengths_are_clamped_and_rows_without_positions_are_zero():
    planes = random_cache_q4(3, 4, 2, 64, 128)
    q = q_bits(4, 4, 3, 4, 128)
    lens = [-5, 1000, 2, 0]
    o = run_attention(planes, q, lens, 2, 0.1, False)
    check_attention(o, attention_ref(planes, q, lens, 2, 0.1), False)
    assert not o[0].any() and not o[3].any()
    assert not o[2, 0].any() and o[2, 1].any() and o[2, 2].any()      # tokens 1 and 2 see 1 and 2 positions


@pytest.mark.parametrize("Tq", [1, 4])
def test_nothing_at_or_past_the_length_reaches_the_result(Tq):
    planes = [p.copy() for p in random_cache_q4(5, 3, 2, 128, 128)]
    q = q_bits(6, 3, Tq, 8, 128)
    lens = [77, 33, 128]
    a = run_attention(planes, q, lens, 4, 0.09)
    for b, n in enumerate(lens):
        planes[0][b, :, n:] = 0xff
        planes[1][b, :, n:] = 0x7c00                                   # inf
        planes[2][b, :, n:] = 0x07
        planes[3][b, :, n:] = 0x7e00                                   # NaN
    assert np.array_equal(a, run_attention(planes, q, lens, 4, 0.09))


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("scale,k_size,v_size,q_size", [
    (2.0, 1.0, 1.0, 1.0),          # scores of order 100: one position takes all
    (0.0, 1.0, 1.0, 1.0),          # equal weights
    (-0.1, 1.0, 1.0, 1.0),
    (0.088, 1.0, 1e-4, 1.0),       # value scales deep in fp16's subnormals' neighbourhood
    (0.088, 1.0, 3e4, 1e-3),
    (3e3, 3e-3, 1.0, 2e-3),        # small queries and keys, a large softmax scale
    (1e-8, 3e4, 1.0, 3e3),
])
def test_sizes_of_scores_and_values(scale, k_size, v_size, q_size, f16):
    planes = random_cache_q4(7, 2, 2, 512, 128, k_size, v_size)
    q = q_bits(8, 2, 1, 8, 128, size=q_size)
    lens = [512, 300]
    o = run_attention(planes, q, lens, 4, scale, f16)
    if f16 and v_size > 1e4:
        o = np.clip(o, -65504, 65504)
    check_attention(o, attention_ref(planes, q, lens, 4, scale), f16)


@pytest.mark.parametrize("f16", [True, False])
def test_value_scales_far_apart(f16):
    """Positions and blocks whose value scales differ by factors of up to 2^12,
    some zero: the dominant position may have the smallest values."""
    planes = [p.copy() for p in random_cache_q4(9, 1, 2, 256, 128)]
    r = np.random.default_rng(10)
    f = np.exp2(r.integers(-12, 1, planes[3].shape)).astype(np.float64)
    vs = (planes[3].view(np.float16).astype(np.float64) * f).astype(np.float16)
    vs[0, :, ::7] = 0
    vs[0, 1, :, 2] = 0
    planes[3] = vs.view(np.uint16)
    q = q_bits(11, 1, 2, 10, 128)
    for scale in (0.088, 1.0):
        o = run_attention(planes, q, [256], 5, scale, f16)
        check_attention(o, attention_ref(planes, q, [256], 5, scale), f16)


def test_zero_caches_and_zero_queries():
    planes = [p.copy() for p in random_cache_q4(12, 2, 1, 96, 64)]
    planes[1][0] = 0                                                  # all keys 0: plain mean
    planes[3][1] = 0                                                  # all values 0
    q = q_bits(13, 2, 1, 3, 64)
    q[0, 0, 1] = 0
    o = run_attention(planes, q, [90, 90], 3, 0.125, False)
    check_attention(o, attention_ref(planes, q, [90, 90], 3, 0.125), False)
    assert not o[1].any()


@pytest.mark.parametrize("f16", [True, False])
def test_negative_scales(f16):
    """Scales of either sign (a cache written by hand): the largest magnitude of
    a unit's value scales is a negative one's, or a positive one's beside them."""
    planes = [p.copy() for p in random_cache_q4(21, 2, 2, 128, 128)]
    planes[1][:, :, ::3] ^= 0x8000
    planes[3][0, :, ::2] ^= 0x8000
    planes[3][1, :, 1:] |= 0x8000
    vs = planes[3].view(np.float16)
    vs[0, :, 5] *= np.float16(-900)
    vs[1, :, 0] *= np.float16(900)
    q = q_bits(22, 2, 1, 8, 128)
    o = run_attention(planes, q, [128, 100], 4, 0.088, f16)
    check_attention(o, attention_ref(planes, q, [128, 100], 4, 0.088), f16)


@pytest.mark.parametrize("f16", [True, False])
def test_values_that_are_not_finite_stay_in_their_head_and_query_row(f16):
    B, Hkv, G, Tmax = 2, 3, 4, 2048
    planes = random_cache_q4(23, B, Hkv, Tmax, 128)
    q = q_bits(24, B, 1, Hkv * G, 128)
    lens = [2000, 70]
    clean = run_attention(planes, q, lens, G, 0.088, f16)
    bad = [p.copy() for p in planes]
    bad[1][0, 1, 777, 2] = 0x7e00                                     # a NaN key scale: head 1 of sequence 0
    bad[3][1, 2, 33] = 0x7e00                                         # NaN value scales: head 2 of sequence 1
    o = run_attention(bad, q, lens, G, 0.088, f16).reshape(B, Hkv, G, 128)
    want = clean.reshape(B, Hkv, G, 128)
    for b, h in np.ndindex(B, Hkv):
        if (b, h) in ((0, 1), (1, 2)):
            assert np.isnan(o[b, h]).all()
        else:
            assert np.array_equal(o[b, h], want[b, h])
    qn = q.copy()
    qn[0, 0, 5, 9], qn[1, 0, 2, 100] = 0x7e00, 0x7c00                 # NaN, inf
    o, want = run_attention(planes, qn, lens, G, 0.088, f16), clean
    for b, i in np.ndindex(B, Hkv * G):
        if (b, i) in ((0, 5), (1, 2)):
            assert np.isnan(o[b, 0, i]).all()
        else:
            assert np.allclose(o[b, 0, i], want[b, 0, i], rtol=2.0 ** -10, atol=2.0 ** -12)


def test_determinism_and_one_workspace_for_all_shapes():
    import torch
    ws = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(128, 32, 16), DEV)
    outs = []
    for _ in range(2):
        for B, Tq, Hkv, G, D, Tmax, lens in [(2, 1, 4, 4, 128, 8192, [8192, 7001]), (1, 8, 2, 8, 128, 1024, [1000]),
                                             (9, 1, 2, 3, 64, 64, list(range(9)))]:
            planes = random_cache_q4(14, B, Hkv, Tmax, D)
            outs.append(run_attention(planes, q_bits(15, B, Tq, Hkv * G, D), lens, G, 0.1, False, ws=ws))
    assert int(ws.count_nonzero().item()) == 0
    for a, b in zip(outs[:3], outs[3:]):
        assert np.array_equal(a, b)
    torch.cuda.synchronize()


def test_two_streams_with_two_workspaces_and_a_replayed_graph():
    """Two captured calls with a workspace each, replayed at once on two
    streams while the lengths change between replays."""
    import torch
    B, Hkv, G, D, Tmax = 2, 4, 4, 128, 4096
    planes = random_cache_q4(16, B, Hkv, Tmax, D)
    kv = bq.kv_cache_q4(*[to_dev(p) for p in planes])
    q = q_bits(17, B, 1, Hkv * G, D)
    qd = to_dev(q)
    runs = []
    for _ in range(2):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        o = torch.empty(q.shape, dtype=torch.float32, device=DEV)
        ws = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(D, 1, G), DEV)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            bq.attn_decode_q4(kv, qd, lens, G, 0.088, o, ws)
        runs.append((s, g, lens, o, ws))
    for n in ([4096, 1], [0, 33], [2050, 4001]):
        for k, (s, g, lens, o, ws) in enumerate(runs):
            lens.copy_(torch.tensor(n if k == 0 else n[::-1], dtype=torch.int32))
        torch.cuda.synchronize()
        for s, g, *_ in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for k, (s, g, lens, o, ws) in enumerate(runs):
            check_attention(o.cpu().numpy(), attention_ref(planes, q, n if k == 0 else n[::-1], G, 0.088), False)
            assert int(ws.count_nonzero().item()) == 0


def test_cache_offsets_past_32_bits():
    """A cache whose third sequence starts 2^32 bytes into the code planes."""
    import torch
    B, Hkv, Tmax, D, G, n = 3, 1, 1 << 25, 128, 4, 100
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB of free device memory")
    part = random_cache_q4(18, 1, 1, n, D)
    full = []
    for p in part:
        t = torch.empty((B, Hkv, Tmax, p.shape[-1]), dtype=torch.int16 if p.dtype == np.uint16 else torch.uint8, device=DEV)
        t[2, 0, :n] = to_dev(p)[0, 0]
        full.append(t)
    q = q_bits(19, B, 1, G, D)
    o = torch.full(q.shape, float("nan"), dtype=torch.float32, device=DEV)
    ws = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(D, 1, G), DEV)
    bq.attn_decode_q4(bq.kv_cache_q4(*full), to_dev(q), torch.tensor([0, 0, n], dtype=torch.int32, device=DEV), G, 0.1, o, ws)
    torch.cuda.synchronize()
    check_attention(o[2:].cpu().numpy(), attention_ref(part, q[2:], [n], G, 0.1), False)
    assert not o[:2].any().item()
