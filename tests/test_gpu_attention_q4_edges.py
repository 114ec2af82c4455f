"""Decode attention over a Q4 KV cache (bq_attn_decode_q4) where its rounding,
its reference and its masks can go wrong: fp16 output against fp32 output, the
same contents in caches of other sizes."""
import numpy as np
import pytest

from tests.kv_helpers import random_cache_q4, run_attention

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
