"""Writing and reading the KV caches at the edges of what a call names: rows from
a sequence's count on, offsets past 32 bits in the Q8 cache and in rows."""
import numpy as np
import pytest

import oracle
from quantised_weight_gemv_b200 import bq
from tests.gpu_helpers import DEV
from tests.kv_helpers import deq_q4, quant_rows
from tests.test_gpu_kv_cache import dtype, ints, make_kv, new_cache, place, planes_of, rows, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt,B,T,Hkv,D,Tmax,start,count", [
    (4, 4, 40, 3, 128, 64, [0, 20, 3, 63], [0, 1, 33, 1]),
    (4, 3, 70, 2, 64, 128, [5, 0, 60], [17, 64, 3]),
    # four rows a thread: counts at, one short of and one past a block's and a warp's rows
    (4, 8, 1400, 5, 128, 1408, [0, 1, 0, 3, 0, 0, 5, 8], [0, 1, 16, 17, 63, 64, 65, 1400]),
    (4, 6, 2600, 5, 64, 2624, [0, 7, 0, 0, 24, 0], [1, 127, 128, 129, 2600, 0]),
    (8, 4, 300, 2, 128, 384, [0, 77, 3, 84], [0, 1, 129, 300]),
])
def test_rows_from_the_count_on_do_not_matter(fmt, B, T, Hkv, D, Tmax, start, count, src):
    """They hold NaN: nothing of them is stored or reported."""
    planes = new_cache(fmt, B, Hkv, Tmax, D)
    kv = make_kv(fmt, planes)
    k, v, kf, vf = rows(60 + T, B, T, Hkv, D, src)
    k, v = k.clone(), v.clone()
    for b, n in enumerate(count):
        k[b, n:], v[b, n:] = float("nan"), float("nan")
    st = status()
    bq.kv_append(kv, k, v, ints(start), ints(count), st)
    assert int(st.item()) == 0
    for got, w in zip(planes_of(kv), place(fmt, planes, kf, vf, start, count)):
        assert np.array_equal(got, w)


@pytest.mark.parametrize("src", ["f32", "f16"])
@pytest.mark.parametrize("fmt", [4, 8])
def test_rows_from_the_count_on_are_not_read(fmt, src):
    """Seen by the time: 16 sequences of 4096 rows, 0.27 or 0.54 GB, with a count
    of 1 each take less than half of what all rows take, where reading them all
    takes as long."""
    import torch
    B, T, H, D = 16, 4096, 8, 128
    kv = make_kv(fmt, new_cache(fmt, B, H, T, D, fill=0))
    x = torch.randn((B, T, 2 * H, D), device=DEV).to(dtype(src))
    start = ints([0] * B)

    def us(count):
        best = float("inf")
        for _ in range(8):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            for _ in range(4):                        # (4 launches: the device, not the host's calls)
                bq.kv_append(kv, x[:, :, :H], x[:, :, H:], start, count)
            e[1].record()
            torch.cuda.synchronize()
            best = min(best, e[0].elapsed_time(e[1]) * 250)
        return best

    us(None)
    every, few = us(None), us(ints([1] * B))
    assert few < every / 2, (few, every)


@pytest.mark.parametrize("T", [3, 100])
def test_q8_cache_offsets_past_32_bits(T):
    """A Q8 cache whose third sequence starts 2^32 bytes into the code planes."""
    import torch
    B, H, Tmax, D = 3, 1, 1 << 24, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free device memory")
    refs = [torch.empty(s, dtype=t, device=DEV) for s, t in
            (((B, H, Tmax, D), torch.int8), ((B, H, Tmax, D // 32), torch.int16),
             ((B, H, D, Tmax), torch.int8), ((B, H, Tmax, D // 32), torch.int16))]
    kv = bq.kv_cache(*refs)
    k, v, kf, vf = rows(70, B, T, H, D, "f32")
    start = [0, 5, Tmax - T]
    bq.kv_append(kv, k, v, ints(start))
    ko, vo = torch.zeros((B, T, H, D), device=DEV), torch.zeros((B, T, H, D), device=DEV)
    bq.kv_read(kv, ko, vo, ints(start))
    for x, y in ((kf, ko), (vf, vo)):
        c, s = quant_rows(8, x)
        want = c.view(np.int8).astype(np.float64) * oracle.half_to_double(s).repeat(32, -1)
        assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", [4, 8])
def test_row_offsets_past_32_bits(fmt):
    """Source and destination rows 2^32 elements apart (8.6 GB of fp16)."""
    import torch
    D, far = 128, 1 << 32
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free device memory")
    buf = torch.empty(far + 2 * D, dtype=torch.float16, device=DEV)
    src = buf.as_strided((1, 2, 1, D), (far + 2 * D, far, D, 1))        # two tokens
    seq = buf.as_strided((2, 1, 1, D), (far, D, D, 1))                  # two sequences
    x = torch.from_numpy(np.random.default_rng(71).standard_normal((2, D)).astype(np.float16)).to(DEV)
    for rows_, B in ((src, 1), (seq, 2)):
        T = 2 // B
        rows_.copy_(x.view(B, T, 1, D))
        kv = make_kv(fmt, new_cache(fmt, B, 1, 128, D))
        bq.kv_append(kv, rows_, rows_, ints([9] * B))
        want = place(fmt, new_cache(fmt, B, 1, 128, D), *[x.float().cpu().numpy().reshape(B, T, 1, D)] * 2, [9] * B, [T] * B)
        for got, w in zip(planes_of(kv), want):
            assert np.array_equal(got, w)
        rows_.zero_()
        ko = torch.zeros((B, T, 1, D), dtype=torch.float16, device=DEV)
        bq.kv_read(kv, ko, rows_, ints([9] * B))
        assert torch.equal(ko, rows_) and bool((ko != 0).any(-1).all())


@pytest.mark.parametrize("fmt,D,Tmax", [(4, 64, 32), (8, 128, 128)])
def test_more_sequences_than_a_grid_has_rows(fmt, D, Tmax):
    """70000 sequences: a token each at odd places, some with none."""
    import torch
    B = 70000
    kv = make_kv(fmt, new_cache(fmt, B, 1, Tmax, D))
    k, v, kf, vf = rows(72, B, 1, 1, D, "f16")
    start, count = np.arange(B) * 7 % Tmax, (np.arange(B) % 5 != 2).astype(np.int32)
    st = status()
    bq.kv_append(kv, k, v, ints(start), ints(count), st)
    assert int(st.item()) == 0
    for got, w in zip(planes_of(kv), place(fmt, new_cache(fmt, B, 1, Tmax, D), kf, vf, start, count)):
        assert np.array_equal(got, w)
    ko, vo = torch.zeros((B, 1, 1, D), device=DEV), torch.zeros((B, 1, 1, D), device=DEV)
    bq.kv_read(kv, ko, vo, ints(start), ints(count), st)
    assert int(st.item()) == 0
    for x, y in ((kf, ko), (vf, vo)):
        c, s = quant_rows(fmt, x)
        want = (deq_q4(c, s) if fmt == 4 else c.view(np.int8) * oracle.half_to_double(s).repeat(32, -1))
        assert np.array_equal(y.cpu().numpy(), want * count[:, None, None, None])
