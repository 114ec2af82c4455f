"""Writing the Q4 and Q8 KV caches (bq_kv_append_*) and reading them back
(bq_kv_read_*): codes and scales bit for bit those of the oracle's quantisers,
every other byte of the cache and of the destination untouched, over element
types, strides, odd starts, ragged counts, positions outside the cache, values
that cannot be quantised, streams and graphs; and the whole path together
(append, attention, read back) as a decode loop runs it."""
import numpy as np
import pytest

import oracle
from quantised_weight_gemv_b200 import bq
from tests.gpu_helpers import DEV
from tests.kv_helpers import attention_ref, check_attention, deq_q4, quant_rows, to_dev
from tests.test_gpu_attention import REL, ABS

pytestmark = pytest.mark.gpu
TORCH = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def dtype(name):
    import torch
    return getattr(torch, TORCH[name])


def new_cache(fmt, B, Hkv, Tmax, D, fill=0x5a):
    """Planes filled with one byte, as numpy arrays in the cache's layouts."""
    nb = D // 32
    codes = [(B, Hkv, Tmax, D // 2)] * 2 if fmt == 4 else [(B, Hkv, Tmax, D), (B, Hkv, D, Tmax)]
    planes = []
    for s in codes:
        planes += [np.full(s, fill, np.uint8), np.full((B, Hkv, Tmax, nb), fill * 257, np.uint16)]
    return planes


def make_kv(fmt, planes):
    return (bq.kv_cache_q4 if fmt == 4 else bq.kv_cache)(*[to_dev(p) for p in planes])


def planes_of(kv):
    return [t.cpu().numpy().view(np.uint16 if t.element_size() == 2 else np.uint8) for t in kv._refs]


def place(fmt, planes, k, v, start, count):
    """The planes after appending fp32 rows k, v [B, T, Hkv, D], by the oracle's quantiser."""
    planes = [p.copy() for p in planes]
    Tmax = planes[0].shape[2]
    for plane, x in ((0, k), (2, v)):
        c, s = quant_rows(fmt, x)
        c = c.view(np.uint8)
        for b in range(x.shape[0]):
            for i in range(min(max(int(count[b]), 0), x.shape[1])):
                p = int(start[b]) + i
                if not 0 <= p < Tmax:
                    continue
                if fmt == 8 and plane == 2:
                    planes[2][b, :, :, p] = c[b, i]
                else:
                    planes[plane][b, :, p] = c[b, i]
                planes[plane + 1][b, :, p] = s[b, i]
    return planes


def rows(seed, B, T, H, D, src, gap=0):
    """k, v as slices of one projection output on the device, and as fp32 numpy."""
    import torch
    r = np.random.default_rng(seed)
    x = r.standard_normal((B, T, 3 * H + gap, D)) * np.exp2(r.integers(-6, 6, (B, T, 3 * H + gap, D // 32))).repeat(32, -1)
    d = torch.from_numpy(x.astype(np.float32)).to(DEV).to(dtype(src))
    k, v = d[:, :, H:2 * H], d[:, :, 2 * H:3 * H]
    return k, v, k.float().cpu().numpy(), v.float().cpu().numpy()


def ints(a):
    return to_dev(np.asarray(a, dtype=np.int32))


def status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device=DEV)


APPENDS = [
    # fmt, B, T, Hkv, D, Tmax, start, count
    (4, 1, 1, 1, 64, 32, [0], None),
    (4, 3, 1, 5, 128, 96, [95, 0, 33], None),
    (4, 2, 37, 2, 128, 64, [11, 27], [37, 5]),
    (4, 2, 64, 3, 64, 64, [0, 0], [64, 0]),
    (4, 1, 1025, 4, 128, 2048, [777], None),
    # enough rows for four a thread
    (4, 2, 2051, 5, 128, 2112, [13, 0], [2051, 1999]),
    (4, 3, 2600, 5, 64, 2624, [24, 0, 7], [2600, 0, 2593]),
    (8, 1, 1, 1, 128, 128, [127], None),
    (8, 4, 1, 3, 128, 256, [0, 63, 64, 200], [1, 1, 0, 1]),
    (8, 2, 37, 2, 128, 128, [11, 91], [37, 5]),
    (8, 2, 130, 2, 128, 256, [126, 3], [130, 129]),
    (8, 1, 1025, 2, 128, 2048, [1023], None),
]


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt,B,T,Hkv,D,Tmax,start,count", APPENDS)
def test_append_is_bit_exact_and_touches_nothing_else(fmt, B, T, Hkv, D, Tmax, start, count, src):
    planes = new_cache(fmt, B, Hkv, Tmax, D)
    kv = make_kv(fmt, planes)
    k, v, kf, vf = rows(T + Tmax, B, T, Hkv, D, src)
    st = status()
    bq.kv_append(kv, k, v, ints(start), None if count is None else ints(count), st)
    want = place(fmt, planes, kf, vf, start, count or [T] * B)
    assert int(st.item()) == 0
    for got, w in zip(planes_of(kv), want):
        assert np.array_equal(got, w)


def values(fmt, planes, b, h, p):
    """fp64 key and value of one position."""
    if fmt == 4:
        return [deq_q4(planes[i][b, h, p], planes[i + 1][b, h, p]) for i in (0, 2)]
    c = [planes[0][b, h, p], planes[2][b, h, :, p]]
    return [c[i].view(np.int8).astype(np.float64) * oracle.half_to_double(planes[2 * i + 1][b, h, p]).repeat(32)
            for i in range(2)]


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt,B,T,Hkv,D,Tmax,start,count", APPENDS)
def test_read_is_exact_and_leaves_other_rows(fmt, B, T, Hkv, D, Tmax, start, count, out):
    import torch
    r = np.random.default_rng(Tmax)
    planes = new_cache(fmt, B, Hkv, Tmax, D)
    for i in (0, 2):                                  # every code, scales of all sizes (subnormal ones too)
        planes[i][:] = r.integers(0, 256, planes[i].shape)
        planes[i + 1][:] = r.integers(0, 0x6000, planes[i + 1].shape)
    kv = make_kv(fmt, planes)
    ko = torch.full((B, T, Hkv, D), 7.0, dtype=dtype(out), device=DEV)
    wide = torch.full((B, T, Hkv + 1, D + 32), 7.0, dtype=dtype(out), device=DEV)
    vo = wide[:, :, 1:, :D]                           # a strided destination
    st = status()
    bq.kv_read(kv, ko, vo, ints(start), None if count is None else ints(count), st)
    assert int(st.item()) == 0
    want = np.full((2, B, T, Hkv, D), 7.0)
    for b in range(B):
        for i in range(T if count is None else count[b]):
            for h in range(Hkv):
                want[:, b, i, h] = values(fmt, planes, b, h, start[b] + i)
    want = torch.from_numpy(want).to(torch.float32).to(dtype(out))     # values are exact in fp32
    assert torch.equal(ko.cpu(), want[0]) and torch.equal(vo.cpu(), want[1])
    assert bool((wide[:, :, 0] == 7).all()) and bool((wide[..., D:] == 7).all())
    only = torch.full_like(ko, 7.0)
    bq.kv_read(kv, None, only, ints(start), None if count is None else ints(count))
    assert torch.equal(only.cpu(), want[1])
    only.fill_(7)
    bq.kv_read(kv, only, None, ints(start), None if count is None else ints(count))
    assert torch.equal(only.cpu(), want[0])


@pytest.mark.parametrize("fmt", [4, 8])
def test_rounding_next_to_halves_is_the_quantisers(fmt):
    """Rows made of quotients at and one fp32 step either side of every half:
    where a quotient by a reciprocal would round the other way."""
    import torch
    L = 7 if fmt == 4 else 127
    rng = np.random.default_rng(1)
    out = []
    for d in np.concatenate([rng.uniform(2.0 ** -14, 60, 300), np.exp2(rng.uniform(-24, -14, 60)), [2.0 ** -24, 3 * 2.0 ** -24]]):
        d = np.float32(np.float16(d))
        if d == 0:
            continue
        half = (rng.integers(-L, L, 31) + 0.5).astype(np.float64) * np.float64(d)
        x = half.astype(np.float32)
        x = np.where(rng.integers(0, 3, 31) == 0, np.nextafter(x, np.float32(np.inf)), x)
        x = np.where(rng.integers(0, 3, 31) == 0, np.nextafter(x, np.float32(-np.inf)), x)
        out.append(np.concatenate([[np.float32(L) * d], x]).astype(np.float32))
    out = np.stack(out)
    T = len(out) // 4
    x = out[:4 * T].reshape(1, T, 1, 128)
    Tmax = 128
    planes = new_cache(fmt, 1, 1, Tmax, 128)
    kv = make_kv(fmt, planes)
    xd = torch.from_numpy(x).to(DEV)
    st = status()
    bq.kv_append(kv, xd, -xd, ints([5]), None, st)
    assert int(st.item()) == 0
    for got, w in zip(planes_of(kv), place(fmt, planes, x, -x, [5], [T])):
        assert np.array_equal(got, w)


@pytest.mark.parametrize("fmt", [4, 8])
def test_zero_tiny_and_unquantisable_blocks(fmt):
    """Zero blocks, scales that round to zero or to a subnormal; then NaN, inf
    and a scale beyond fp16, which are stored as zeros and reported."""
    import torch
    x = np.zeros((1, 6, 1, 128), dtype=np.float32)
    x[0, 1, 0, :32] = 1e-9
    x[0, 2, 0, 32:64] = np.linspace(-1e-6, 1e-6, 32)
    x[0, 3] = np.random.default_rng(0).standard_normal(128)
    planes = new_cache(fmt, 1, 1, 128, 128)
    kv = make_kv(fmt, planes)
    st = status()
    xd = torch.from_numpy(x).to(DEV)
    bq.kv_append(kv, xd, xd, ints([3]), None, st)
    assert int(st.item()) == 0
    for got, w in zip(planes_of(kv), place(fmt, planes, x, x, [3], [6])):
        assert np.array_equal(got, w)
    bad = x.copy()
    bad[0, 3, 0, 5], bad[0, 4, 0, 40], bad[0, 5, 0, 127] = np.nan, -np.inf, 3e7
    clean = bad.copy()
    clean[0, 3, 0, :32], clean[0, 4, 0, 32:64], clean[0, 5, 0, 96:] = 0, 0, 0
    kv = make_kv(fmt, planes)
    bd = torch.from_numpy(bad).to(DEV)
    bq.kv_append(kv, bd, bd, ints([3]), None, st)
    assert int(st.item()) == 1 << bq.BQ_ERR_RANGE
    for got, w in zip(planes_of(kv), place(fmt, planes, clean, clean, [3], [6])):
        assert np.array_equal(got, w)


BAD_PLACES = [([-3, 0], [5, 5], True), ([126, 0], [5, 5], True), ([128, 2], [1, 1], True),
              ([2 ** 31 - 1, -2 ** 31], [5, 5], True), ([0, 1], [6, 5], True), ([0, 1], [-1, 5], True),
              ([123, 0], [5, 0], False), ([500, 0], [0, 5], False)]


@pytest.mark.parametrize("start,count,flag", BAD_PLACES)
@pytest.mark.parametrize("fmt", [4, 8])
def test_positions_outside_the_cache_are_skipped_and_reported(fmt, start, count, flag):
    import torch
    B, T, H, D, Tmax = 2, 5, 2, 128, 128
    planes = new_cache(fmt, B, H, Tmax, D, fill=0x11)
    kv = make_kv(fmt, planes)
    k, v, kf, vf = rows(9, B, T, H, D, "f32")
    st = status()
    bq.kv_append(kv, k, v, ints(start), ints(count), st)
    assert int(st.item()) == (1 << bq.BQ_ERR_POSITION if flag else 0)
    want = place(fmt, planes, kf, vf, start, count)
    for got, w in zip(planes_of(kv), want):
        assert np.array_equal(got, w)
    ko = torch.full((B, T, H, D), 7.0, device=DEV)
    vo = ko.clone()
    st = status()
    bq.kv_read(kv, ko, vo, ints(start), ints(count), st)
    assert int(st.item()) == (1 << bq.BQ_ERR_POSITION if flag else 0)
    ref = np.full((2, B, T, H, D), 7.0)
    for b in range(B):
        for i in range(min(max(count[b], 0), T)):
            if 0 <= start[b] + i < Tmax:
                for h in range(H):
                    ref[:, b, i, h] = values(fmt, want, b, h, start[b] + i)
    assert np.array_equal(ko.cpu().numpy(), ref[0]) and np.array_equal(vo.cpu().numpy(), ref[1])
    bq.kv_append(kv, k, v, ints(start), ints(count))                    # no status word: same, unreported
    torch.cuda.synchronize()


@pytest.mark.parametrize("src", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", [4, 8])
def test_every_16_bit_magnitude_as_a_block_maximum(fmt, src):
    """Block i's largest magnitude is 16-bit pattern i, its other elements random
    parts of it: scales (subnormal and zero ones among them) and codes are the
    quantiser's; blocks whose scale overflows fp16 are zeros and reported."""
    import torch
    top = np.arange(0x7c00 if src == "f16" else 0x7f80, dtype=np.uint16)
    top = torch.from_numpy(np.resize(top, -(-top.size // 8) * 8).view(np.int16)).view(dtype(src)).float().numpy()
    f = np.random.default_rng(16).uniform(-1, 1, (top.size, 32)).astype(np.float32)
    f[np.arange(top.size), np.arange(top.size) % 32] = 1
    f[::2] = np.sign(f[::2]) * np.rint(np.abs(f[::2]) * 14) / 14             # (many near halves)
    x = torch.from_numpy(f * top[:, None]).to(dtype(src)).reshape(1, -1, 2, 128)
    n = x.shape[1]
    Tmax = -(-n // 128) * 128
    kv = make_kv(fmt, new_cache(fmt, 1, 2, Tmax, 128))
    st = status()
    bq.kv_append(kv, x.to(DEV), x.to(DEV), ints([0]), None, st)
    xf = x.float().numpy().copy()
    blocks = xf.reshape(-1, 32)
    over = np.abs(blocks).max(1) / np.float32(7 if fmt == 4 else 127) >= 65520
    blocks[over] = 0
    assert int(st.item()) == (1 << bq.BQ_ERR_RANGE if over.any() else 0)
    for got, w in zip(planes_of(kv), place(fmt, new_cache(fmt, 1, 2, Tmax, 128), xf, xf, [0], [n])):
        assert np.array_equal(got, w)


@pytest.mark.parametrize("src", ["f32", "f16"])
@pytest.mark.parametrize("fmt", [4, 8])
def test_two_streams_append_neighbouring_positions(fmt, src):
    """Two calls at once into one cache, whose ranges meet inside a value tile
    and inside a word of transposed value bytes, many times over."""
    import torch
    B, H, Tmax, D = 2, 4, 512, 128
    streams = [torch.cuda.Stream() for _ in range(2)]
    for cut in (37, 130, 255):
        kv = make_kv(fmt, new_cache(fmt, B, H, Tmax, D))
        k, v, kf, vf = rows(cut, B, 400, H, D, src)
        n = 400 - cut
        args = [(k[:, :cut], v[:, :cut], ints([3] * B)), (k[:, cut:], v[:, cut:], ints([3 + cut] * B))]
        torch.cuda.synchronize()
        for _ in range(20):
            for s, (kk, vv, start) in zip(streams, args):
                bq.kv_append(kv, kk, vv, start, stream=s)
        torch.cuda.synchronize()
        want = place(fmt, new_cache(fmt, B, H, Tmax, D), kf, vf, [3] * B, [cut + n] * B)
        for got, w in zip(planes_of(kv), want):
            assert np.array_equal(got, w)


def test_broadcast_rows_and_a_single_token_of_a_longer_tensor():
    """Stride 0 over tokens (one row written to every position), and a T = 1
    slice whose unused strides are odd."""
    planes = new_cache(4, 1, 2, 64, 128)
    kv = make_kv(4, planes)
    k, v, kf, vf = rows(10, 1, 1, 2, 128, "f32")
    bq.kv_append(kv, k.expand(1, 40, 2, 128), v.expand(1, 40, 2, 128), ints([20]))
    want = place(4, planes, kf.repeat(40, 1), vf.repeat(40, 1), [20], [40])
    for got, w in zip(planes_of(kv), want):
        assert np.array_equal(got, w)
    k, v, kf, vf = rows(11, 1, 9, 2, 128, "f16")
    bq.kv_append(kv, k[:, 4:5], v[:, 4:5], ints([0]))
    want = place(4, want, kf[:, 4:5], vf[:, 4:5], [0], [1])
    for got, w in zip(planes_of(kv), want):
        assert np.array_equal(got, w)


def test_cache_offsets_past_32_bits():
    import torch
    B, H, Tmax, D = 3, 1, 1 << 25, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of free device memory")
    refs = [torch.empty((B, H, Tmax, w), dtype=t, device=DEV)
            for w, t in ((64, torch.uint8), (4, torch.int16), (64, torch.uint8), (4, torch.int16))]
    kv = bq.kv_cache_q4(*refs)
    k, v, kf, vf = rows(12, B, 3, H, D, "f32")
    start = [0, 5, Tmax - 3]
    bq.kv_append(kv, k, v, ints(start))
    ko, vo = torch.zeros((B, 3, H, D), device=DEV), torch.zeros((B, 3, H, D), device=DEV)
    bq.kv_read(kv, ko, vo, ints(start))
    for x, y in ((kf, ko), (vf, vo)):
        c, s = quant_rows(4, x)
        assert np.array_equal(y.cpu().numpy(), deq_q4(c, s))


@pytest.mark.parametrize("D,G,Tq", [(128, 5, 1), (64, 4, 1), (128, 4, 3)])
def test_decode_loop_append_attend_read(D, G, Tq):
    """A batch's decode loop as a user runs it: prompts of unequal lengths
    appended at once, then steps of Tq tokens (append, then attention), the step
    captured into a graph on a side stream and replayed with new rows, starts
    and lengths; every step against fp64, and the cache read back at the end."""
    import torch
    B, H, Tmax, steps = 3, 2, 192, 6
    planes = new_cache(4, B, H, Tmax, D, fill=0)
    kv = make_kv(4, planes)
    prompt = [70, 1, 33]
    k, v, kf, vf = rows(20, B, max(prompt), H, D, "f16")
    bq.kv_append(kv, k, v, ints([0] * B), ints(prompt))
    want = place(4, planes, kf, vf, [0] * B, prompt)
    hist = np.array(prompt)
    q = torch.zeros((B, Tq, H * G, D), dtype=torch.float16, device=DEV)
    qkv = torch.zeros((B, Tq, 2 * H, D), device=DEV)
    start, lens = ints([0] * B), ints([0] * B)
    o = torch.zeros((B, Tq, H * G, D), dtype=torch.float32, device=DEV)
    ws = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(D, Tq, G), DEV)
    st = status()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        bq.kv_append(kv, qkv[:, :, :H], qkv[:, :, H:], start, None, st)
        bq.attn_decode_q4(kv, q, lens, G, D ** -0.5, o, ws, st)
    r = np.random.default_rng(21)
    for _ in range(steps):
        x = r.standard_normal((B, Tq, 2 * H, D)).astype(np.float32)
        qh = r.standard_normal((B, Tq, H * G, D)).astype(np.float16)
        qkv.copy_(torch.from_numpy(x))
        q.copy_(torch.from_numpy(qh))
        start.copy_(torch.from_numpy(hist.astype(np.int32)))
        lens.copy_(torch.from_numpy((hist + Tq).astype(np.int32)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = place(4, want, x[:, :, :H], x[:, :, H:], hist, [Tq] * B)
        hist = hist + Tq
        check_attention(o.cpu().numpy(), attention_ref(want, qh.view(np.uint16), hist, G, D ** -0.5), False)
    assert int(st.item()) == 0
    for got, w in zip(planes_of(kv), want):
        assert np.array_equal(got, w)
    ko = torch.zeros((B, Tmax, H, D), device=DEV)
    bq.kv_read(kv, ko, None, ints([0] * B), ints(hist))
    for b in range(B):
        ref = deq_q4(want[0][b, :, :hist[b]], want[1][b, :, :hist[b]]).transpose(1, 0, 2)
        assert np.array_equal(ko[b, :hist[b]].cpu().numpy(), ref) and not ko[b, hist[b]:].any().item()


def test_q8_append_feeds_the_q8_attention():
    """Tokens appended one at a time to the Q8 cache, then bq_attn_decode_q8 over it."""
    import torch
    B, H, G, D, Tmax, n = 2, 2, 4, 128, 256, 150
    planes = new_cache(8, B, H, Tmax, D)
    kv = make_kv(8, planes)
    k, v, kf, vf = rows(30, B, n, H, D, "f32")
    bq.kv_append(kv, k[:, :100], v[:, :100], ints([0, 0]))
    for t in range(100, n):
        bq.kv_append(kv, k[:, t:t + 1], v[:, t:t + 1], ints([t, t]))
    want = place(8, planes, kf, vf, [0, 0], [n, n])
    got = planes_of(kv)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)
    q = np.random.default_rng(31).standard_normal((B, H * G, D)).astype(np.float16).view(np.uint16)
    lens = np.array([n, 77], dtype=np.int32)
    o = torch.empty((B, H * G, D), device=DEV)
    ws = bq.workspace(bq.lib().bq_attn_workspace_bytes(B, H), DEV)
    bq.attn_decode_q8(kv, to_dev(q), to_dev(lens), G, 0.09, o, ws)
    o_ref, abso, _ = oracle.attn_decode_q8(want[0].view(np.int8), want[1], want[2].view(np.int8), want[3], q, lens, 0.09)
    assert np.all(np.abs(o.cpu().numpy() - o_ref) <= REL * abso + ABS)
