"""Helpers of the KV cache tests: caches built by the oracle's quantisers (no
code of the CUDA library), and decode attention over a Q4 cache in fp64 numpy."""
import numpy as np

import oracle
from quantised_weight_gemv_b200 import bq
from tests.gpu_helpers import DEV


def to_dev(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).to(DEV)


def quant_rows(fmt, x):
    """fp32 rows [..., D] -> (codes [..., D/2 or D], scales [..., D/32]), by the oracle."""
    D = x.shape[-1]
    c, s = (oracle.quantize_q4 if fmt == 4 else oracle.quantize_q8)(
        np.ascontiguousarray(x.reshape(-1, D), dtype=np.float32))
    return (c.reshape(*x.shape[:-1], -1),
            np.ascontiguousarray(s[:, :D // 32]).reshape(*x.shape[:-1], D // 32))


def deq_q4(codes, scales):
    """fp64 values [..., D] of Q4 rows (byte i of a block: element i low, i + 16 high)."""
    c = codes.reshape(*codes.shape[:-1], -1, 16).astype(np.int64)
    v = np.concatenate([c & 15, c >> 4], -1).astype(np.float64) - 8
    return (v * oracle.half_to_double(scales)[..., None]).reshape(*codes.shape[:-1], -1)


def random_cache_q4(seed, B, Hkv, Tmax, D, k_size=1.0, v_size=1.0):
    """Q4 planes (kc, ks, vc, vs) of normal keys and values."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((2, B, Hkv, Tmax, D)).astype(np.float32)
    return (*quant_rows(4, x[0] * np.float32(k_size)), *quant_rows(4, x[1] * np.float32(v_size)))


def attention_ref(planes, q_bits, lens, G, scale):
    """(o, sum_t p_t |V|, slack, floor) in fp64 for q_bits [B, Tq, Hkv*G, D].

    slack[b, i, j] bounds the relative error that fp32 scores bring into a
    softmax weight.  A score is sum over blocks of dK * (sum_d u q - 8 sum_d q)
    with codes u <= 15: its terms add up to at most S = scale * sum_d |q_d|
    23 dK, each accumulation step keeps them to 2^-23 of that, and a block takes
    three steps (four with the sum over blocks); exp doubles it (numerator and
    sum).  The exponent's argument adds 2^-23 of its own magnitude.

    floor[b, i, j] is absolute: a weight p_t dV enters the value product as
    2^(s_t - m) dV in fp16, whose spacing is 2^-24 below 2^-14, so each of n
    positions may be off by 2^-25 times a code of at most 8.  The reference m is
    at most max_t s_t + E - 11 with 2^E <= 1.07 max(dV, 2^-14), and the sum of
    2^(s_t) is at least 2^(max s_t): off by at most n 8 2^-25 2^(E - 11) <=
    n 2^-32 max(dV, 2^-14) in o.  It shows where the leading positions' codes
    are 0 and o consists of positions with weights below 2^-20."""
    kc, ks, vc, vs = planes
    q = q_bits.view(np.float16).astype(np.float64)
    B, Tq, H, D = q.shape
    o, ao, slack, floor = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    for b in range(B):
        n = min(max(int(lens[b]), 0), kc.shape[2])
        if n == 0:
            continue
        for h in range(H // G):
            K, V = deq_q4(kc[b, h, :n], ks[b, h, :n]), deq_q4(vc[b, h, :n], vs[b, h, :n])
            dk = np.abs(oracle.half_to_double(ks[b, h, :n]))
            for i in range(Tq):
                m = n - (Tq - 1 - i)
                if m <= 0:
                    continue
                for j in range(h * G, (h + 1) * G):
                    s = scale * (K[:m] @ q[b, i, j])
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o[b, i, j], ao[b, i, j] = p @ V[:m], p @ np.abs(V[:m])
                    floor[b, i, j] = m * 2.0 ** -32 * max(np.abs(oracle.half_to_double(vs[b, h, :m])).max(), 2.0 ** -14)
                    S = abs(scale) * 23 * (dk[:m] @ np.abs(q[b, i, j]).reshape(-1, 32).sum(-1)).max()
                    slack[b, i, j] = 2 * 4 * 2.0 ** -23 * S + 2.0 ** -22 * 1.4427 * np.abs(s).max()
    return o, ao, slack, floor


def check_attention(o, ref, f16):
    """|o - o_ref| <= A (r + slack + 2^-16) + floor + |o_ref| 2^-11 + 2^-24, A = sum p |V|:
    r = 2^-11 is a softmax weight's one rounding to fp16 when the output is
    fp16 (two fp16 terms otherwise: below 2^-20), 2^-16 = 128 fp32 roundings of
    sums of signed terms, and the last two are the fp16 output's rounding."""
    o_ref, ao, slack, floor = ref
    o = np.asarray(o, dtype=np.float64)
    assert o.shape == o_ref.shape and np.all(np.isfinite(o))
    bound = ao * ((2.0 ** -11 if f16 else 2.0 ** -20) + 2.0 ** -16 + slack[..., None]) + floor[..., None]
    bound += (2.0 ** -11 * np.abs(o_ref) + 2.0 ** -24) if f16 else 2.0 ** -126
    bad = np.argwhere(np.abs(o - o_ref) > bound)
    assert bad.size == 0, (len(bad), bad[:4].tolist(), float(np.max(np.abs(o - o_ref) / bound)))


def run_attention(planes, q_bits, lens, G, scale, f16=True, ws=None, stream=None):
    import torch
    B, Tq, H, D = q_bits.shape
    kv = bq.kv_cache_q4(*[to_dev(p) for p in planes])
    o = torch.full(q_bits.shape, float("nan"), dtype=torch.float16 if f16 else torch.float32, device=DEV)
    if ws is None:
        ws = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(D, Tq, G), DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    bq.attn_decode_q4(kv, to_dev(q_bits), to_dev(np.asarray(lens, dtype=np.int32)), G, scale, o, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert int(ws.count_nonzero().item()) == 0       # counters and partials are cleared
    return o.float().cpu().numpy()
