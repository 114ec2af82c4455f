"""Operators of the quantised KV cache: what is measured, and their plain forms.

Three operators around the cache that decode attention reads:

  append     new keys and values are quantised as they are written to the cache
             (32-element blocks along the head dimension, one fp16 scale a block);
             Q4 cache (4-bit codes) or Q8 cache (8-bit codes, values transposed)
  read       a range of cached positions read back as fp32, fp16 or bf16
  attention  decode attention over the Q4 cache, for one query token a sequence
             or several (the drafted tokens of a verification step)

With `own` false, run() computes them with elementary torch operations; with
`own` true it makes the library's calls.  An append case appends, then reads
the appended positions back: what the cache holds in 4 or 8 bits is returned
as the values it stands for.
"""
import math
import random

import torch

own = False
DEV = "cuda"
_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one sequence of a hidden-5120 decoder (8 KV heads, 5 query heads each) at a short
        # context: a single launch of a few microseconds, where latency is all
        dict(name="attn_b1_t4096", op="attn", B=1, Hkv=8, G=5, D=128, Tq=1, Tmax=4096, mix=0, out="f16"),
        # the same layer at its full context
        dict(name="attn_b1_t32768", op="attn", B=1, Hkv=8, G=5, D=128, Tq=1, Tmax=32768, mix=0, out="f16"),
        # a batch of such sequences, all full: the steady stream of the largest decode step
        dict(name="attn_b8_t32768", op="attn", B=8, Hkv=8, G=5, D=128, Tq=1, Tmax=32768, mix=0, out="f16"),
        # a hidden-2048 decoder's batch under continuous batching: every length from 0 up, one slot
        # idle; fp32 output for a caller that reduces further
        dict(name="attn_b8_mixed", op="attn", B=8, Hkv=4, G=4, D=128, Tq=1, Tmax=8192, mix=1, out="f32"),
        # speculative decoding: 8 drafted tokens a sequence verified at once, each seeing its own prefix
        dict(name="attn_verify_b8_q8", op="attn", B=8, Hkv=8, G=5, D=128, Tq=8, Tmax=8192, mix=2, out="f16"),
        # many short chats on a model with 64-wide heads
        dict(name="attn_b64_d64", op="attn", B=64, Hkv=8, G=4, D=64, Tq=1, Tmax=1024, mix=3, out="f16"),
        # a decode step's new token a sequence, straight from the fp32 q|k|v projection's output
        dict(name="append_q4_step", op="append", fmt=4, B=8, Hkv=8, G=5, D=128, T=1, Tmax=4096, mix=4, src="f32", out="f16"),
        dict(name="append_q8_step", op="append", fmt=8, B=8, Hkv=8, G=5, D=128, T=1, Tmax=4096, mix=5, src="f32", out="f16"),
        # a long prompt written in one go, an odd number of tokens at an odd position
        dict(name="append_q4_prompt", op="append", fmt=4, B=1, Hkv=8, G=5, D=128, T=16381, Tmax=32768, mix=6, src="bf16", out="bf16"),
        # ragged prompts of a batch into the Q8 cache
        dict(name="append_q8_prompts", op="append", fmt=8, B=8, Hkv=4, G=4, D=128, T=2047, Tmax=8192, mix=7, src="f16", out="f16"),
        # a full context read back for a consumer that wants 16-bit keys and values
        dict(name="read_q4_t32768", op="read", fmt=4, B=1, Hkv=8, D=128, T=32768, Tmax=32768, mix=0, out="f16"),
        # ragged prefixes of a batch of the Q8 cache, in fp32 (export, comparison)
        dict(name="read_q8_prefixes", op="read", fmt=8, B=8, Hkv=4, D=128, T=4095, Tmax=8192, mix=8, out="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "read"])
    if op == "attn":
        D, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 5, 8])
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
        Tq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        most = 8 * 8 * 32768 * 128                     # elements of K of the largest listed case
        Tmax = 32 * _spread(rng, 1, min(1024, 5 * most // (32 * Hkv * D * Tq * G)))
        B = _spread(rng, 1, max(1, min(128, most // (Hkv * Tmax * D), 5 * most // (Hkv * Tmax * D * Tq * G))))
        return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, Tq=Tq, Tmax=Tmax, mix=rng.randrange(1 << 20),
                    out=rng.choice(["f16", "f16", "f32"]))
    fmt = rng.choice([4, 8])
    D = 128 if fmt == 8 else rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    T = rng.choice([1, _spread(rng, 1, 16384)])
    B = _spread(rng, 1, max(1, min(64, 16384 * 8 // (T * Hkv))))
    unit = 128 if fmt == 8 else 32
    Tmax = unit * (-(-T // unit) + _spread(rng, 1, 16))
    case = dict(op=op, fmt=fmt, B=B, Hkv=Hkv, D=D, T=T, Tmax=Tmax, mix=rng.randrange(1 << 20),
                out=rng.choice(["f32", "f16", "bf16"]))
    if op == "append":
        case.update(G=rng.choice([1, 4, 5]), src=rng.choice(["f32", "f16", "bf16"]))
    return case


def _lengths(case):
    """Valid positions a sequence (attention): mix 0 fills every cache, otherwise
    uniform in 1 .. Tmax, and the second of three or more sequences is idle (0)."""
    if not case["mix"]:
        return [case["Tmax"]] * case["B"]
    rng = random.Random(case["mix"])
    lens = [rng.randint(1, case["Tmax"]) for _ in range(case["B"])]
    if case["B"] > 2:
        lens[1] = 0
    return lens


def _ranges(case):
    """First position and number of rows a sequence (append, read): mix 0 starts
    at 0 with all T rows; otherwise odd places, and 1 .. T rows where T > 1."""
    B, T, room = case["B"], case["T"], case["Tmax"] - case["T"]
    if not case["mix"]:
        return [0] * B, [T] * B
    rng = random.Random(case["mix"])
    starts = [rng.randint(0, room) for _ in range(B)]
    counts = [T if B == 1 else rng.randint(max(1, T // 4), T) for _ in range(B)]
    return starts, counts


def _cache_shape(case, fmt):
    B, H, S, D = case["B"], case["Hkv"], case["Tmax"], case["D"]
    return B, H, S, D, D // 32


def _rows(gen, shape, spread):
    """Keys or values as projections give them: normal, with channels of unequal size."""
    size = torch.exp(spread * torch.randn(shape[-1], generator=gen, device=DEV))
    return torch.randn(shape, generator=gen, device=DEV) * size


def _filled(gen, case, fmt):
    """A cache of seeded keys and values: (k_codes, k_scales, v_codes, v_scales)."""
    B, H, S, D, nb = _cache_shape(case, fmt)
    planes = []
    for spread in (0.5, 0.2):
        x = _rows(gen, (B, H, S, D), spread).view(B, H, S, nb, 32)
        level = 7.0 if fmt == 4 else 127.0
        d = (x.abs().amax(-1) / level).half()
        c = torch.round(x / d.float().unsqueeze(-1)).clamp_(-level, level)
        del x
        if fmt == 4:
            c = (c + 8).to(torch.uint8)
            c = (c[..., :16] | (c[..., 16:] << 4)).reshape(B, H, S, D // 2)
        else:
            c = c.to(torch.int8).reshape(B, H, S, D)
            if planes:
                c = c.transpose(2, 3)
        planes += [c.contiguous(), d.contiguous()]
    return planes


def _empty(case, fmt):
    B, H, S, D, nb = _cache_shape(case, fmt)
    z = lambda *s, t: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    sc = [z(B, H, S, nb, t=torch.float16) for _ in range(2)]
    if fmt == 4:
        return [z(B, H, S, D // 2, t=torch.uint8), sc[0], z(B, H, S, D // 2, t=torch.uint8), sc[1]]
    return [z(B, H, S, D, t=torch.int8), sc[0], z(B, H, D, S, t=torch.int8), sc[1]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 2 + 1)
    op, B, H, D = case["op"], case["B"], case["Hkv"], case["D"]
    fmt = case.get("fmt", 4)
    st = {"case": case}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if op == "attn":
        st["planes"] = _filled(gen, case, 4)
        st["q"] = torch.randn((B, case["Tq"], H * case["G"], D), generator=gen, device=DEV).half()
        st["lens"] = ints(_lengths(case))
        st["o"] = torch.zeros((B, case["Tq"], H * case["G"], D), dtype=_DT[case["out"]], device=DEV)
    else:
        T = case["T"]
        st["planes"] = _filled(gen, case, fmt) if op == "read" else _empty(case, fmt)
        start, count = _ranges(case)
        st["start"], st["count"] = ints(start), ints(count)
        if op == "append":
            # k and v are column ranges of one projection output [B, T, (Hq + 2 Hkv) D]
            Hq = H * case["G"]
            qkv = torch.empty((B, T, Hq + 2 * H, D), dtype=_DT[case["src"]], device=DEV)
            qkv[:, :, Hq:Hq + H] = _rows(gen, (B, T, H, D), 0.5)
            qkv[:, :, Hq + H:] = _rows(gen, (B, T, H, D), 0.2)
            st["k"], st["v"] = qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
        st["ko"] = torch.zeros((B, T, H, D), dtype=_DT[case["out"]], device=DEV)
        st["vo"] = torch.zeros_like(st["ko"])
    if own:
        from quantised_weight_gemv_b200 import bq
        st["bq"] = bq
        st["kv"] = (bq.kv_cache_q4 if fmt == 4 else bq.kv_cache)(*st["planes"])
        st["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op == "attn":
            st["ws"] = bq.workspace(bq.lib().bq_attn_q4_workspace_bytes(D, case["Tq"], case["G"]), DEV)
    return st


def run(st):
    case = st["case"]
    if own:
        bq = st["bq"]
        if case["op"] == "attn":
            bq.attn_decode_q4(st["kv"], st["q"], st["lens"], case["G"], case["D"] ** -0.5, st["o"], st["ws"], st["status"])
            return st["o"]
        if case["op"] == "append":
            bq.kv_append(st["kv"], st["k"], st["v"], st["start"], st["count"], st["status"])
        bq.kv_read(st["kv"], st["ko"], st["vo"], st["start"], st["count"], st["status"])
        return st["ko"], st["vo"]
    if case["op"] == "attn":
        return _plain_attention(st)
    if case["op"] == "append":
        _plain_append(st)
    return _plain_read(st)


# ------------------------------------------------------------- plain forms ----
def _values(codes, scales):
    """Q4 rows [..., D/2] and scales [..., D/32] as fp32 values [..., D]."""
    c = codes.unflatten(-1, (-1, 16))
    c = torch.cat([c & 15, c >> 4], -1).float() - 8
    return (c * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_attention(st):
    case = st["case"]
    B, H, G, Tq, S, D = (case[n] for n in ("B", "Hkv", "G", "Tq", "Tmax", "D"))
    kc, ks, vc, vs = st["planes"]
    q = st["q"].float().view(B, Tq, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Tq * G, D)
    s = torch.matmul(q, _values(kc, ks).transpose(2, 3)) * D ** -0.5
    last = st["lens"].view(B, 1) - (Tq - 1 - torch.arange(Tq, device=DEV))              # [B, Tq]
    dead = torch.arange(S, device=DEV) >= last.repeat_interleave(G, 1).unsqueeze(-1)      # [B, Tq G, S]
    s = s.masked_fill(dead.unsqueeze(1), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    n = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _values(vc, vs)) / torch.where(n == 0, torch.ones_like(n), n)
    return o.view(B, H, Tq, G, D).permute(0, 2, 1, 3, 4).reshape(B, Tq, H * G, D).to(_DT[case["out"]])


def _places(st):
    """Position [B, T] of every row, and whether it is one of the sequence's count."""
    t = torch.arange(st["case"]["T"], device=DEV)
    return st["start"].long().unsqueeze(1) + t, t < st["count"].unsqueeze(1)


def _plain_append(st):
    case = st["case"]
    fmt, B, T, H, D = (case[n] for n in ("fmt", "B", "T", "Hkv", "D"))
    pos, live = _places(st)
    b = torch.arange(B, device=DEV).unsqueeze(1)
    level = 7.0 if fmt == 4 else 127.0
    for plane, (x, codes, scales) in enumerate(((st["k"], *st["planes"][:2]), (st["v"], *st["planes"][2:]))):
        # in 64 bits: a quotient next to a half must round as its fp32 value does
        x = x.double().reshape(B, T, H, D // 32, 32)
        d = (x.abs().amax(-1) / level).float().half()
        r = (x / torch.where(d == 0, torch.ones_like(d), d).double().unsqueeze(-1)).float().double()
        r = torch.where((d == 0).unsqueeze(-1), torch.zeros_like(r), torch.sign(r) * torch.floor(r.abs() + 0.5))
        if fmt == 4:
            c = (r + 8).clamp_(0, 15).to(torch.uint8)
            c = (c[..., :16] | (c[..., 16:] << 4)).reshape(B, T, H, D // 2)
        else:
            c = r.clamp_(-127, 127).to(torch.int8).reshape(B, T, H, D)
        rows = codes.transpose(1, 2) if fmt == 4 or plane == 0 else codes.permute(0, 3, 1, 2)  # [B, S, H, row]
        rows[b, pos] = torch.where(live[..., None, None], c, rows[b, pos])
        scs = scales.transpose(1, 2)
        scs[b, pos] = torch.where(live[..., None, None], d, scs[b, pos])


def _plain_read(st):
    case = st["case"]
    pos, live = _places(st)
    b = torch.arange(case["B"], device=DEV).unsqueeze(1)
    for plane, out in enumerate((st["ko"], st["vo"])):
        codes, scales = st["planes"][2 * plane:2 * plane + 2]
        d = scales.transpose(1, 2)[b, pos]
        if case["fmt"] == 4:
            x = _values(codes.transpose(1, 2)[b, pos], d)
        else:
            c = (codes.transpose(1, 2) if plane == 0 else codes.permute(0, 3, 1, 2))[b, pos]
            x = (c.float().unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).flatten(-2)
        out.copy_(torch.where(live[..., None, None], x.to(out.dtype), out))
    return st["ko"], st["vo"]


# ---------------------------------------------------------------- the work ----
def work(case):
    H, D = case["Hkv"], case["D"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if case["op"] == "attn":
        rows = case["Tq"] * case["G"] * H * D
        pos = sum(_lengths(case)) * H                  # (position, KV head) pairs
        return {"bytes": pos * 2 * (D // 2 + D // 16) + case["B"] * (rows * (2 + size[case["out"]]) + 4),
                "flops": pos * 4 * D * case["Tq"] * case["G"]}
    n = 2 * sum(_ranges(case)[1]) * H * D              # elements of K and V
    held = n // 2 + n // 16 if case["fmt"] == 4 else n + n // 16
    if case["op"] == "append":
        return {"bytes": n * (size[case["src"]] + size[case["out"]]) + held, "flops": 5 * n}
    return {"bytes": n * size[case["out"]] + held, "flops": 2 * n}


# ------------------------------------------------------ from the definition ----
def exact(case, seed):
    """The operators from their definition in 64 bits, one sequence and KV head after another."""
    st = prepare(case, seed)
    B, H, D, nb = case["B"], case["Hkv"], case["D"], case["D"] // 32
    if case["op"] == "attn":
        kc, ks, vc, vs = st["planes"]
        Tq, G = case["Tq"], case["G"]
        o = torch.zeros((B, Tq, H * G, D), dtype=torch.float64, device=DEV)

        def dense(codes, scales, n):                   # element i of a block: low nibble i, high nibble i - 16
            w = torch.empty((n, nb, 32), dtype=torch.float64, device=DEV)
            w[:, :, :16] = (codes[:n].view(n, nb, 16) % 16).double()
            w[:, :, 16:] = (codes[:n].view(n, nb, 16) // 16).double()
            return ((w - 8.0) * scales[:n].double()[:, :, None]).view(n, D)

        for b, n in enumerate(_lengths(case)):
            for h in range(H):
                if n == 0:
                    continue
                K, V = dense(kc[b, h], ks[b, h], n), dense(vc[b, h], vs[b, h], n)
                for i in range(Tq):
                    seen = n - (Tq - 1 - i)
                    if seen > 0:
                        logit = st["q"][b, i, h * G:(h + 1) * G].double() @ K[:seen].T / math.sqrt(D)
                        o[b, i, h * G:(h + 1) * G] = torch.softmax(logit, -1) @ V[:seen]
        return o
    start, count = _ranges(case)
    fmt, T, outs = case["fmt"], case["T"], []
    for plane in range(2):
        out = torch.zeros((B, T, H, D), dtype=torch.float64, device=DEV)
        codes, scales = st["planes"][2 * plane:2 * plane + 2]
        for b in range(B):
            if case["op"] == "append":
                x = (st["k"], st["v"])[plane][b, :count[b]].double().reshape(count[b], H, nb, 32)
                top = 7 if fmt == 4 else 127
                d = (x.abs().max(-1, keepdim=True).values / top).to(torch.float32).to(torch.float16).double()
                t = (x / d).to(torch.float32).double()
                t = torch.nan_to_num(torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t)))
                val = torch.clamp(t, -8 if fmt == 4 else -127, top) * d
            else:
                lo, hi = start[b], start[b] + count[b]
                d = scales[b, :, lo:hi].double().transpose(0, 1).unsqueeze(-1)
                if fmt == 4:
                    by = codes[b, :, lo:hi].transpose(0, 1).reshape(count[b], H, nb, 16)
                    val = torch.cat([by % 16, by // 16], -1).double().sub(8.0) * d
                else:
                    by = codes[b, :, lo:hi] if plane == 0 else codes[b, :, :, lo:hi].transpose(1, 2)
                    val = by.transpose(0, 1).reshape(count[b], H, nb, 32).double() * d
            out[b, :count[b]] = val.reshape(count[b], H, D)
        outs.append(out)
    return tuple(outs)
