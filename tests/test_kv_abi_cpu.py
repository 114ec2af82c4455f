"""The KV cache entry points without a GPU: bq_kv.h is exported and bound with
its own types, and every argument the host can check is refused before any
device call (fake pointers are never dereferenced), by the C ABI and by the
Python binding."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from quantised_weight_gemv_b200 import bq
from tests.conftest import ROOT
from tests.test_abi_cpu import _ctype_of
from tests.test_binding_cpu import _Dev

FAKE = 0x7f0000000000


def test_header_functions_are_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "bq_kv.h")).read()
    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    found = re.findall(r"BQ_API\s+([^;(]*?)\b(bq_\w+)\s*\(([^)]*)\)\s*;", src)
    assert {name for _, name, _ in found} == set(bq._KV_SIGS)
    for ret, name, params in found:
        norm = lambda t: " ".join(re.sub(r"\s*\*", " *", re.sub(r"\bconst\b", " ", t)).split())  # noqa: E731
        want = [_ctype_of(norm(re.match(r"^(.*?)(\w+)$", norm(p)).group(1))) for p in params.split(",")]
        assert bq._KV_SIGS[name] == (_ctype_of(norm(ret)), want), name
        assert hasattr(bq.lib(), name)
    assert bq.bq_status_string(bq.BQ_ERR_POSITION) == "cache position or row count out of range"


def test_structs_match_the_header_layout(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "bq_kv.h"', "int main(void) {"]
    want = []
    for s in (bq.bq_kv_cache_q4, bq.bq_kv_rows):
        n = s.__name__
        lines.append(f'printf("%zu\\n", sizeof({n}));')
        want.append(ctypes.sizeof(s))
        for f, _ in s._fields_:
            lines.append(f'printf("%zu\\n", offsetof({n}, {f}));')
            want.append(getattr(s, f).offset)
    c = tmp_path / "layout.c"
    c.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    assert [int(x) for x in out.split()] == want


def rows_rc(fn, kv=None, k=FAKE, v=FAKE, strides=(0, 1024, 128) * 2, dtype=0, T=4, B=2, Hkv=8, start=FAKE, count=FAKE):
    q8 = fn.endswith("q8")
    if kv is None:
        kv = (bq.bq_kv_cache if q8 else bq.bq_kv_cache_q4)(FAKE, FAKE, FAKE, FAKE, 128, 256)
    rows = bq.bq_kv_rows(k, v, *strides, dtype, T)
    return getattr(bq.lib(), fn)(ctypes.byref(kv) if kv else None, ctypes.byref(rows), B, Hkv, start, count, None, None)


@pytest.mark.parametrize("fn", ["bq_kv_append_q4", "bq_kv_append_q8", "bq_kv_read_q4", "bq_kv_read_q8"])
def test_rows_argument_validation_before_launch(fn):
    cache = bq.bq_kv_cache if fn.endswith("q8") else bq.bq_kv_cache_q4
    make = lambda D=128, T=256, p=FAKE: cache(FAKE, p, FAKE, FAKE, D, T)  # noqa: E731
    assert rows_rc(fn, kv=False) == bq.BQ_ERR_NULL
    assert rows_rc(fn, kv=make(p=None)) == bq.BQ_ERR_NULL
    assert rows_rc(fn, k=None, v=None) == bq.BQ_ERR_NULL
    if "append" in fn:
        assert rows_rc(fn, k=None) == bq.BQ_ERR_NULL and rows_rc(fn, v=None) == bq.BQ_ERR_NULL
    assert rows_rc(fn, start=None) == bq.BQ_ERR_NULL
    assert getattr(bq.lib(), fn)(ctypes.byref(make()), None, 1, 1, FAKE, None, None, None) == bq.BQ_ERR_NULL
    for D in (32, 96, 256):
        assert rows_rc(fn, kv=make(D=D)) == bq.BQ_ERR_SHAPE
    assert rows_rc(fn, kv=make(T=0)) == rows_rc(fn, kv=make(T=250)) == rows_rc(fn, kv=make(T=-128)) == bq.BQ_ERR_SHAPE
    assert rows_rc(fn, T=0) == rows_rc(fn, T=257) == rows_rc(fn, Hkv=0) == bq.BQ_ERR_SHAPE
    assert rows_rc(fn, Hkv=65536, kv=make(T=128)) == bq.BQ_ERR_SHAPE
    assert rows_rc(fn, dtype=3) == rows_rc(fn, dtype=-1) == bq.BQ_ERR_SHAPE
    assert rows_rc(fn, kv=make(T=1 << 28), B=8, Hkv=1) == bq.BQ_ERR_SHAPE           # 2^31 positions
    assert rows_rc(fn, B=0) == bq.BQ_ERR_BATCH
    assert rows_rc(fn, k=FAKE + 4) == rows_rc(fn, v=FAKE + 8) == bq.BQ_ERR_ALIGN
    for i in range(6):
        s = [1024] * 6
        s[i] += 2
        assert rows_rc(fn, strides=s) == bq.BQ_ERR_ALIGN
        s[i] += 2                                                                   # 4 elements: 16 bytes in fp32 only
        assert rows_rc(fn, strides=s, dtype=1) == bq.BQ_ERR_ALIGN
    assert rows_rc(fn, kv=make(p=FAKE + 2)) == bq.BQ_ERR_ALIGN
    assert rows_rc(fn, start=FAKE + 2) == rows_rc(fn, count=FAKE + 1) == bq.BQ_ERR_ALIGN


def attn_rc(kv=None, q=FAKE, lens=FAKE, B=2, Tq=1, Hkv=4, G=5, scale=0.088, o=FAKE, od=0, ws=FAKE, nws=1 << 30):
    kv = kv if kv is not None else bq.bq_kv_cache_q4(FAKE, FAKE, FAKE, FAKE, 128, 1024)
    return bq.lib().bq_attn_decode_q4(ctypes.byref(kv) if kv else None, q, lens, B, Tq, Hkv, G, scale, o, od, ws, nws,
                                      None, None)


def test_attention_argument_validation_before_launch():
    make = lambda D=128, T=1024, p=FAKE: bq.bq_kv_cache_q4(FAKE, FAKE, p, FAKE, D, T)  # noqa: E731
    assert attn_rc(kv=False) == attn_rc(kv=make(p=None)) == bq.BQ_ERR_NULL
    for name in ("q", "lens", "o", "ws"):
        assert attn_rc(**{name: None}) == bq.BQ_ERR_NULL
    assert attn_rc(kv=make(D=96)) == attn_rc(kv=make(T=1000)) == attn_rc(kv=make(T=0)) == bq.BQ_ERR_SHAPE
    assert attn_rc(G=0) == attn_rc(G=17) == attn_rc(Tq=0) == attn_rc(Tq=33) == attn_rc(Hkv=0) == bq.BQ_ERR_SHAPE
    assert attn_rc(od=2) == attn_rc(od=-1) == bq.BQ_ERR_SHAPE
    for s in (float("nan"), float("inf"), float("-inf")):
        assert attn_rc(scale=s) == bq.BQ_ERR_SHAPE
    assert attn_rc(kv=make(T=1 << 28), B=2, Hkv=4) == bq.BQ_ERR_SHAPE
    assert attn_rc(B=0) == bq.BQ_ERR_BATCH
    assert attn_rc(kv=make(p=FAKE + 8)) == bq.BQ_ERR_ALIGN
    assert attn_rc(q=FAKE + 2) == attn_rc(o=FAKE + 4) == attn_rc(ws=FAKE + 8) == attn_rc(lens=FAKE + 2) == bq.BQ_ERR_ALIGN
    f = bq.lib().bq_attn_q4_workspace_bytes
    assert f(96, 1, 1) == f(128, 0, 1) == f(128, 33, 1) == f(64, 1, 0) == f(64, 1, 17) == 0
    assert attn_rc(nws=f(128, 1, 5) - 1) == bq.BQ_ERR_WORKSPACE


def dev(*shape, dtype=torch.float32):
    return _Dev(torch.zeros(shape, dtype=dtype))


def cache_q4(B=2, H=4, T=64, D=128):
    return (dev(B, H, T, D // 2, dtype=torch.uint8), dev(B, H, T, D // 32, dtype=torch.int16),
            dev(B, H, T, D // 2, dtype=torch.uint8), dev(B, H, T, D // 32, dtype=torch.int16))


def test_binding_refuses_wrong_caches():
    kc, ks, vc, vs = cache_q4()
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        bq.kv_cache_q4(torch.zeros((2, 4, 64, 64), dtype=torch.uint8), ks, vc, vs)
    for bad in ((kc, ks, dev(2, 4, 64, 32, dtype=torch.uint8), vs), (kc, vs, vc, dev(2, 4, 64, 8, dtype=torch.int16)),
                (dev(2, 4, 64, 64), ks, vc, vs), (kc, dev(2, 4, 64, 4), vc, vs),
                (_Dev(torch.zeros((2, 4, 64, 128), dtype=torch.uint8)[..., ::2]), ks, vc, vs),
                cache_q4(D=96)):
        with pytest.raises(ValueError, match="do not match the cache layout"):
            bq.kv_cache_q4(*bad)
    other = dev(2, 4, 64, 64, dtype=torch.uint8)
    other.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="on one device"):
        bq.kv_cache_q4(kc, ks, other, vs)


@pytest.mark.parametrize("call", [bq.kv_append, bq.kv_read])
def test_binding_refuses_wrong_rows(call):
    kv = bq.kv_cache_q4(*cache_q4())
    ok, start = dev(2, 3, 4, 128), dev(2, dtype=torch.int32)
    host = torch.zeros((2, 3, 4, 128))
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        call(kv, host, ok, start)
    with pytest.raises(ValueError, match="must be given"):
        call(kv, None, None, start)
    for bad in (dev(2, 3, 4, 64), dev(3, 3, 4, 128), dev(2, 4, 128), dev(2, 2, 4, 128),
                _Dev(torch.zeros((2, 3, 4, 256))[..., ::2]), _Dev(torch.zeros((2, 3, 128, 4)).transpose(2, 3))):
        with pytest.raises(ValueError, match="v must be"):
            call(kv, ok, bad, start)
    with pytest.raises(ValueError, match="one dtype"):
        call(kv, ok, dev(2, 3, 4, 128, dtype=torch.float16), start)
    with pytest.raises(ValueError, match="not float32, float16 or bfloat16"):
        call(kv, dev(2, 3, 4, 128, dtype=torch.float64), dev(2, 3, 4, 128, dtype=torch.float64), start)
    with pytest.raises(ValueError, match="start must be int32"):
        call(kv, ok, ok, dev(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="start must be given"):
        call(kv, ok, ok, None)
    with pytest.raises(ValueError, match="count must be int32"):
        call(kv, ok, ok, start, dev(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="kv must come from"):
        call(object(), ok, ok, start)
    if call is bq.kv_read:
        with pytest.raises(ValueError, match="rows overlap"):
            call(kv, _Dev(torch.zeros((2, 1, 4, 128)).expand(2, 3, 4, 128)), ok, start)
    else:
        with pytest.raises(ValueError, match="k and v must be given"):
            call(kv, ok, None, start)


def test_binding_refuses_wrong_attention_arguments():
    kv = bq.kv_cache_q4(*cache_q4())
    q, lens, o = dev(2, 20, 128, dtype=torch.float16), dev(2, dtype=torch.int32), dev(2, 20, 128)
    ws = dev(1 << 20, dtype=torch.uint8)
    f = bq.attn_decode_q4
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        f(kv, torch.zeros((2, 20, 128), dtype=torch.float16), lens, 5, 0.1, o, ws)
    for bad in (dev(2, 24, 128, dtype=torch.float16), dev(2, 20, 128), dev(2, 20, 128, dtype=torch.bfloat16),
                dev(2, 2, 16, 128, dtype=torch.float16)):
        with pytest.raises(ValueError, match="q must be contiguous fp16"):
            f(kv, bad, lens, 5, 0.1, o, ws)
    with pytest.raises(ValueError, match="lens must be int32"):
        f(kv, q, dev(2, dtype=torch.int64), 5, 0.1, o, ws)
    for bad in (dev(2, 20, 64), dev(2, 20, 128, dtype=torch.bfloat16), dev(2, 1, 20, 128)):
        with pytest.raises(ValueError, match="o must be contiguous"):
            f(kv, q, lens, 5, 0.1, bad, ws)
    with pytest.raises(ValueError, match="kv must come from kv_cache_q4"):
        f(object(), q, lens, 5, 0.1, o, ws)
    for bad in ((None, lens, o, ws), (q, None, o, ws), (q, lens, None, ws), (q, lens, o, None)):
        with pytest.raises(ValueError, match="must be given"):
            f(kv, bad[0], bad[1], 5, 0.1, bad[2], bad[3])


def test_overlap_rule():
    ov = bq._overlaps
    assert not ov((2, 3, 4), (12, 4, 1)) and not ov((1, 3, 4), (0, 4, 1)) and not ov((3, 2, 4), (4, 12, 1))
    assert ov((2, 3, 4), (0, 4, 1)) and ov((2, 4), (3, 1)) and not ov((2, 4), (4, 1))


@pytest.mark.parametrize("fn", ["bq_kv_read_q4", "bq_kv_read_q8"])
def test_a_read_into_one_buffer_is_refused(fn):
    """k and v at one address, where keys and values would overwrite each other."""
    for dtype in (0, 1, 2):
        assert rows_rc(fn, dtype=dtype) == bq.BQ_ERR_SHAPE


def test_an_attention_output_over_its_queries_is_refused():
    assert attn_rc(od=1) == attn_rc(od=0) == bq.BQ_ERR_SHAPE
