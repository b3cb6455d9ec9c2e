"""The attention operators' C ABI and host logic without a GPU: the exports are
what include/qoq_attn.h declares, bad arguments are refused before any device
is touched, the scaled frequencies follow their formulas, and the plain
implementation the GPU tests compare with holds against hand-worked values."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import attn_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qoq_attn.h")
INVALID = -1


@pytest.fixture(scope="module")
def L():
    from w4a8_integer_gemm_b200 import build_lib
    build_lib.build()
    import w4a8_integer_gemm_b200 as q
    return q.lib()


def test_exports(L):
    import w4a8_integer_gemm_b200 as q
    names = set(re.findall(r"QOQ_API\s+[\w\s\*]+?\b(qattn_\w+)\s*\(", open(HEADER).read()))
    assert names == set(q.ATTN_SIGNATURES)
    out = os.popen(f"nm -D --defined-only {q.LIB_PATH}").read().split("\n")
    assert {l.split()[-1] for l in out if l.strip() and l.split()[-1].startswith("qattn_")} == names


A = ctypes.c_void_p(0x10000)     # aligned, never dereferenced: the checks come first
ODD = ctypes.c_void_p(0x10002)
NAN = float("nan")

CALLS = {
    "qattn_rotary": [("x", A), ("ldx", 512), ("pos", A), ("freq", A), ("T", 4), ("H", 4), ("d", 128), ("rot", 64),
                     ("inter", 0), ("amp", 1.0), ("y", A), ("ldy", 512), ("stream", None)],
    "qattn_cache_append": [("k", A), ("ldk", 256), ("v", A), ("ldv", 256), ("q", A), ("ldq", 1024), ("qo", A),
                           ("ldqo", 1024), ("T", 4), ("Hq", 8), ("Hkv", 2), ("d", 128), ("freq", A), ("rot", 128),
                           ("inter", 0), ("amp", 1.0), ("bits", 4), ("page", 64), ("pages", 9), ("kc", A), ("vc", A),
                           ("kp", A), ("vp", A), ("table", A), ("tp", 3), ("cu", A), ("len", A), ("B", 2),
                           ("stream", None)],
    "qattn_cache_read": [("kc", A), ("vc", A), ("kp", A), ("vp", A), ("bits", 4), ("page", 64), ("pages", 9),
                         ("Hkv", 2), ("d", 128), ("table", A), ("tp", 3), ("cu", A), ("len", A), ("B", 2), ("T", 4),
                         ("K", A), ("V", A), ("stream", None)],
    "qattn_paged_attention": [("q", A), ("ldq", 1024), ("T", 4), ("Hq", 8), ("Hkv", 2), ("d", 128), ("kc", A), ("vc", A),
                              ("kp", A), ("vp", A), ("bits", 4), ("page", 64), ("pages", 9), ("table", A), ("tp", 3),
                              ("cu", A), ("len", A), ("B", 2), ("max_new", 4), ("scale", 0.1), ("out", A),
                              ("ldo", 1024), ("ws", A), ("wsb", 1 << 40), ("stream", None)],
    "qattn_prompt_attention": [("q", A), ("ldq", 1024), ("k", A), ("ldk", 256), ("v", A), ("ldv", 256), ("T", 4), ("Hq", 8),
                               ("Hkv", 2), ("d", 128), ("cu", A), ("B", 2), ("scale", 0.1), ("out", A), ("ldo", 1024),
                               ("stream", None)],
}
# values every argument of that name has to refuse
BAD = {"d": [0, 96, 256, -64], "bits": [0, 2, 16], "page": [0, 8, 24, 48, 256], "tp": [0, -1, 1 << 24], "T": [-1, 1 << 22],
       "B": [-1, 1 << 17], "Hkv": [0, -1, 3], "rot": [-16, 8, 24, 144], "inter": [2, -1], "amp": [NAN, math.inf],
       "scale": [NAN, math.inf], "max_new": [0, -3], "wsb": [0], "H": [0, 1025], "pages": [0, -1]}


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(L, name):
    f, args = getattr(L, name), CALLS[name]

    def call(**kw):
        return f(*[kw.get(n, v) for n, v in args])

    for n, v in args:
        if isinstance(v, ctypes.c_void_p) and n != "q":
            assert call(**{n: None}) == INVALID, n
            odd = ctypes.c_void_p(0x10001) if n in ("pos", "table", "cu", "len") else ODD
            assert call(**{n: odd}) == INVALID, n
        if n.startswith("ld"):
            assert call(**{n: v - 8}) == INVALID and call(**{n: v + 4}) == INVALID, n
        for bad in BAD.get(n, []):
            if name == "qattn_rotary" and n == "d" and bad == 256:
                continue                                      # rotary alone takes heads up to 512
            if name == "qattn_rotary" and n == "d" and bad == 96:
                continue
            if name == "qattn_cache_read" and n == "Hkv" and bad == 3:
                continue                                      # no query heads there
            assert call(**{n: bad}) == INVALID, (n, bad)
    assert call(T=0) == 0
    if any(n == "B" for n, _ in args):
        assert call(B=0) == 0
    if any(n == "Hq" for n, _ in args):
        assert call(Hq=9) == INVALID and call(Hq=1) == INVALID and call(Hq=2 * 65) == INVALID and call(Hq=2048) == INVALID
    if name == "qattn_cache_append":
        assert call(rot=0) == INVALID                         # q given, nothing to rotate it by


def test_workspace_query(L):
    f = L.qattn_paged_attention_workspace_bytes
    ok = [4, 2, 8, 2, 128, 3, 64, 4]
    assert f(*ok) >= 0
    for i, v in ((0, 0), (1, 0), (0, -1), (2, 9), (3, 0), (4, 96), (5, 0), (6, 40), (7, 0)):
        a = list(ok)
        a[i] = v
        assert f(*a) == 0


def test_frequencies():
    from w4a8_integer_gemm_b200 import rotary_frequencies
    f, amp = rotary_frequencies(128, 1e4)
    assert f.dtype == torch.float64 and f.numel() == 64 and amp == 1.0
    assert f[0] == 1.0 and abs(float(f[32]) - 1e4 ** -0.5) < 1e-15
    assert torch.equal(rotary_frequencies(128, 1e4, "linear", 4.0)[0], f / 4)
    n, _ = rotary_frequencies(128, 1e4, "ntk", 4.0)
    assert n[0] == 1.0 and abs(float(n[-1] * 4 / f[-1]) - 1) < 1e-12          # the slowest pair stretched by 4
    b, amp = rotary_frequencies(128, 5e5, "bands", 8.0, original=8192, low=1.0, high=4.0)
    g, _ = rotary_frequencies(128, 5e5)
    turns = 8192 * g / (2 * math.pi)
    assert amp == 1.0 and torch.equal(b[turns > 4], g[turns > 4]) and torch.allclose(b[turns < 1], g[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and bool(((b[mid] < g[mid]) & (b[mid] > g[mid] / 8)).all())
    y, amp = rotary_frequencies(64, 1e4, "yarn", 16.0, original=4096, low=1.0, high=32.0)
    h, _ = rotary_frequencies(64, 1e4)
    assert abs(amp - (0.1 * math.log(16) + 1)) < 1e-15
    assert y[0] == h[0] and abs(float(y[-1] * 16 / h[-1]) - 1) < 1e-12 and bool((y <= h).all() and (y >= h / 16.0001).all())
    for kw in (dict(rot=7), dict(rot=0), dict(rot=64, scaling="other"), dict(rot=64, factor=0.5),
               dict(rot=64, scaling="bands", low=4.0, high=1.0), dict(rot=64, base=-1.0)):
        with pytest.raises(ValueError):
            rotary_frequencies(**kw)


def test_reference_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]], dtype=np.float16)
    quarter = [np.pi / 2]                                     # one pair turned by a quarter at position 1
    assert np.allclose(ref.rotate64(x, [1], quarter, True)[0, 0], [-2, 1, 3, 4])
    assert np.allclose(ref.rotate64(x, [1], [np.pi / 2, 0.0], False)[0, 0], [-3, 2, 1, 4])
    c, s, m = ref.quantise(np.array([0.0, 15.0, 7.4, 7.5, 8.5], dtype=np.float16), 4)
    assert list(c) == [0, 15, 7, 8, 8] and s == 1 and m == 0  # ties to even
    c, s, m = ref.quantise(np.full(8, -3.5, dtype=np.float16), 4)
    assert not c.any() and s == 0 and m == np.float16(-3.5)
    c, s, m = ref.quantise(np.array([-65504, 65504], dtype=np.float16), 4)
    assert float(m) + 15 * float(s) <= 65504                  # the scale is rounded down: no value overflows
    out, _ = ref.attend(np.ones((2, 4)), np.zeros((3, 4)), np.arange(12.0).reshape(3, 4),
                        np.array([[True, True, False], [False] * 3]), 1.0)
    assert np.allclose(out, [[2, 3, 4, 5], [0, 0, 0, 0]])
