"""Attention operators around the W4A8 layer (include/qoq_attn.h).

Rotary positions, a paged key/value cache in 4 or 8 bits that is quantised
as it is written, the attention of new tokens over it, and the causal
attention of whole prompts.  As in the package itself, every function has
the name of the C entry point it calls and only marshals arguments.

    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)                # qkv fp16 [T, Hq + 2 Hkv, d]
    cache = paged_kv_cache(pages, Hkv, d, bits=4)
    rot = Rotary(rotary_frequencies(d, base=5e5)[0].cuda())
    q = qattn_cache_append(k, v, cache, table, cu, kv_len, rotary=rot, q=q)
    o = qattn_paged_attention(q, cache, table, cu, kv_len)  # fp16 [T, Hq, d]

The batch: `cu` int32 [B + 1] (row offsets of the sequences' new tokens),
`kv_len` int32 [B] (cached tokens, the new ones included), `table` int32
[B, pages per sequence] (page numbers; one outside the pool is an absent
page).  All of it stays on the device, so the calls can be captured.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

# name -> (restype, argtypes); the surface of include/qoq_attn.h
ATTN_SIGNATURES = {
    "qattn_rotary": (_I, [_P, _L, _P, _P, _I, _I, _I, _I, _I, _F, _P, _L, _P]),
    "qattn_cache_append": (_I, [_P, _L, _P, _L, _P, _L, _P, _L, _I, _I, _I, _I, _P, _I, _I, _F, _I, _I, _I,
                                _P, _P, _P, _P, _P, _I, _P, _P, _I, _P]),
    "qattn_cache_read": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P, _P, _I, _I, _P, _P, _P]),
    "qattn_paged_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "qattn_paged_attention": (_I, [_P, _L, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P, _P, _I, _I, _F,
                                   _P, _L, _P, _SZ, _P]),
    "qattn_prompt_attention": (_I, [_P, _L, _P, _L, _P, _L, _I, _I, _I, _I, _P, _I, _F, _P, _L, _P]),
}


def _fn(name):
    from . import lib
    return getattr(lib(), name)


def _check(name: str, status: int):
    if status != 0:
        from . import QoQError
        raise QoQError(name, status)


def _on(stream, device):
    """(raw stream, context in which outputs and scratch are allocated): memory is taken from the pool of the
    stream that uses it."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream, contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _heads(x: torch.Tensor, name: str, device=None, heads=None, d=None, rows=None):
    """x fp16 [T, H, d] on the current device, the heads of a row next to one another; any row stride that is a
    multiple of 8."""
    if not x.is_cuda or x.dtype != torch.float16 or x.dim() != 3:
        raise ValueError(f"{name} must be a CUDA float16 tensor [T, H, d]")
    T, H, D = x.shape
    if T > 0 and (x.stride(2) != 1 or (H > 1 and x.stride(1) != D)):
        raise ValueError(f"{name}: each row's heads must be contiguous")
    if device is None:
        if x.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name} is on another device than the current one")
    elif x.device != device:
        raise ValueError(f"{name} is on another device")
    if (heads is not None and H != heads) or (d is not None and D != d) or (rows is not None and T != rows):
        raise ValueError(f"{name} has shape {tuple(x.shape)}")
    return x.data_ptr(), (x.stride(0) if T > 1 else H * D)


def _index(x: torch.Tensor, name: str, shape, device):
    if not x.is_cuda or x.dtype != torch.int32 or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor on the rows' device")
    if x.dim() != len(shape) or any(s is not None and s != n for s, n in zip(shape, x.shape)):
        raise ValueError(f"{name} has shape {tuple(x.shape)}")
    return x.data_ptr()


# ---------------------------------------------------------------- rotary ----
@dataclass
class Rotary:
    """How positions turn channels: radians per position of each pair (float64 [rot / 2] on the GPU), the pairs'
    layout, and a factor on the result."""
    freq: torch.Tensor
    interleaved: bool = False
    amplitude: float = 1.0

    def args(self, device):
        f = self.freq
        if not f.is_cuda or f.dtype != torch.float64 or f.dim() != 1 or not f.is_contiguous() or f.device != device:
            raise ValueError("freq must be a contiguous float64 tensor [rot / 2] on the rows' device")
        return f.data_ptr(), 2 * f.numel(), int(bool(self.interleaved)), float(self.amplitude)


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original: int = 8192, low: float = 1.0, high: float = 4.0) -> Tuple[torch.Tensor, float]:
    """(frequencies float64 [rot / 2] on the CPU, amplitude) for `rot` rotated channels: base^(-2i / rot), scaled for
    contexts `factor` times as long as the `original` ones:
      None       as they are;
      "linear"   all divided by factor (positions interpolated);
      "ntk"      base * factor^(rot / (rot - 2)): the slowest pair is stretched by factor, the fastest not at all;
      "bands"    by the turns a pair makes over the original context: below `low` divided by factor, above `high`
                 as they are, in between a blend linear in the turns;
      "yarn"     the same between `low` and `high` turns, but the blend linear in the pair's index, and amplitude
                 0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2 or base <= 0 or factor < 1 or original < 1:
        raise ValueError("rotary_frequencies: rot even and >= 2, base > 0, factor >= 1, original >= 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("rotary_frequencies: ntk scaling needs rot >= 4")
        return (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    f = base ** (-2 * i / rot)
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling not in ("bands", "yarn"):
        raise ValueError(f"rotary_frequencies: unknown scaling {scaling!r}")
    if not 0 < low < high:
        raise ValueError("rotary_frequencies: 0 < low < high")
    turns = original * f / (2 * math.pi)
    if scaling == "bands":
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0

    def pair_of(n):     # the (fractional) pair that makes n turns over the original context
        return rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
    first, last = max(math.floor(pair_of(high)), 0), min(math.ceil(pair_of(low)), rot - 1)
    keep = 1 - ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
    return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def qattn_rotary(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """x fp16 [T, H, d] with the first 2 * len(freq) channels of each head turned by positions int32 [T]; out may be
    x."""
    px, ldx = _heads(x, "x")
    T, H, d = x.shape
    pp = _index(positions, "positions", (T,), x.device)
    freq, rot, inter, amp = rotary.args(x.device)
    s, alloc = _on(stream, x.device)
    if out is None:
        with alloc:
            out = torch.empty(T, H, d, dtype=torch.float16, device=x.device)
    po, ldo = _heads(out, "out", x.device, H, d, T)
    _check("qattn_rotary", _fn("qattn_rotary")(px, ldx, pp, freq, T, H, d, rot, inter, amp, po, ldo, s))
    return out


# ----------------------------------------------------------------- cache ----
@dataclass
class PagedKVCache:
    """A pool of pages of 4- or 8-bit keys and values (layouts of include/qoq_attn.h)."""
    k_codes: torch.Tensor   # uint8 [pages, Hkv, page_size, d * bits / 8]
    v_codes: torch.Tensor
    k_par: torch.Tensor     # fp16 [pages, Hkv, page_size, 2]: scale, minimum
    v_par: torch.Tensor
    bits: int               # 4 or 8

    @property
    def pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def d(self) -> int:
        return self.k_codes.shape[3] * 8 // self.bits

    def args(self, device):
        """(k_codes, v_codes, k_par, v_par, bits, page_size, pages, Hkv, d), checked."""
        if self.bits not in (4, 8):
            raise ValueError("a cache has 4 or 8 bits")
        n = self.k_codes.shape
        for t, name, dtype in ((self.k_codes, "k_codes", torch.uint8), (self.v_codes, "v_codes", torch.uint8),
                               (self.k_par, "k_par", torch.float16), (self.v_par, "v_par", torch.float16)):
            if t.dtype != dtype or t.device != device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor on the rows' device")
            if len(n) != 4 or t.shape != (n if dtype == torch.uint8 else n[:3] + (2,)):
                raise ValueError(f"{name} has shape {tuple(t.shape)}")
        return (self.k_codes.data_ptr(), self.v_codes.data_ptr(), self.k_par.data_ptr(), self.v_par.data_ptr(),
                self.bits, n[2], n[0], n[1], n[3] * 8 // self.bits)


def paged_kv_cache(pages: int, Hkv: int, d: int, bits: int = 4, page_size: int = 64, device="cuda") -> PagedKVCache:
    """An empty pool. Its contents are whatever the memory held: pages are read only where tokens were written."""
    if bits not in (4, 8) or d not in (64, 128) or page_size not in (16, 32, 64, 128) or pages < 0 or Hkv < 1:
        raise ValueError("paged_kv_cache: bits 4 or 8, d 64 or 128, page_size 16, 32, 64 or 128")
    codes = [torch.empty(pages, Hkv, page_size, d * bits // 8, dtype=torch.uint8, device=device) for _ in range(2)]
    par = [torch.empty(pages, Hkv, page_size, 2, dtype=torch.float16, device=device) for _ in range(2)]
    return PagedKVCache(*codes, *par, bits)


def _batch(table, cu, kv_len, device):
    """(table, table_pages, cu, kv_len, B), checked."""
    if table.dim() != 2:
        raise ValueError("table must be [B, pages per sequence]")
    B, P = table.shape
    return (_index(table, "table", (B, P), device), P, _index(cu, "cu", (B + 1,), device),
            _index(kv_len, "kv_len", (B,), device), B)


def qattn_cache_append(k: torch.Tensor, v: torch.Tensor, cache: PagedKVCache, table: torch.Tensor, cu: torch.Tensor,
                       kv_len: torch.Tensor, rotary: Optional[Rotary] = None, q: Optional[torch.Tensor] = None,
                       q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Quantises the new tokens' k and v fp16 [T, Hkv, d] into their pages.  With `rotary` the keys are turned by
    their positions first; with `rotary` and q fp16 [T, Hq, d], returns q turned by them (in q_out, which may be
    q).  Rows of no sequence are left alone, in the cache and in q_out."""
    pk, ldk = _heads(k, "k")
    T, Hkv, d = k.shape
    dev = k.device
    pv, ldv = _heads(v, "v", dev, Hkv, d, T)
    kc, vc, kp, vp, bits, page, pages, ch, cd = cache.args(dev)
    if (ch, cd) != (Hkv, d):
        raise ValueError("the cache's heads differ from those of k")
    if q is not None and rotary is None:
        raise ValueError("q is only rotated: it needs `rotary`")
    freq, rot, inter, amp = rotary.args(dev) if rotary is not None else (None, 0, 0, 1.0)
    b = _batch(table, cu, kv_len, dev)
    s, alloc = _on(stream, dev)
    pq = ldq = po = ldo = None
    Hq = 0
    if q is not None:
        pq, ldq = _heads(q, "q", dev, None, d, T)
        Hq = q.shape[1]
        if q_out is None:
            with alloc:
                q_out = torch.empty(T, Hq, d, dtype=torch.float16, device=dev)
        po, ldo = _heads(q_out, "q_out", dev, Hq, d, T)
    _check("qattn_cache_append",
           _fn("qattn_cache_append")(pk, ldk, pv, ldv, pq, ldq or 0, po, ldo or 0, T, Hq, Hkv, d, freq, rot, inter, amp,
                                     bits, page, pages, kc, vc, kp, vp, *b[:4], b[4], s))
    return q_out if q is not None else None


def qattn_cache_read(cache: PagedKVCache, table: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor, total: int,
                     K: Optional[torch.Tensor] = None, V: Optional[torch.Tensor] = None, stream=None):
    """(K, V) fp16 [total, Hkv, d]: the last cu[b+1] - cu[b] cached tokens of each sequence, as the values their codes
    stand for (zeros where a page is absent)."""
    dev = cache.k_codes.device
    if dev.index != torch.cuda.current_device():
        raise ValueError("the cache is on another device than the current one")
    kc, vc, kp, vp, bits, page, pages, Hkv, d = cache.args(dev)
    b = _batch(table, cu, kv_len, dev)
    s, alloc = _on(stream, dev)
    with alloc:
        K = torch.empty(total, Hkv, d, dtype=torch.float16, device=dev) if K is None else K
        V = torch.empty(total, Hkv, d, dtype=torch.float16, device=dev) if V is None else V
    for x, name in ((K, "K"), (V, "V")):
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        _heads(x, name, dev, Hkv, d, total)
    _check("qattn_cache_read", _fn("qattn_cache_read")(kc, vc, kp, vp, bits, page, pages, Hkv, d, *b[:4], b[4], total,
                                                       K.data_ptr(), V.data_ptr(), s))
    return K, V


# ------------------------------------------------------------- attention ----
def qattn_paged_attention_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, d: int, table_pages: int, page_size: int,
                                          max_new: int) -> int:
    return int(_fn("qattn_paged_attention_workspace_bytes")(T, B, Hq, Hkv, d, table_pages, page_size, max_new))


def qattn_paged_attention(q: torch.Tensor, cache: PagedKVCache, table: torch.Tensor, cu: torch.Tensor,
                          kv_len: torch.Tensor, scale: Optional[float] = None, max_new: Optional[int] = None,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Attention of the new tokens' q fp16 [T, Hq, d] over the cache, which holds their keys and values already:
    each sees the cached tokens up to its own position.  `max_new`: an upper bound of the sequences' new tokens
    where the caller has one (1 for a decode step); it only picks kernels.  `scale` defaults to 1 / sqrt(d)."""
    pq, ldq = _heads(q, "q")
    T, Hq, d = q.shape
    dev = q.device
    kc, vc, kp, vp, bits, page, pages, Hkv, cd = cache.args(dev)
    if cd != d:
        raise ValueError("the cache's head dimension differs from that of q")
    b = _batch(table, cu, kv_len, dev)
    most = max(1, T if max_new is None else int(max_new))
    s, alloc = _on(stream, dev)
    with alloc:
        if out is None:
            out = torch.empty(T, Hq, d, dtype=torch.float16, device=dev)
        if workspace is None:
            need = qattn_paged_attention_workspace_bytes(T, b[4], Hq, Hkv, d, b[1], page, most)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    po, ldo = _heads(out, "out", dev, Hq, d, T)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the rows' device")
    _check("qattn_paged_attention",
           _fn("qattn_paged_attention")(pq, ldq, T, Hq, Hkv, d, kc, vc, kp, vp, bits, page, pages, *b[:4], b[4], most,
                                        d ** -0.5 if scale is None else float(scale), po, ldo, workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), s))
    return out


def qattn_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor,
                           scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Causal attention within each packed prompt: q fp16 [T, Hq, d], k and v fp16 [T, Hkv, d], cu int32 [B + 1] ->
    fp16 [T, Hq, d].  `scale` defaults to 1 / sqrt(d)."""
    pq, ldq = _heads(q, "q")
    T, Hq, d = q.shape
    dev = q.device
    pk, ldk = _heads(k, "k", dev, None, d, T)
    Hkv = k.shape[1]
    pv, ldv = _heads(v, "v", dev, Hkv, d, T)
    pc = _index(cu, "cu", (None,), dev)
    s, alloc = _on(stream, dev)
    if out is None:
        with alloc:
            out = torch.empty(T, Hq, d, dtype=torch.float16, device=dev)
    po, ldo = _heads(out, "out", dev, Hq, d, T)
    _check("qattn_prompt_attention",
           _fn("qattn_prompt_attention")(pq, ldq, pk, ldk, pv, ldv, T, Hq, Hkv, d, pc, cu.numel() - 1,
                                         d ** -0.5 if scale is None else float(scale), po, ldo, s))
    return out
