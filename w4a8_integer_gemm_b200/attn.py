"""Attention operators around the W4A8 layer (include/qoq_attn.h).

Rotary positions, a paged key/value cache in 4 or 8 bits that is quantised
as it is written, the attention of new tokens over it, and the causal
attention of whole prompts.  As in the package itself, every function has
the name of the C entry point it calls and only marshals arguments.

    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)                # qkv fp16 [T, Hq + 2 Hkv, d]
    cache = paged_kv_cache(pages, Hkv, d, bits=4)
    rot = Rotary(rotary_frequencies(d, base=5e5)[0].cuda())
    q = qattn_cache_append(k, v, cache, table, cu, kv_len, rotary=rot, q=q)
    o = qattn_paged_attention(q, cache, table, cu, kv_len, max_new=1)  # fp16 [T, Hq, d]; 1: a decode step

The batch: `cu` int32 [B + 1] (row offsets of the sequences' new tokens),
`kv_len` int32 [B] (cached tokens, the new ones included), `table` int32
[B, pages per sequence] (page numbers; one outside the pool is an absent
page).  All of it stays on the device, so the calls can be captured.
"""
from __future__ import annotations

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


_FN = {}    # the library's functions by name, looked up once

# What torch.cuda.current_stream() and current_device() return, without building objects: a decode step's calls are
# a few microseconds of GPU work each, and the two cost as much.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name: str, *args):
    f = _FN.get(name)
    if f is None:
        from . import lib
        f = _FN[name] = getattr(lib(), name)
    status = f(*args)
    if status != 0:
        from . import QoQError
        raise QoQError(name, status)


def _stream(stream, device: int):
    """The raw stream to launch on."""
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _empty(x: torch.Tensor, stream, shape, dtype):
    """Memory beside x, from the pool of the stream that uses it."""
    if stream is None:
        return x.new_empty(shape, dtype=dtype)               # (half of torch.empty's time)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    with torch.cuda.stream(stream):
        return x.new_empty(shape, dtype=dtype)


def _device(x: torch.Tensor, name: str) -> int:
    """The index of x's device, which has to be the current one."""
    i = x.get_device()
    if i < 0 or i != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return i


def _heads(x: torch.Tensor, name: str, device: int, heads=None, d=None, rows=None):
    """(address, row stride) of x fp16 [T, H, d], the heads of a row next to one another."""
    if x.dtype is not torch.float16 or x.dim() != 3 or x.get_device() != device:
        raise ValueError(f"{name} must be a float16 tensor [T, H, d] on the current CUDA device")
    T, H, D = x.shape
    if (heads is not None and H != heads) or (d is not None and D != d) or (rows is not None and T != rows):
        raise ValueError(f"{name} has shape {tuple(x.shape)}")
    s = x.stride()
    if T > 0 and (s[2] != 1 or (H > 1 and s[1] != D)):
        raise ValueError(f"{name}: each row's heads must be contiguous")
    return x.data_ptr(), s[0] if T > 1 else H * D


def _result(out, name: str, x: torch.Tensor, stream, device: int, T: int, H: int, d: int):
    """(out, its address, its row stride) for fp16 [T, H, d]; a new tensor when out is None."""
    if out is None:
        out = _empty(x, stream, (T, H, d), torch.float16)
        return out, out.data_ptr(), H * d
    return out, *_heads(out, name, device, H, d, T)


def _index(x: torch.Tensor, name: str, device: int, n=None):
    """The address of a contiguous int32 array [n]."""
    if x.dtype is not torch.int32 or x.get_device() != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on the rows' device")
    if x.dim() != 1 or (n is not None and x.shape[0] != n):
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

    def args(self, device: int):
        f = self.freq
        if f.dtype is not torch.float64 or f.dim() != 1 or f.get_device() != device or not f.is_contiguous():
            raise ValueError("freq must be a contiguous float64 tensor [rot / 2] on the rows' device")
        return f.data_ptr(), 2 * f.numel(), int(bool(self.interleaved)), float(self.amplitude)


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original: int = 8192, low: float = 1.0, high: Optional[float] = None) -> Tuple[torch.Tensor, float]:
    """(frequencies float64 [rot / 2] on the CPU, amplitude) for `rot` rotated channels: base^(-2i / rot), scaled for
    contexts `factor` times as long as the `original` ones:
      None       as they are;
      "linear"   all divided by factor (positions interpolated);
      "ntk"      base * factor^(rot / (rot - 2)): the slowest pair is stretched by factor, the fastest not at all;
      "bands"    by the turns a pair makes over the original context: below `low` divided by factor, above `high`
                 as they are, in between a blend linear in the turns;
      "yarn"     the same between `low` and `high` turns, but the blend linear in the pair's index, and amplitude
                 0.1 ln(factor) + 1.
    `high` is 4 for "bands" and 32 for "yarn" unless given."""
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
    if high is None:
        high = 4.0 if scaling == "bands" else 32.0
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
    dev = _device(x, "x")
    px, ldx = _heads(x, "x", dev)
    T, H, d = x.shape
    pp = _index(positions, "positions", dev, T)
    freq, rot, inter, amp = rotary.args(dev)
    out, po, ldo = _result(out, "out", x, stream, dev, T, H, d)
    _call("qattn_rotary", px, ldx, pp, freq, T, H, d, rot, inter, amp, po, ldo, _stream(stream, dev))
    return out


# ----------------------------------------------------------------- cache ----
@dataclass(frozen=True)
class PagedKVCache:
    """A pool of pages of 4- or 8-bit keys and values (layouts of include/qoq_attn.h)."""
    k_codes: torch.Tensor   # uint8 [pages, Hkv, page_size, d * bits / 8]
    v_codes: torch.Tensor
    k_par: torch.Tensor     # fp16 [pages, Hkv, page_size, 2]: scale, minimum
    v_par: torch.Tensor
    bits: int               # 4 or 8

    _made = None            # (no field: what _args was made from; a handle that was pickled without it checks itself)

    def __post_init__(self):
        self._check()

    def _check(self):
        """Checks the arrays, and keeps what they come to as arguments beside what it was made from."""
        if self.bits not in (4, 8):
            raise ValueError("a cache has 4 or 8 bits")
        kc, vc, kp, vp = self.k_codes, self.v_codes, self.k_par, self.v_par
        n, dev = kc.shape, kc.get_device()
        if len(n) != 4 or vc.shape != n or kp.shape != (n[0], n[1], n[2], 2) or vp.shape != kp.shape:
            raise ValueError("the cache's arrays do not fit one another")
        if kc.dtype is not torch.uint8 or vc.dtype is not torch.uint8 or kp.dtype is not torch.float16 or \
                vp.dtype is not torch.float16:
            raise ValueError("a cache has uint8 codes and float16 parameters")
        for t in (kc, vc, kp, vp):
            if t.get_device() != dev or not t.is_contiguous():
                raise ValueError("the cache's arrays must be contiguous, on one device")
        made = (kc.data_ptr(), vc.data_ptr(), kp.data_ptr(), vp.data_ptr(), kc.numel(), vc.numel(), kp.numel(), vp.numel())
        object.__setattr__(self, "_made", made)
        object.__setattr__(self, "_args", (dev, (*made[:4], self.bits, n[2], n[0], n[1], n[3] * 8 // self.bits)))

    @property
    def pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def page_size(self) -> int:
        return self.k_codes.shape[2]

    @property
    def d(self) -> int:
        return self.k_codes.shape[3] * 8 // self.bits

    def args(self, device: int):
        """(k_codes, v_codes, k_par, v_par, bits, page_size, pages, Hkv, d)"""
        # A copied or unpickled handle, or one whose tensors were given other memory, has come by _args without a check:
        # they count only for the memory they were made for (0.9 us a call; all checks every time 2.2).
        kc, vc, kp, vp = self.k_codes, self.v_codes, self.k_par, self.v_par
        if self._made != (kc.data_ptr(), vc.data_ptr(), kp.data_ptr(), vp.data_ptr(), kc.numel(), vc.numel(), kp.numel(),
                          vp.numel()):
            self._check()
        dev, args = self._args
        if dev != device:
            raise ValueError("the cache is on another device than the rows")
        return args


def paged_kv_cache(pages: int, Hkv: int, d: int, bits: int = 4, page_size: int = 64, device="cuda") -> PagedKVCache:
    """An empty pool. Its contents are whatever the memory held: pages are read only where tokens were written."""
    if bits not in (4, 8) or d not in (64, 128) or page_size not in (16, 32, 64, 128) or pages < 0 or Hkv < 1:
        raise ValueError("paged_kv_cache: bits 4 or 8, d 64 or 128, page_size 16, 32, 64 or 128")
    codes = [torch.empty(pages, Hkv, page_size, d * bits // 8, dtype=torch.uint8, device=device) for _ in range(2)]
    par = [torch.empty(pages, Hkv, page_size, 2, dtype=torch.float16, device=device) for _ in range(2)]
    return PagedKVCache(*codes, *par, bits)


def _batch(table, cu, kv_len, device: int):
    """(table, table_pages, cu, kv_len, B), checked."""
    if table.dtype is not torch.int32 or table.dim() != 2 or table.get_device() != device or not table.is_contiguous():
        raise ValueError("table must be a contiguous int32 tensor [B, pages per sequence] on the rows' device")
    B, P = table.shape
    return table.data_ptr(), P, _index(cu, "cu", device, B + 1), _index(kv_len, "kv_len", device, B), B


def qattn_cache_append(k: torch.Tensor, v: torch.Tensor, cache: PagedKVCache, table: torch.Tensor, cu: torch.Tensor,
                       kv_len: torch.Tensor, rotary: Optional[Rotary] = None, q: Optional[torch.Tensor] = None,
                       q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Quantises the new tokens' k and v fp16 [T, Hkv, d] into their pages.  With `rotary` the keys are turned by
    their positions first; with `rotary` and q fp16 [T, Hq, d], returns q turned by them (in q_out, which may be
    q).  Rows of no sequence are left alone, in the cache and in q_out."""
    dev = _device(k, "k")
    pk, ldk = _heads(k, "k", dev)
    T, Hkv, d = k.shape
    pv, ldv = _heads(v, "v", dev, Hkv, d, T)
    kc, vc, kp, vp, bits, page, pages, ch, cd = cache.args(dev)
    if ch != Hkv or cd != d:
        raise ValueError("the cache's heads differ from those of k")
    freq, rot, inter, amp = rotary.args(dev) if rotary is not None else (None, 0, 0, 1.0)
    tab, P, pc, pl, B = _batch(table, cu, kv_len, dev)
    pq = po = None
    ldq = ldo = Hq = 0
    if q is not None:
        if rotary is None:
            raise ValueError("q is only rotated: it needs `rotary`")
        pq, ldq = _heads(q, "q", dev, None, d, T)
        Hq = q.shape[1]
        q_out, po, ldo = _result(q_out, "q_out", q, stream, dev, T, Hq, d)
    _call("qattn_cache_append", pk, ldk, pv, ldv, pq, ldq, po, ldo, T, Hq, Hkv, d, freq, rot, inter, amp, bits, page,
          pages, kc, vc, kp, vp, tab, P, pc, pl, B, _stream(stream, dev))
    return q_out if q is not None else None


def qattn_cache_read(cache: PagedKVCache, table: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor, total: int,
                     K: Optional[torch.Tensor] = None, V: Optional[torch.Tensor] = None, stream=None):
    """(K, V) fp16 [total, Hkv, d]: the last cu[b+1] - cu[b] cached tokens of each sequence, as the values their codes
    stand for (zeros where a page is absent)."""
    dev = _device(cache.k_codes, "the cache")
    kc, vc, kp, vp, bits, page, pages, Hkv, d = cache.args(dev)
    tab, P, pc, pl, B = _batch(table, cu, kv_len, dev)
    K, pk, lk = _result(K, "K", cache.k_par, stream, dev, total, Hkv, d)
    V, pv, lv = _result(V, "V", cache.k_par, stream, dev, total, Hkv, d)
    if lk != Hkv * d or lv != Hkv * d:
        raise ValueError("K and V must be contiguous")
    _call("qattn_cache_read", kc, vc, kp, vp, bits, page, pages, Hkv, d, tab, P, pc, pl, B, total, pk, pv,
          _stream(stream, dev))
    return K, V


# ------------------------------------------------------------- attention ----
def qattn_paged_attention_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, d: int, table_pages: int, page_size: int,
                                          max_new: int) -> int:
    from . import lib
    return int(lib().qattn_paged_attention_workspace_bytes(T, B, Hq, Hkv, d, table_pages, page_size, max_new))


def qattn_paged_attention(q: torch.Tensor, cache: PagedKVCache, table: torch.Tensor, cu: torch.Tensor,
                          kv_len: torch.Tensor, scale: Optional[float] = None, max_new: Optional[int] = None,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Attention of the new tokens' q fp16 [T, Hq, d] over the cache, which holds their keys and values already:
    each sees the cached tokens up to its own position.  `max_new`: an upper bound of the sequences' new tokens
    where the caller has one (1 for a decode step); it only picks kernels, and a decode step without it takes half as
    long again.  `scale` defaults to 1 / sqrt(d)."""
    dev = _device(q, "q")
    pq, ldq = _heads(q, "q", dev)
    T, Hq, d = q.shape
    kc, vc, kp, vp, bits, page, pages, Hkv, cd = cache.args(dev)
    if cd != d:
        raise ValueError("the cache's head dimension differs from that of q")
    tab, P, pc, pl, B = _batch(table, cu, kv_len, dev)
    most = max(1, T if max_new is None else int(max_new))
    out, po, ldo = _result(out, "out", q, stream, dev, T, Hq, d)
    if workspace is None:
        need = qattn_paged_attention_workspace_bytes(T, B, Hq, Hkv, d, P, page, most)
        workspace = _empty(q, stream, (max(need, 16),), torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the rows' device")
    _call("qattn_paged_attention", pq, ldq, T, Hq, Hkv, d, kc, vc, kp, vp, bits, page, pages, tab, P, pc, pl, B, most,
          d ** -0.5 if scale is None else float(scale), po, ldo, workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), _stream(stream, dev))
    return out


def qattn_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor,
                           scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Causal attention within each packed prompt: q fp16 [T, Hq, d], k and v fp16 [T, Hkv, d], cu int32 [B + 1] ->
    fp16 [T, Hq, d].  `scale` defaults to 1 / sqrt(d)."""
    dev = _device(q, "q")
    pq, ldq = _heads(q, "q", dev)
    T, Hq, d = q.shape
    pk, ldk = _heads(k, "k", dev, None, d, T)
    Hkv = k.shape[1]
    pv, ldv = _heads(v, "v", dev, Hkv, d, T)
    pc = _index(cu, "cu", dev)
    out, po, ldo = _result(out, "out", q, stream, dev, T, Hq, d)
    _call("qattn_prompt_attention", pq, ldq, pk, ldk, pv, ldv, T, Hq, Hkv, d, pc, cu.shape[0] - 1,
          d ** -0.5 if scale is None else float(scale), po, ldo, _stream(stream, dev))
    return out
