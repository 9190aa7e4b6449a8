"""The attention layers of a hybrid stack (GDN-2 layers interleaved with causal
sliding-window attention: aixai.ru blog, aiexpert.news/pt), next to the
recurrence's entry points: argument marshalling for the operators
``include/gdn2.h`` declares under "attention layers of a hybrid stack".

    freqs = rope_frequencies(128)
    q, k = qk_norm_rope(q, k, freqs, wq, wk, positions)
    o, lse = attn_fwd(q, k, v, cu_seqlens=None, window=2048)      # prompts, training
    grads = attn_bwd(q, k, v, o, lse, dout, window=2048)
    grads = qk_norm_rope_bwd(q0, k0, freqs, dq, dk, wq, wk, positions)

    kv_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale)   # serving
    o, lse = attn_paged(q, k_cache, v_cache, block_table, seq_lens, ...)
    k, v = kv_cache_read(slots, k_cache, v_cache, k_scale, v_scale)

Shapes: q, o [B, T, Hq, d]; k, v [B, T, Hk, d], d 64 or 128, Hq a multiple of
Hk; packed sequences have B = 1 and ``cu_seqlens`` int32 [N + 1].  Tensors are
float32 or bfloat16, contiguous, on one device; work goes to that device's
current stream.  Caches are [pages, Hk, page size, d] of the tensors' dtype,
or ``torch.float8_e4m3fn`` with uint8 exponent bytes [pages, Hk, page size].
"""
from __future__ import annotations

import math
import operator

import torch

from . import GDN2_BF16, GDN2_F32, _check, _dtype_code, _ptr, lib

GDN2_F8E4M3 = 2
ROPE_INTERLEAVED = 1 << 0
ROPE_NO_NORM = 1 << 1


def _device(*tensors) -> int:
    """The index of the one GPU that holds a call's tensors, all contiguous."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0 or not t.is_contiguous()):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("libgdn2 takes contiguous device tensors")
            raise ValueError(f"tensors on different devices ({tensors[0].device} and {t.device})")
    return dev


def _like(t, name: str, shape, dtype) -> None:
    """A tensor of a call (``_device`` has seen it) of this shape and dtype."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _stream_of(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# torch's own accessor of the same handle where it has one: a microsecond less
# a call than the Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _call(dev: int, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, whatever device is current."""
    if dev == torch.cuda.current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status)


def _heads(q, k, *like_k) -> tuple:
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, H, d]")
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    _like(k, "k", (B, T, Hk, d), q.dtype)
    for t, name in like_k:
        _like(t, name, (B, T, Hk, d), q.dtype)
    return B, T, Hq, Hk, d


def _packed(cu_seqlens, B) -> int:
    """num_seqs of a call (0: B sequences of equal length)."""
    if cu_seqlens is None:
        return 0
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor of num_seqs + 1 values")
    if B != 1:
        raise ValueError("packed sequences need B == 1")
    return cu_seqlens.numel() - 1


def _window(window) -> int:
    """A window as the C ABI's int, which a larger one would wrap around in:
    one of 2^31 - 1 tokens hides nothing."""
    window = operator.index(window)
    if window < 0:
        raise ValueError(f"negative window {window}")
    return min(window, 2 ** 31 - 1)


def _workspace(ws, need: int, dev: int):
    """(tensor or None, bytes) of a given workspace, or of a new one."""
    if ws is None:
        if need == 0:
            return None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the call's device")
    return ws, ws.numel() * ws.element_size()


# ---------------------------------------------------------- norm and rotation
def rope_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device="cuda") -> torch.Tensor:
    """Rotation frequencies, float64 [rotary_dim / 2], radians per position:
    f_j = theta^(-2j / rotary_dim), and for contexts ``factor`` times longer
    than the trained ``original_length``
      "linear"  f_j / factor (positions interpolated);
      "ntk"     theta replaced by theta * factor^(rotary_dim / (rotary_dim - 2)),
                which divides the slowest frequency by factor and keeps the
                fastest;
      "yarn"    by parts: pairs that make fewer than beta_slow turns over
                original_length are interpolated, those with more than
                beta_fast keep f_j, in between the two are mixed linearly in
                the number of turns (YaRN, arXiv:2309.00071, section 3.2; its
                attention temperature goes into ``scale``).  Checkpoints
                trained with a mix that is linear in the pair's index between
                two correction indices have other frequencies in between:
                give ``freqs`` their own table."""
    if rotary_dim <= 0 or rotary_dim % 8:
        raise ValueError("rotary_dim must be a positive multiple of 8")
    if not factor > 0:
        raise ValueError("factor must be positive")
    if scaling == "ntk":
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    f = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_length is None:
            raise ValueError("yarn scaling needs original_length")
        if not beta_fast > beta_slow:
            raise ValueError("yarn scaling needs beta_fast > beta_slow")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device)


def _rope_args(q, k, freqs, wq, wk, positions, interleaved, norm):
    B, T, Hq, Hk, d = _heads(q, k)
    _like(wq, "wq", (d,), torch.float32)
    _like(wk, "wk", (d,), torch.float32)
    _like(positions, "positions", (B, T), torch.int32)
    rot = 0
    if freqs is not None:
        if freqs.dtype != torch.float64 or freqs.dim() != 1:
            raise TypeError("freqs must be a 1-D float64 tensor")
        rot = 2 * freqs.numel()
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (0 if norm else ROPE_NO_NORM)
    return B, T, Hq, Hk, d, rot, flags


def qk_norm_rope(q, k, freqs, wq=None, wk=None, positions=None, interleaved: bool = False, norm: bool = True,
                 eps: float = 1e-6, out=None):
    """Per-head root-mean-square norm of q and k (weights ``wq``, ``wk``
    float32 [d] or None), then the rotation of their first 2 len(freqs)
    channels by position (``positions`` int32 [B, T], None: 0 .. T-1;
    ``freqs`` float64 from ``rope_frequencies``, None: no rotation).
    ``norm=False`` rotates alone.  ``out``: preallocated (q, k) outputs, which
    may be q and k themselves.  Returns (q, k)."""
    dev = _device(q, k, freqs, wq, wk, positions)
    B, T, Hq, Hk, d, rot, flags = _rope_args(q, k, freqs, wq, wk, positions, interleaved, norm)
    if out is None:
        out = torch.empty_like(q), torch.empty_like(k)
    else:
        _device(q, *out)
        _like(out[0], "out[0]", q.shape, q.dtype)
        _like(out[1], "out[1]", k.shape, q.dtype)
    _call(dev, lib().gdn2_qk_norm_rope_fwd, _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(freqs), _ptr(positions), B, T,
          Hq, Hk, d, rot, eps, _dtype_code(q), flags, _ptr(out[0]), _ptr(out[1]))
    return out[0], out[1]


def qk_norm_rope_bwd(q, k, freqs, dq_out, dk_out, wq=None, wk=None, positions=None, interleaved: bool = False,
                     norm: bool = True, eps: float = 1e-6, workspace=None, out=None):
    """Backward of ``qk_norm_rope``: from the gradients of its outputs, a dict
    with dq, dk and (float32 [d]; with the norm only) dwq, dwk.  The weight
    gradients are those at weight one where a weight is None.  ``out`` may
    hold preallocated tensors under those names."""
    dev = _device(q, k, freqs, dq_out, dk_out, wq, wk, positions)
    B, T, Hq, Hk, d, rot, flags = _rope_args(q, k, freqs, wq, wk, positions, interleaved, norm)
    _like(dq_out, "dq_out", q.shape, q.dtype)
    _like(dk_out, "dk_out", k.shape, q.dtype)
    out = dict(out or {})
    for name, like in (("dq", q), ("dk", k)):
        if name not in out:
            out[name] = torch.empty_like(like)
        _like(out[name], name, like.shape, q.dtype)
    need = 0
    if norm:
        for name in ("dwq", "dwk"):
            if name not in out:
                out[name] = torch.empty(d, dtype=torch.float32, device=dev)
            _like(out[name], name, (d,), torch.float32)
        need = int(lib().gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d))
    _device(q, *out.values())
    ws, ws_bytes = _workspace(workspace, need, dev)
    _call(dev, lib().gdn2_qk_norm_rope_bwd, _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(freqs), _ptr(positions),
          _ptr(dq_out), _ptr(dk_out), B, T, Hq, Hk, d, rot, eps, _dtype_code(q), flags, _ptr(out["dq"]),
          _ptr(out["dk"]), _ptr(out.get("dwq")), _ptr(out.get("dwk")), _ptr(ws), ws_bytes)
    return out


# ------------------------------------------------------------ whole sequences
def attn_fwd(q, k, v, cu_seqlens=None, window: int = 0, scale: float | None = None, out=None, lse=None,
             want_lse: bool = True):
    """Causal attention over whole sequences, with ``window`` > 0 over each
    token's last ``window`` keys (itself included).  ``scale`` defaults to
    d^-0.5.  Returns (o, lse): lse float32 [B, T, Hq] is what the backward
    needs (None when ``want_lse`` is False and none is given)."""
    window = _window(window)
    dev = _device(q, k, v, cu_seqlens)
    B, T, Hq, Hk, d = _heads(q, k, (v, "v"))
    ns = _packed(cu_seqlens, B)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
    _device(q, out, lse)
    _like(out, "out", q.shape, q.dtype)
    _like(lse, "lse", (B, T, Hq), torch.float32)
    _call(dev, lib().gdn2_attn_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, T, Hq, Hk, d, ns, window,
          d ** -0.5 if scale is None else scale, _dtype_code(q), _ptr(out), _ptr(lse))
    return out, lse


def attn_bwd_workspace_bytes(B: int, T: int, Hq: int, Hk: int, d: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace ``attn_bwd`` needs (B = 1 and the total T when
    packed; the same for either dtype)."""
    return int(lib().gdn2_attn_bwd_workspace_bytes(B, T, Hq, Hk, d))


def attn_bwd(q, k, v, o, lse, dout, cu_seqlens=None, window: int = 0, scale: float | None = None, workspace=None,
             out=None):
    """Backward of ``attn_fwd``: from its o and lse on the same inputs and
    dL/do, a dict with dq, dk, dv.  ``out`` may hold preallocated tensors
    under those names."""
    window = _window(window)
    dev = _device(q, k, v, o, lse, dout, cu_seqlens)
    B, T, Hq, Hk, d = _heads(q, k, (v, "v"))
    ns = _packed(cu_seqlens, B)
    _like(o, "o", q.shape, q.dtype)
    _like(dout, "dout", q.shape, q.dtype)
    _like(lse, "lse", (B, T, Hq), torch.float32)
    out = dict(out or {})
    for name, like in (("dq", q), ("dk", k), ("dv", v)):
        if name not in out:
            out[name] = torch.empty_like(like)
        _like(out[name], name, like.shape, q.dtype)
    _device(q, *out.values())
    ws, ws_bytes = _workspace(workspace, attn_bwd_workspace_bytes(B, T, Hq, Hk, d), dev)
    _call(dev, lib().gdn2_attn_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(cu_seqlens), B, T,
          Hq, Hk, d, ns, window, d ** -0.5 if scale is None else scale, _dtype_code(q), _ptr(out["dq"]),
          _ptr(out["dk"]), _ptr(out["dv"]), _ptr(ws), ws_bytes)
    return out


# ------------------------------------------------------------- paged cache
def _cache(k_cache, v_cache, k_scale, v_scale, dtype) -> tuple:
    """(pages, Hk, page size, d, cache dtype code)"""
    if k_cache.dim() != 4:
        raise ValueError("caches must be [pages, Hk, page size, d]")
    if k_cache.dtype not in (dtype, torch.float8_e4m3fn):
        raise TypeError(f"a cache of {k_cache.dtype} does not go with {dtype} (its own dtype or torch.float8_e4m3fn)")
    _like(v_cache, "v_cache", k_cache.shape, k_cache.dtype)
    P, Hk, page, d = k_cache.shape
    f8 = k_cache.dtype == torch.float8_e4m3fn
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if f8 != (t is not None):
            raise ValueError(f"{name} goes with a torch.float8_e4m3fn cache")
        _like(t, name, (P, Hk, page), torch.uint8)
    code = GDN2_F8E4M3 if f8 else (GDN2_BF16 if dtype == torch.bfloat16 else GDN2_F32)
    return P, Hk, page, d, code


def kv_cache_write(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None) -> None:
    """Stores keys and values [..., Hk, d] of n tokens into ``slots`` (int64,
    n values; slot = page * page size + row; outside the cache, as -1:
    skipped; no slot twice).  A ``torch.float8_e4m3fn`` cache takes them
    quantised, with a power-of-two scale per (token, kv head) row."""
    dev = _device(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    dt = _dtype_code(k)
    P, Hk, page, d, code = _cache(k_cache, v_cache, k_scale, v_scale, k.dtype)
    n = slots.numel()
    if slots.dtype != torch.int64:
        raise TypeError("slots must be int64")
    if k.dim() < 2 or tuple(k.shape[-2:]) != (Hk, d) or k.numel() != n * Hk * d:
        raise ValueError(f"k must hold {n} tokens of [{Hk}, {d}]")
    _like(v, "v", k.shape, k.dtype)
    _call(dev, lib().gdn2_kv_cache_write, _ptr(k), _ptr(v), _ptr(slots), n, Hk, d, P, page, dt, code, _ptr(k_cache),
          _ptr(v_cache), _ptr(k_scale), _ptr(v_scale))


def kv_cache_read(slots, k_cache, v_cache, k_scale=None, v_scale=None, dtype=None, out=None):
    """The keys and values of ``slots`` (int64 [n]), each [n, Hk, d] of
    ``dtype`` (a quantised cache: bfloat16 by default, both exact, but for
    float32 rows under 2^-116, whose smallest values bfloat16 rounds; else the
    cache's own).  A slot outside the cache reads as zeros.  ``out``:
    preallocated (k, v).  Returns (k, v)."""
    dev = _device(slots, k_cache, v_cache, k_scale, v_scale)
    if dtype is None:
        dtype = torch.bfloat16 if k_cache.dtype == torch.float8_e4m3fn else k_cache.dtype
    P, Hk, page, d, code = _cache(k_cache, v_cache, k_scale, v_scale, dtype)
    if slots.dtype != torch.int64 or slots.dim() != 1:
        raise TypeError("slots must be 1-D int64")
    n = slots.numel()
    if out is None:
        out = tuple(torch.empty((n, Hk, d), dtype=dtype, device=dev) for _ in range(2))
    _device(slots, *out)
    _like(out[0], "out[0]", (n, Hk, d), dtype)
    _like(out[1], "out[1]", (n, Hk, d), dtype)
    _call(dev, lib().gdn2_kv_cache_read, _ptr(slots), n, Hk, d, P, page, _dtype_code(out[0]), code, _ptr(k_cache),
          _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(out[0]), _ptr(out[1]))
    return out[0], out[1]


def attn_paged_workspace_bytes(q, k_cache, block_table, cu_seqlens=None, window: int = 0) -> int:
    """Bytes of workspace ``attn_paged`` needs for these tensors (0: none)."""
    B, T, Hq, d = q.shape
    ns = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    return int(lib().gdn2_attn_paged_workspace_bytes(B, T, Hq, k_cache.shape[1], d, ns, k_cache.shape[2],
                                                     block_table.shape[1], _window(window)))


def attn_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, k_scale=None, v_scale=None,
               window: int = 0, scale: float | None = None, out=None, lse=None, want_lse: bool = False,
               workspace=None):
    """Attention of new tokens over a paged cache that already holds their own
    keys and values (``kv_cache_write``).  q [N, T, Hq, d] (T new tokens for
    each of N sequences; decode is T = 1) or packed [1, T, Hq, d] with
    ``cu_seqlens`` (a chunk of a prompt among single tokens, say; a batch of
    single tokens alone runs faster unpacked);
    ``block_table`` int32 [N, max pages], ``seq_lens`` int32 [N] keys of each
    sequence, the new ones included.  Returns (o, lse or None)."""
    window = _window(window)
    dev = _device(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, k_scale, v_scale)
    if q.dim() != 4:
        raise ValueError("q must be [N, T, Hq, d]")
    B, T, Hq, d = q.shape
    dt = _dtype_code(q)
    P, Hk, page, dc, code = _cache(k_cache, v_cache, k_scale, v_scale, q.dtype)
    if dc != d:
        raise ValueError(f"the cache's head width {dc} is not q's {d}")
    ns = _packed(cu_seqlens, B)
    N = ns if ns else B
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, max pages]")
    _like(block_table, "block_table", (N, block_table.shape[1]), torch.int32)
    _like(seq_lens, "seq_lens", (N,), torch.int32)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
    _device(q, out, lse)
    _like(out, "out", q.shape, q.dtype)
    _like(lse, "lse", (B, T, Hq), torch.float32)
    mp = block_table.shape[1]
    need = 0
    if workspace is None:
        need = int(lib().gdn2_attn_paged_workspace_bytes(B, T, Hq, Hk, d, ns, page, mp, window))
    ws, ws_bytes = _workspace(workspace, need, dev)
    _call(dev, lib().gdn2_attn_paged, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
          _ptr(block_table), _ptr(seq_lens), _ptr(cu_seqlens), B, T, Hq, Hk, d, ns, P, page, mp, window,
          d ** -0.5 if scale is None else scale, dt, code, _ptr(out), _ptr(lse), _ptr(ws), ws_bytes)
    return out, lse
