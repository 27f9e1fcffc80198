"""Rotary positions and the 8-bit key / value cache (append, attention with the
rank-factorised bias, eviction): the Python side of the serving entry points in
include/rfb_attn.h.

Tensors that a call makes (outputs, workspace) are allocated on the stream
that it runs on.  Every call may be captured into a CUDA graph; lengths and
positions are read on the device, so a replayed step follows them.

The tensors are checked, made and handed to the C entry points by the
extension _serving_bind (csrc/serve/bind.cpp): a decode step makes thousands of
such calls a second, and marshalling them here, as binding.py does for the long
calls, took two to three times as long as the calls themselves.
"""
from __future__ import annotations

import ctypes
import math
import operator

import torch

from .binding import _on_device, load_library

CACHE_BLOCK = 32  # tokens per scale
E4M3 = torch.float8_e4m3fn
_LAYOUTS = {"half": 0, "interleaved": 1}

_bind = None


def _load_bind():
    """The extension, given the addresses of the library's functions."""
    global _bind
    lib = load_library()
    try:
        from . import _serving_bind
    except ImportError as e:
        raise RuntimeError("the serving extension is not built for this Python and torch "
                           "(run `python -m rank_biased_window_b200.build`)") from e
    if _serving_bind.torch_version != torch.__version__:
        raise RuntimeError(f"the serving extension was built for torch {_serving_bind.torch_version} "
                           "(run `python -m rank_biased_window_b200.build`)")
    names = ("rfb_rotary", "rfb_cache_append", "rfb_attn_fwd_cache_workspace_size",
             "rfb_attn_fwd_cache_counts", "rfb_cache_evict", "rfb_strerror", "rfb_last_cuda_error")
    _serving_bind.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))
    _bind = _serving_bind
    return _bind


def _require(name, t, dtype, shape, device, contiguous=True):
    """Type, device, shape and layout of one tensor; one combined test when all is well."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device
            and t.shape == shape and (not contiguous or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _cuda(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    return t.device


def _on_stream(device, stream, call, *args):
    """call(*args) with the caller's stream current, so that what it allocates
    belongs to the stream it runs on."""
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    with torch.cuda.stream(stream):
        return call(*args)


# ------------------------------------------------------------------- rotary
def rotary_frequencies(rot, base=10000.0, *, scaling="none", factor=1.0, original_length=None,
                       turns=(32.0, 1.0), device=None):
    """Angles per position of the rot / 2 pairs (fp64 [rot / 2], radians) and
    the amplitude of the rotation.

    ``scaling`` stretches the positions for contexts ``factor`` times the
    trained length: "linear" divides every frequency by the factor; "base"
    raises the base so that the slowest pair slows by the factor and the
    fastest keeps its frequency; "by_parts" keeps the pairs that turn more
    than ``turns[0]`` times within ``original_length``, divides those that
    turn less than ``turns[1]`` times, ramps between (over the pair index,
    from the floor of the first to the ceiling of the second), and has the
    amplitude 0.1 ln(factor) + 1.
    """
    rot = int(rot)
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even and >= 0")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError("base must be finite and > 1")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("factor must be finite and >= 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    amplitude = 1.0
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    freqs = float(base) ** (-2.0 * i / max(rot, 1))
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "by_parts":
        if original_length is None or original_length <= 0:
            raise ValueError("by_parts needs original_length, the trained length")
        if not turns[0] > turns[1] > 0:
            raise ValueError("turns must be (more, fewer), both positive")

        def pair(n):  # index of the pair that turns n times within the trained length
            return rot * math.log(original_length / (n * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(turns[0])), 0), min(math.ceil(pair(turns[1])), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freqs = freqs / factor * ramp + freqs * (1.0 - ramp)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError("scaling must be none, linear, base or by_parts")
    return freqs.to(device) if device is not None else freqs, amplitude


def _rotary(q, k, positions, freqs, layout, amplitude, inverse, q_out, k_out, stream):
    bind = _bind
    if bind is None:
        _cuda("q", q)
        bind = _load_bind()
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    args = (q, k, positions, freqs, _LAYOUTS[layout], amplitude, inverse, q_out, k_out)
    if stream is None:
        return bind.rotary(*args)
    return _on_stream(_cuda("q", q), stream, bind.rotary, *args)


def rotary_fwd(q, k, positions, freqs, *, layout="half", amplitude=1.0, q_out=None, k_out=None,
               stream=None):
    """Rotary positions on q [B, H, N, d] and k [B, Hk, N, d] (or None) in one
    kernel: returns the contiguous rotated tensors.

    q and k may be views with any batch, head and token strides (for example
    [B, N, H, d] transposed), so that the rotation also brings them into the
    layout that attention takes; q_out and k_out must not share memory with
    them.  positions: int32 [N] or [B, N]; freqs: fp64
    [rot / 2] from rotary_frequencies (channels from rot on pass through).
    """
    return _rotary(q, k, positions, freqs, layout, amplitude, 0, q_out, k_out, stream)


def rotary_bwd(dq, dk, positions, freqs, *, layout="half", amplitude=1.0, q_out=None, k_out=None,
               stream=None):
    """Gradients of q and k from those of rotary_fwd's outputs (the inverse turn)."""
    return _rotary(dq, dk, positions, freqs, layout, amplitude, 1, q_out, k_out, stream)


class RFBRotary(torch.autograd.Function):
    """Autograd wrapper of rotary_fwd / rotary_bwd.  The rotation is linear and its
    gradient the inverse one, so the backward is this function again."""

    @staticmethod
    def forward(ctx, q, k, positions, freqs, layout, amplitude, inverse=False):
        ctx.save_for_backward(positions, freqs)
        ctx.layout, ctx.amplitude, ctx.inverse = layout, amplitude, inverse
        turn = rotary_bwd if inverse else rotary_fwd
        return turn(q, k, positions, freqs, layout=layout, amplitude=amplitude)

    @staticmethod
    def backward(ctx, dq, dk):
        positions, freqs = ctx.saved_tensors

        def rows(t):
            return t if t is None or t.stride(3) == 1 or t.shape[3] == 1 else t.contiguous()
        # a gradient that nobody wants (a frozen q, or k) is not turned
        need_q, need_k = ctx.needs_input_grad[:2]
        first, second = (rows(dq), rows(dk) if need_k else None) if need_q else (rows(dk), None)
        grads = RFBRotary.apply(first, second, positions, freqs, ctx.layout, ctx.amplitude,
                                not ctx.inverse)
        gq, gk = grads if need_q else (None, grads[0])
        return gq, gk, None, None, None, None, None


def rfb_rotary(q, k, positions, freqs, layout="half", amplitude=1.0):
    """rotary_fwd, differentiable in q and k; its outputs are what rfb_attention takes."""
    return RFBRotary.apply(q, k, positions, freqs, layout, float(amplitude))


# -------------------------------------------------------------------- cache
def _held(name):
    """A tensor or size that a cache is made of.  The calls hold the tensors themselves, so
    another one in its place would be read by some and not by others."""
    def refuse(self, _):
        raise AttributeError(f"a Cache8 keeps the {name} it was made with: write into the tensors, "
                             "or make a new Cache8")
    return property(operator.attrgetter("_" + name), refuse)


class Cache8:
    """Keys, values and key factors of B sequences in 8 bits.

    k, v: e4m3 [B, Hk, cap, d]; w: e4m3 [B, Hk, cap, r] or None; k_scale,
    v_scale, w_scale: fp32 [B, Hk, cap / 32], one power of two per head and 32
    tokens; mass: fp32 [B, Hk, cap], the attention weight that each token
    gathered, or None.  The object holds the tensors, whose contents may be
    written but which cannot be exchanged (the mass can); how many tokens a
    sequence has is the caller's (int32 [B] on the device), one for all layers
    of a model.
    """

    _FIXED = ("k", "v", "w", "k_scale", "v_scale", "w_scale", "device", "B", "Hk", "cap", "d", "r")
    __slots__ = ("mass", "_tensors", *("_" + name for name in _FIXED))

    def __init__(self, k, v, w, k_scale, v_scale, w_scale, mass=None):
        dev = _cuda("k", k)
        if k.dim() != 4:
            raise ValueError("k must be [B, Hk, cap, d]")
        B, Hk, cap, d = k.shape
        if d not in (32, 64, 128):
            raise ValueError("d must be 32, 64 or 128")
        if cap % CACHE_BLOCK:
            raise ValueError(f"the capacity must be a multiple of {CACHE_BLOCK}")
        r = 0 if w is None else w.shape[-1]
        if w is not None and (r % 8 or not 8 <= r <= 64):
            raise ValueError("r must be a multiple of 8 in [8, 64]")
        if (w is None) != (w_scale is None):
            raise ValueError("w and w_scale go together")
        for name, t, c in (("k", k, d), ("v", v, d), ("w", w, r)):
            if t is not None:
                _require(name, t, E4M3, (B, Hk, cap, c), dev)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale), ("w_scale", w_scale)):
            if t is not None:
                _require(name, t, torch.float32, (B, Hk, cap // CACHE_BLOCK), dev)
        if mass is not None:
            _require("mass", mass, torch.float32, (B, Hk, cap), dev)
        self.mass = mass
        for name, x in zip(self._FIXED, (k, v, w, k_scale, v_scale, w_scale, dev, B, Hk, cap, d, r)):
            setattr(self, "_" + name, x)
        self._tensors = (_bind or _load_bind()).cache(k, v, w, k_scale, v_scale, w_scale)

    def __reduce__(self):  # copy and pickle
        return Cache8, (self.k, self.v, self.w, self.k_scale, self.v_scale, self.w_scale, self.mass)

    @classmethod
    def create(cls, B, heads_kv, capacity, d, r=0, *, mass=False, device="cuda"):
        """An empty cache of `capacity` tokens (rounded up to whole blocks) a sequence."""
        cap = -(-int(capacity) // CACHE_BLOCK) * CACHE_BLOCK
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())

        def codes(c):
            return torch.zeros((B, heads_kv, cap, c), dtype=torch.uint8, device=dev).view(E4M3)

        def scales():
            return torch.ones((B, heads_kv, cap // CACHE_BLOCK), device=dev)
        return cls(codes(d), codes(d), codes(r) if r else None, scales(), scales(),
                   scales() if r else None,
                   torch.zeros((B, heads_kv, cap), device=dev) if mass else None)

    def values(self, name):
        """The values that the codes of "k", "v" or "w" stand for, fp32."""
        codes, scales = getattr(self, name), getattr(self, name + "_scale")
        return codes.float() * scales.repeat_interleave(CACHE_BLOCK, dim=2)[..., None]


for _name in Cache8._FIXED:
    setattr(Cache8, _name, _held(_name))
del _name


def cache_append(cache, k, v, w=None, *, start, counts=None, stream=None):
    """Writes rows k, v [B, Hk, n, d] and w [B, Hk, n, r] (bf16) into the cache
    at positions start[b] .. start[b] + counts[b] - 1 (counts None: all n).

    The rows may be views with any batch, head and token strides that are
    multiples of 8.  Rows at or behind the capacity are dropped.  start and
    counts are int32 [B] on the device; the caller keeps the lengths.
    """
    if not isinstance(cache, Cache8):
        raise TypeError("cache must be a Cache8")
    args = (cache._tensors, cache.mass, k, v, w, start, counts)
    if stream is None:
        _bind.append(*args)
    else:
        _on_stream(cache.device, stream, _bind.append, *args)
    return cache


def attn_cache_workspace_size(cache, heads, Nq, with_mass=False) -> int:
    """Bytes of workspace that attn_fwd_cache needs on the cache's device."""
    with _on_device(cache.device):
        return int(load_library().rfb_attn_fwd_cache_workspace_size(
            cache.B, heads, cache.Hk, Nq, cache.cap, cache.d, 1 if with_mass else 0))


def attn_fwd_cache(q, u, cache, lengths, scale=None, *, causal=True, counts=None, mass=None,
                   mass_out=None, decay=1.0, out=None, lse=None, workspace=None, stream=None):
    """O, LSE of Nq query tokens a sequence over the cached tokens, with the
    bias U W^T: q [B, H, Nq, d], u [B, H, Nq, r] (None when the cache holds no
    factors), H a multiple of the cache's heads, lengths int32 [B].

    causal: the queries are the last Nq of the lengths[b] tokens, and query i
    sees the tokens up to its own; otherwise every query sees all of them.  A
    query without tokens gets O = 0 and LSE = -inf.  counts (int32 [B]): a batch
    padded to Nq rows, whose sequences have the first counts[b] of them, as
    cache_append takes its rows; those are then the last counts[b] tokens, and
    the rows behind them get O = 0, LSE = -inf and add no weight.  mass_out (fp32 [B, Hk,
    cap]) receives decay * mass + the softmax weights that each token got,
    summed over the queries of its head; it may be mass itself (cache.mass, to
    gather what cache_evict goes by), and mass None counts as zeros.  out, lse,
    mass_out and workspace must not share memory with one another or with
    anything that is read.
    """
    if not isinstance(cache, Cache8):
        raise TypeError("cache must be a Cache8")
    args = (cache._tensors, q, u, lengths, scale, causal, mass, mass_out, decay, out, lse, workspace,
            counts)
    if stream is None:
        return _bind.attn(*args)
    return _on_stream(cache.device, stream, _bind.attn, *args)


def cache_evict(cache, lengths, keep, recent=0, *, out=None, stream=None):
    """Shrinks each sequence to at most `keep` tokens by accumulated attention
    weight (cache.mass): the last `recent` tokens stay, and of those before
    them the ones with the largest mass, head by head, in their order.

    The kept tokens move to the front of the cache, or of `out` (a Cache8 in
    memory of its own with the same heads and channels, of capacity >= keep).  Returns
    the new lengths (int32 [B]) and the tokens' former positions (int32 [B,
    Hk, keep], -1 behind the last).
    """
    if not isinstance(cache, Cache8):
        raise TypeError("cache must be a Cache8")
    to = cache if out is None else out
    if not isinstance(to, Cache8):
        raise TypeError("out must be a Cache8")
    dev = cache.device
    if cache.mass is None or to.mass is None:
        raise ValueError("eviction needs caches with mass")
    if (to.device, to.B, to.Hk, to.d, to.r) != (dev, cache.B, cache.Hk, cache.d, cache.r):
        raise ValueError("out must have the cache's device, sequences, heads and channels")
    keep, recent = int(keep), int(recent)
    if not 1 <= keep <= to.cap:
        raise ValueError(f"keep must be in [1, {to.cap}], the receiving capacity")
    if recent < 0:
        raise ValueError("recent must be >= 0")
    args = (cache._tensors, cache.mass, to._tensors, to.mass, lengths, keep, min(recent, keep))
    if stream is None:
        return _bind.evict(*args)
    return _on_stream(dev, stream, _bind.evict, *args)
