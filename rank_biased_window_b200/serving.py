"""Rotary positions and the 8-bit key / value cache (append, attention with the
rank-factorised bias, eviction): the Python side of the serving entry points in
include/rfb_attn.h.

Argument marshalling only, as in binding.py.  Tensors that a call makes
(outputs, workspace) are allocated on the stream that it runs on.  Every call
may be captured into a CUDA graph; lengths and positions are read on the
device, so a replayed step follows them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import RFB_ERR_WORKSPACE, _check, _on_device, load_library

CACHE_BLOCK = 32  # tokens per scale
E4M3 = torch.float8_e4m3fn
_LAYOUTS = {"half": 0, "interleaved": 1}
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


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


_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _launch(device, stream, call, *args):
    """call(*args, stream pointer) with the device and the stream current, so
    that what the call allocates belongs to the stream it runs on.  The usual
    case, the current stream of the current device, changes neither."""
    if stream is None:
        index = device.index
        if index == _current_device():
            return call(*args, _raw_stream(index))
    with _on_device(device):
        if stream is None:
            return call(*args, _raw_stream(device.index))
        with torch.cuda.stream(stream):
            return call(*args, stream.cuda_stream)


def _p(t):
    return None if t is None else t.data_ptr()


def _empty_like(t):
    """A contiguous tensor of t's shape and type."""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


_Strides6, _Strides9 = ctypes.c_longlong * 6, ctypes.c_longlong * 9


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


def _rotary(q, k, positions, freqs, layout, amplitude, inverse, q_out, k_out, st):
    dev, dtype, shape = q.device, q.dtype, q.shape
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if dtype not in _DTYPES:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {dtype}")
    if len(shape) != 4:
        raise ValueError("q must be [B, H, N, d]")
    B, H, N, d = shape
    sq, Hk, sk = q.stride(), 0, (0, 0, 0, 1)
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be [B, H, N, d]")
        Hk, sk = k.shape[1], k.stride()
        _require("k", k, dtype, (B, Hk, N, d), dev, False)
    if d > 1 and (sq[3] != 1 or sk[3] != 1):
        raise ValueError(f"{'q' if sq[3] != 1 else 'k'} must have contiguous channels")
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be [rot / 2]")
    pairs = freqs.shape[0]
    _require("freqs", freqs, torch.float64, (pairs,), dev)
    if 2 * pairs > d:
        raise ValueError(f"freqs has {pairs} pairs, more than half of d = {d}")
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
        raise ValueError("positions must be [N] or [B, N]")
    own_rows = positions.dim() == 2
    _require("positions", positions, torch.int32, (B, N) if own_rows else (N,), dev)
    if q_out is None:
        q_out = _empty_like(q)
    else:
        _require("q_out", q_out, dtype, shape, dev)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = _empty_like(k)
    else:
        _require("k_out", k_out, dtype, k.shape, dev)
    strides = _Strides6(sq[0], sq[1], sq[2], sk[0], sk[1], sk[2])
    at = ctypes.addressof(strides)
    rc = load_library().rfb_rotary(
        q.data_ptr(), _p(k), q_out.data_ptr(), _p(k_out), positions.data_ptr(), freqs.data_ptr(),
        B, H, Hk, N, d, 2 * pairs, at, at + 24, N if own_rows else 0, _LAYOUTS[layout],
        _DTYPES[dtype], amplitude, inverse, st)
    if rc:
        _check(rc, "rfb_rotary")
    return q_out, k_out


def rotary_fwd(q, k, positions, freqs, *, layout="half", amplitude=1.0, q_out=None, k_out=None,
               stream=None):
    """Rotary positions on q [B, H, N, d] and k [B, Hk, N, d] (or None) in one
    kernel: returns the contiguous rotated tensors.

    q and k may be views with any batch, head and token strides (for example
    [B, N, H, d] transposed), so that the rotation also brings them into the
    layout that attention takes.  positions: int32 [N] or [B, N]; freqs: fp64
    [rot / 2] from rotary_frequencies (channels from rot on pass through).
    """
    return _launch(_cuda("q", q), stream, _rotary, q, k, positions, freqs, layout, amplitude, 0,
                   q_out, k_out)


def rotary_bwd(dq, dk, positions, freqs, *, layout="half", amplitude=1.0, q_out=None, k_out=None,
               stream=None):
    """Gradients of q and k from those of rotary_fwd's outputs (the inverse turn)."""
    return _launch(_cuda("dq", dq), stream, _rotary, dq, dk, positions, freqs, layout, amplitude, 1,
                   q_out, k_out)


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
        gq, gk = RFBRotary.apply(rows(dq), rows(dk), positions, freqs, ctx.layout, ctx.amplitude,
                                 not ctx.inverse)
        return gq, gk, None, None, None, None, None


def rfb_rotary(q, k, positions, freqs, layout="half", amplitude=1.0):
    """rotary_fwd, differentiable in q and k; its outputs are what rfb_attention takes."""
    return RFBRotary.apply(q, k, positions, freqs, layout, float(amplitude))


# -------------------------------------------------------------------- cache
class Cache8:
    """Keys, values and key factors of B sequences in 8 bits.

    k, v: e4m3 [B, Hk, cap, d]; w: e4m3 [B, Hk, cap, r] or None; k_scale,
    v_scale, w_scale: fp32 [B, Hk, cap / 32], one power of two per head and 32
    tokens; mass: fp32 [B, Hk, cap], the attention weight that each token
    gathered, or None.  The object holds the tensors and their addresses; how
    many tokens a sequence has is the caller's (int32 [B] on the device), one
    for all layers of a model.
    """

    __slots__ = ("k", "v", "w", "k_scale", "v_scale", "w_scale", "mass", "device", "B", "Hk", "cap",
                 "d", "r", "_ptrs", "_workspace_bytes")

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
        self.k, self.v, self.w = k, v, w
        self.k_scale, self.v_scale, self.w_scale = k_scale, v_scale, w_scale
        self.mass, self.device = mass, dev
        self.B, self.Hk, self.cap, self.d, self.r = B, Hk, cap, d, r
        self._ptrs = tuple(_p(t) for t in (k, v, w, k_scale, v_scale, w_scale))
        self._workspace_bytes = {}  # by (heads, Nq, with mass)

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


def cache_append(cache, k, v, w=None, *, start, counts=None, stream=None):
    """Writes rows k, v [B, Hk, n, d] and w [B, Hk, n, r] (bf16) into the cache
    at positions start[b] .. start[b] + counts[b] - 1 (counts None: all n).

    The rows may be views with any batch, head and token strides that are
    multiples of 8.  Rows at or behind the capacity are dropped.  start and
    counts are int32 [B] on the device; the caller keeps the lengths.
    """
    if not isinstance(cache, Cache8):
        raise TypeError("cache must be a Cache8")
    return _launch(cache.device, stream, _append, cache, k, v, w, start, counts)


def _append(cache, k, v, w, start, counts, st):
    dev, B, Hk, d, r = cache.device, cache.B, cache.Hk, cache.d, cache.r
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [B, Hk, n, d]")
    n = k.shape[2]
    _require("k", k, torch.bfloat16, (B, Hk, n, d), dev, False)
    _require("v", v, torch.bfloat16, (B, Hk, n, d), dev, False)
    if r:
        _require("w", w, torch.bfloat16, (B, Hk, n, r), dev, False)
    elif w is not None:
        raise ValueError("w given, but the cache holds no factors (r = 0)")
    _require("start", start, torch.int32, (B,), dev)
    if counts is not None:
        _require("counts", counts, torch.int32, (B,), dev)
    sk, sv, sw = k.stride(), v.stride(), w.stride() if r else (0, 0, 0, 1)
    if sk[3] * sv[3] * sw[3] != 1 or (sk[0] | sk[1] | sk[2] | sv[0] | sv[1] | sv[2] | sw[0] | sw[1]
                                      | sw[2]) % 8:
        if n:
            raise ValueError("k, v and w must have contiguous channels and strides of multiples of 8")
    strides = _Strides9(sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], sw[0], sw[1], sw[2])
    rc = load_library().rfb_cache_append(
        k.data_ptr(), v.data_ptr(), _p(w), ctypes.addressof(strides), *cache._ptrs, _p(cache.mass),
        start.data_ptr(), _p(counts), B, Hk, n, cache.cap, d, r, st)
    if rc:
        _check(rc, "rfb_cache_append")
    return cache


def attn_cache_workspace_size(cache, heads, Nq, with_mass=False) -> int:
    """Bytes of workspace that attn_fwd_cache needs on the cache's device."""
    with _on_device(cache.device):
        return int(load_library().rfb_attn_fwd_cache_workspace_size(
            cache.B, heads, cache.Hk, Nq, cache.cap, cache.d, 1 if with_mass else 0))


def attn_fwd_cache(q, u, cache, lengths, scale=None, *, causal=True, mass=None, mass_out=None,
                   decay=1.0, out=None, lse=None, workspace=None, stream=None):
    """O, LSE of Nq query tokens a sequence over the cached tokens, with the
    bias U W^T: q [B, H, Nq, d], u [B, H, Nq, r] (None when the cache holds no
    factors), H a multiple of the cache's heads, lengths int32 [B].

    causal: the queries are the last Nq of the lengths[b] tokens, and query i
    sees the tokens up to its own; otherwise every query sees all of them.  A
    query without tokens gets O = 0 and LSE = -inf.  mass_out (fp32 [B, Hk,
    cap]) receives decay * mass + the softmax weights that each token got,
    summed over the queries of its head; it may be mass itself (cache.mass, to
    gather what cache_evict goes by), and mass None counts as zeros.
    """
    if not isinstance(cache, Cache8):
        raise TypeError("cache must be a Cache8")
    return _launch(cache.device, stream, _attn, q, u, cache, lengths, scale, causal, mass, mass_out,
                   decay, out, lse, workspace)


def _attn(q, u, cache, lengths, scale, causal, mass, mass_out, decay, out, lse, workspace, st):
    dev, B, Hk, cap, d, r = cache.device, cache.B, cache.Hk, cache.cap, cache.d, cache.r
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d]")
    _, H, Nq, _ = q.shape
    _require("q", q, torch.bfloat16, (B, H, Nq, d), dev)
    if r:
        _require("u", u, torch.bfloat16, (B, H, Nq, r), dev)
    elif u is not None:
        raise ValueError("u given, but the cache holds no factors (r = 0)")
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"{H} query heads are not a multiple of the cache's {Hk}")
    _require("lengths", lengths, torch.int32, (B,), dev)
    if mass is not None:
        if mass_out is None:
            raise ValueError("mass needs mass_out (which may be the same tensor)")
        _require("mass", mass, torch.float32, (B, Hk, cap), dev)
    if mass_out is not None:
        _require("mass_out", mass_out, torch.float32, (B, Hk, cap), dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _require("out", out, torch.bfloat16, (B, H, Nq, d), dev)
    if lse is None:
        lse = cache.k_scale.new_empty((B, H, Nq))
    else:
        _require("lse", lse, torch.float32, (B, H, Nq), dev)
    if workspace is None:
        key = (H, Nq, mass_out is not None)
        need = cache._workspace_bytes.get(key)
        if need is None:
            need = cache._workspace_bytes[key] = attn_cache_workspace_size(cache, *key)
        workspace = cache.k_scale.new_empty((need + 19) // 4)
    elif (not isinstance(workspace, torch.Tensor) or workspace.device != dev
          or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    rc = load_library().rfb_attn_fwd_cache(
        q.data_ptr(), _p(u), *cache._ptrs, lengths.data_ptr(), _p(mass), _p(mass_out), decay,
        out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), B, H, Hk, Nq, cap, d, r,
        d ** -0.5 if scale is None else scale, 1 if causal else 0, st)
    if rc == RFB_ERR_WORKSPACE:
        raise RuntimeError(
            f"rfb_attn_fwd_cache: workspace of "
            f"{attn_cache_workspace_size(cache, H, Nq, mass_out is not None)} bytes needed")
    if rc:
        _check(rc, "rfb_attn_fwd_cache")
    return out, lse


def cache_evict(cache, lengths, keep, recent=0, *, out=None, stream=None):
    """Shrinks each sequence to at most `keep` tokens by accumulated attention
    weight (cache.mass): the last `recent` tokens stay, and of those before
    them the ones with the largest mass, head by head, in their order.

    The kept tokens move to the front of the cache, or of `out` (a Cache8 of
    its own with the same heads and channels, of capacity >= keep).  Returns
    the new lengths (int32 [B]) and the tokens' former positions (int32 [B,
    Hk, keep], -1 behind the last).
    """
    if not isinstance(cache, Cache8):
        raise TypeError("cache must be a Cache8")
    to = cache if out is None else out
    if not isinstance(to, Cache8):
        raise TypeError("out must be a Cache8")
    dev, B, Hk = cache.device, cache.B, cache.Hk
    if cache.mass is None or to.mass is None:
        raise ValueError("eviction needs caches with mass")
    if (to.device, to.B, to.Hk, to.d, to.r) != (dev, B, Hk, cache.d, cache.r):
        raise ValueError("out must have the cache's device, sequences, heads and channels")
    keep, recent = int(keep), int(recent)
    if not 1 <= keep <= to.cap:
        raise ValueError(f"keep must be in [1, {to.cap}], the receiving capacity")
    if recent < 0:
        raise ValueError("recent must be >= 0")
    _require("lengths", lengths, torch.int32, (B,), dev)
    return _launch(dev, stream, _evict, cache, to, lengths, keep, min(recent, keep))


def _evict(cache, to, lengths, keep, recent, st):
    new_lengths = torch.empty_like(lengths)
    kept = lengths.new_empty((cache.B, cache.Hk, keep))
    rc = load_library().rfb_cache_evict(
        *cache._ptrs, cache.mass.data_ptr(), *to._ptrs, to.mass.data_ptr(), lengths.data_ptr(),
        new_lengths.data_ptr(), kept.data_ptr(), cache.B, cache.Hk, cache.cap, to.cap, cache.d,
        cache.r, keep, recent, st)
    if rc:
        _check(rc, "rfb_cache_evict")
    return new_lengths, kept
