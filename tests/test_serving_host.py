"""Serving operators without a GPU: argument checks of the C entry points and
of the Python side, the frequency table, and the tests' own 64-bit definitions
against independent ones."""
import math

import pytest
import torch

from tests import _serving_ref as ref


# ---------------------------------------------------------- C entry points
def _rotary(lib, **kw):
    a = dict(q=None, k=None, qo=None, ko=None, pos=None, f=None, B=1, H=1, Hk=1, N=4, d=64, rot=64,
             qs=None, ks=None, ps=4, layout=0, dtype=0, amp=1.0, inv=0)
    a.update(kw)
    return lib.rfb_rotary(*a.values(), None)


def test_rotary_host_checks(rfb_lib):
    lib = rfb_lib.load_library()
    assert _rotary(lib, B=0) == 0 and _rotary(lib, N=0) == 0 and _rotary(lib, H=0, Hk=0) == 0
    assert _rotary(lib) == 1                      # null pointers
    assert _rotary(lib, B=-1) == 1
    assert _rotary(lib, layout=2) == 1
    assert _rotary(lib, dtype=3) == 1
    assert _rotary(lib, amp=float("nan")) == 1
    assert _rotary(lib, ps=-1) == 1
    assert _rotary(lib, rot=63) == 2
    assert _rotary(lib, rot=66) == 2              # more than d
    assert _rotary(lib, d=2048) == 2


def test_cache_append_host_checks(rfb_lib):
    lib = rfb_lib.load_library()

    def call(B=1, Hk=1, n=1, cap=64, d=64, r=0, ptrs=13):
        return lib.rfb_cache_append(*([None] * ptrs), B, Hk, n, cap, d, r, None)
    assert call(B=0) == 0 and call(n=0) == 0 and call(Hk=0) == 0 and call(cap=0) == 0
    assert call() == 1                            # null pointers
    assert call(n=-1) == 1 and call(B=-1) == 1
    assert call(d=48) == 2 and call(r=4) == 2 and call(r=72) == 2
    assert call(cap=40) == 2                      # not whole blocks


def test_attn_cache_host_checks(rfb_lib):
    lib = rfb_lib.load_library()

    def call(B=1, H=2, Hk=1, Nq=1, cap=64, d=64, r=0, scale=0.1, decay=1.0):
        return lib.rfb_attn_fwd_cache(*([None] * 11), decay, None, None, None, 0, B, H, Hk, Nq,
                                      cap, d, r, scale, 1, None)
    assert call(B=0) == 0 and call(Nq=0) == 0 and call(H=0) == 0
    assert call() == 1                            # null pointers
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1 and call(scale=-1.0) == 1
    assert call(decay=float("nan")) == 1
    assert call(H=3, Hk=2) == 1 and call(Hk=0) == 1
    assert call(d=96) == 2 and call(r=12) == 2 and call(cap=33) == 2
    size = lib.rfb_attn_fwd_cache_workspace_size
    assert size(0, 2, 1, 1, 64, 64, 0) == 0 and size(1, 3, 2, 1, 64, 64, 0) == 0
    assert size(1, 2, 1, 1, 64, 48, 0) == 0


def test_cache_evict_host_checks(rfb_lib):
    lib = rfb_lib.load_library()

    def call(B=1, Hk=1, cap=64, cap_out=64, d=64, r=0, keep=8, recent=0):
        return lib.rfb_cache_evict(*([None] * 17), B, Hk, cap, cap_out, d, r, keep, recent, None)
    assert call(B=0) == 0 and call(Hk=0) == 0
    assert call() == 1                            # null pointers
    assert call(keep=0) == 1 and call(keep=65) == 1 and call(recent=-1) == 1
    assert call(d=16) == 2 and call(cap_out=40) == 2 and call(r=3) == 2


# --------------------------------------------------------------- Python side
def test_python_refuses_host_tensors():
    import rank_biased_window_b200 as rfb
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        rfb.rotary_fwd(q, None, pos, f)
    with pytest.raises(TypeError, match="Tensor"):
        rfb.rotary_fwd([1.0], None, pos, f)
    c = torch.zeros(1, 1, 32, 64, dtype=torch.uint8).view(ref.E4M3)
    s = torch.ones(1, 1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        rfb.Cache8(c, c, None, s, s, None)
    for call in (lambda: rfb.cache_append(c, q, q, start=pos), lambda: rfb.cache_evict(c, pos, 4),
                 lambda: rfb.attn_fwd_cache(q, None, c, pos)):
        with pytest.raises(TypeError, match="Cache8"):
            call()


def test_extension_loads_and_refuses(rfb_lib):
    """The marshalling extension of this build: its symbols resolve, and it refuses before any launch."""
    from rank_biased_window_b200 import serving
    bind = serving._load_bind()
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bind.rotary(q, None, q, q, 0, 1.0, 0, None, None)
    with pytest.raises(TypeError, match="expected 9 arguments"):
        bind.rotary(q)
    # numbers, shapes and types in the messages
    c = torch.zeros(2, 2, 64, 64, dtype=torch.uint8).view(ref.E4M3)
    s, n = torch.ones(2, 2, 2), torch.zeros(2, dtype=torch.int32)
    held = bind.cache(c, c, None, s, s, None)
    q3 = torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16)
    for err, match, args in (
            (ValueError, "3 query heads .* cache's 2", (q3, None, n)),
            (ValueError, r"lengths has shape \(1,\), expected \(2,\)", (q3[:, :2].contiguous(), None, n[:1])),
            (ValueError, r"q has shape \(1, 2, 4, 64\), expected \(2, 2, 4, 64\)", (q, None, n)),
            (TypeError, "q must be torch.bfloat16, got Float", (q3.float(), None, n)),
            (ValueError, "no factors", (q3, q3, n))):
        with pytest.raises(err, match=match):
            bind.attn(held, *args, None, True, None, None, 1.0, None, None, None)
    for call in (bind.append, bind.attn, bind.evict):
        with pytest.raises((TypeError, ValueError)):
            call(*[None] * {bind.append: 7, bind.attn: 12, bind.evict: 7}[call])


def test_rotary_frequencies():
    import rank_biased_window_b200 as rfb
    f, a = rfb.rotary_frequencies(64, 10000.0)
    assert f.dtype is torch.float64 and f.shape == (32,) and a == 1.0
    assert float(f[0]) == 1.0 and math.isclose(float(f[31]), 10000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, _ = rfb.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin, f / 4, rtol=1e-15)
    # "base": the fastest pair as it was, the slowest slowed by the factor
    nb, _ = rfb.rotary_frequencies(64, scaling="base", factor=4.0)
    assert float(nb[0]) == 1.0 and math.isclose(float(nb[31]), float(f[31]) / 4, rel_tol=1e-12)
    # "by_parts": unchanged, divided, and between in the ramp
    bp, a = rfb.rotary_frequencies(64, scaling="by_parts", factor=4.0, original_length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.allclose(bp[turns > 64], f[turns > 64], rtol=1e-14)
    assert torch.allclose(bp[turns < 0.5], f[turns < 0.5] / 4, rtol=1e-14)
    assert bool(((bp <= f) & (bp >= f / 4 * (1 - 1e-12))).all())
    assert math.isclose(a, 0.1 * math.log(4.0) + 1.0)
    assert rfb.rotary_frequencies(0)[0].numel() == 0
    assert rfb.rotary_frequencies(2, scaling="base", factor=8.0)[0].tolist() == [1.0]
    for bad in (dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="by_parts"), dict(rot=8, factor=0.5),
                dict(rot=8, scaling="by_parts", original_length=100, turns=(1.0, 2.0))):
        with pytest.raises(ValueError):
            rfb.rotary_frequencies(**bad)


# ----------------------------------------------------- the tests' definitions
def test_reference_scale_is_the_closed_form():
    for amax in (0.0, 1e-30, 1.0, 447.9, 448.0, 448.1, 3.5, 896.0, 1e9, 1e30):
        s = ref.scale_of(amax)
        e = 0 if amax == 0 else math.ceil(math.log2(amax / 448.0))
        assert s == 2.0 ** min(max(e if amax else -40, -40), 40)


def test_reference_rotary_is_a_complex_turn():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, 2, 5, 8, generator=g, dtype=torch.float64)
    pos, f = torch.tensor([0, 1, -3, 7, 100000]), torch.tensor([1.0, 0.01], dtype=torch.float64)
    y, _ = ref.rotary(x, pos, f, "interleaved")
    z = torch.view_as_complex(x[..., :4].reshape(1, 2, 5, 2, 2).contiguous())
    turn = torch.exp(1j * pos.double()[:, None] * f)
    want = torch.view_as_real(z * turn).reshape(1, 2, 5, 4)
    assert torch.allclose(y[..., :4], want, atol=1e-12) and torch.equal(y[..., 4:], x[..., 4:])
    h, _ = ref.rotary(x[..., [0, 2, 1, 3, 4, 5, 6, 7]], pos, f, "half")
    assert torch.allclose(h[..., [0, 2, 1, 3]], want, atol=1e-12)
    back, _ = ref.rotary(y, pos, f, "interleaved", inverse=True)
    assert torch.allclose(back, x, atol=1e-12)


def test_reference_attention_is_the_oracle(oracle_mod):
    """Without a mask the cached attention is the framework's attention with
    the key side's values in the cache."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, u, w = r(2, 3, 9, 32), r(2, 3, 9, 32), r(2, 3, 9, 32), r(2, 3, 9, 8), r(2, 3, 9, 8)
    o, lse, _, _ = ref.attention(q, u, k, v, w, [9, 9], 0.2, False)
    ro, rl = oracle_mod.fwd(*(t.numpy() for t in (q, k, v, u, w)), 0.2)
    assert torch.allclose(o, torch.from_numpy(ro), atol=1e-12)
    assert torch.allclose(lse, torch.from_numpy(rl), atol=1e-12)
    # the last query of a causal call sees everything, the first of nine one token
    oc, lc, _, _ = ref.attention(q, u, k, v, w, [9, 9], 0.2, True)
    assert torch.allclose(oc[:, :, -1], o[:, :, -1], atol=1e-12)
    assert torch.allclose(oc[:, :, 0], v[:, :, 0], atol=1e-12)
