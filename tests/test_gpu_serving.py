"""Serving operators on the GPU against the 64-bit definitions in
_serving_ref.py: rotary positions, the 8-bit cache's append, attention and
eviction, and all of them as a decoding loop uses them."""
import math

import pytest
import torch

from tests import _serving_ref as ref

pytestmark = pytest.mark.gpu
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------- rotary
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hk,N,d,rot,dtype,strided", [
    (1, 1, 1, 1, 64, 64, torch.bfloat16, False),
    (3, 4, 2, 7, 64, 32, torch.bfloat16, True),
    (2, 6, 1, 130, 128, 128, torch.float16, True),
    (2, 3, 3, 65, 32, 16, torch.float32, False),
    (2, 2, 1, 9, 64, 20, torch.bfloat16, False),      # pairs that fill no vector
    (1, 3, 1, 5, 40, 40, torch.float16, True),
    (1, 2, 2, 6, 33, 6, torch.float32, False),        # rows that are not 16-byte units
    (2, 2, 1, 4, 64, 0, torch.bfloat16, False),       # nothing turns
    (1, 40, 8, 2000, 64, 64, torch.bfloat16, False),  # many heads a thread
])
def test_rotary(rfb_lib, cuda_dev, layout, B, H, Hk, N, d, rot, dtype, strided):
    g = gen(7 * d + rot)

    def x(h):
        t = torch.randn(B, N, h, d, generator=g) if strided else torch.randn(B, h, N, d, generator=g)
        t = t.to(dtype).to(cuda_dev)
        return t.transpose(1, 2) if strided else t
    q, k = x(H), x(Hk)
    pos = torch.randint(-50, 2000000, (B, N), generator=g, dtype=torch.int32)
    pos.view(-1)[0] = 2 ** 31 - 1
    freqs, amp = rfb_lib.rotary_frequencies(rot, scaling="by_parts", factor=2.0,
                                            original_length=1000)
    qo, ko = rfb_lib.rotary_fwd(q, k, pos.to(cuda_dev), freqs.to(cuda_dev), layout=layout,
                                amplitude=amp)
    gq, gk = rfb_lib.rotary_bwd(q, k, pos.to(cuda_dev), freqs.to(cuda_dev), layout=layout,
                                amplitude=amp)
    for name, got, src, inv in (("q", qo, q, False), ("k", ko, k, False), ("dq", gq, q, True),
                                ("dk", gk, k, True)):
        want, room = ref.rotary(src, pos, freqs, layout, amp, inverse=inv)
        assert got.is_contiguous() and got.dtype == dtype
        ref.assert_within(name, got, want, room + want.abs() * ref.HALF_STEP[dtype] + 1e-7)
        if rot < d:
            assert torch.equal(got[..., rot:], src[..., rot:])


def test_rotary_shared_positions_and_single_tensor(rfb_lib, cuda_dev):
    q = torch.randn(3, 2, 5, 64, generator=gen(3)).bfloat16().to(cuda_dev)
    f, _ = rfb_lib.rotary_frequencies(64, device=cuda_dev)
    p = torch.arange(5, dtype=torch.int32, device=cuda_dev)
    one, none = rfb_lib.rotary_fwd(q, None, p, f)
    both, _ = rfb_lib.rotary_fwd(q, q, p.expand(3, 5).contiguous(), f)
    assert none is None and torch.equal(one, both)
    out = torch.empty_like(q)
    assert rfb_lib.rotary_fwd(q, None, p, f, q_out=out)[0] is out and torch.equal(out, one)
    # a row whose start is not 16-byte aligned takes the narrow copies
    wide = torch.zeros(3, 2, 5, 66, dtype=torch.bfloat16, device=cuda_dev)
    wide[..., 1:65] = q
    assert torch.equal(rfb_lib.rotary_fwd(wide[..., 1:65], None, p, f)[0], one)
    assert rfb_lib.rotary_fwd(q[:0], None, p, f)[0].shape == (0, 2, 5, 64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient(rfb_lib, cuda_dev, layout):
    """The autograd wrapper against differences of the 64-bit definition (the
    rotation is linear, so a difference quotient is exact up to rounding)."""
    g = gen(11)
    q = torch.randn(2, 3, 4, 32, generator=g)
    k = torch.randn(2, 1, 4, 32, generator=g)
    dq, dk = torch.randn(2, 3, 4, 32, generator=g), torch.randn(2, 1, 4, 32, generator=g)
    pos = torch.tensor([[0, 1, 5, 900000]] * 2, dtype=torch.int32)
    f, _ = rfb_lib.rotary_frequencies(16)
    qg, kg = q.to(cuda_dev).requires_grad_(), k.to(cuda_dev).requires_grad_()
    qo, ko = rfb_lib.rfb_rotary(qg, kg, pos.to(cuda_dev), f.to(cuda_dev), layout, 1.25)
    # gradients that are expanded or transposed views
    got = torch.autograd.grad([qo, ko], [qg, kg], [dq.to(cuda_dev), dk.to(cuda_dev)],
                              retain_graph=True)
    for got_x, x, dy in ((got[0], q, dq), (got[1], k, dk)):
        want = torch.zeros_like(x, dtype=torch.float64)
        flat = want.view(-1)
        for e in range(0, x.numel(), 7):
            step = torch.zeros(x.numel(), dtype=torch.float64)
            step[e] = 1.0
            d, _ = ref.rotary(step.view_as(x), pos, f, layout, 1.25)
            flat[e] = (d * dy.double()).sum()
        sel = torch.arange(0, x.numel(), 7)
        diff = (got_x.cpu().double().view(-1)[sel] - flat[sel]).abs()
        # two terms of at most 1.25 * 4.5 each, sines 2^-22 off, one fp32 rounding
        assert float(diff.max()) <= 2 * 1.25 * 4.5 * 2.0 ** -21
    ones = torch.ones(1, device=cuda_dev).expand(2, 3, 4, 32)
    a = torch.autograd.grad(qo, qg, ones, retain_graph=True)[0]
    b = torch.autograd.grad(qo, qg, ones.contiguous())[0]
    assert torch.equal(a, b)


def test_rotary_single_tensor_and_second_order(rfb_lib, cuda_dev):
    """k None, one output unused, and a gradient of a gradient (the rotation
    is linear: it is the rotation of what the gradient is multiplied with)."""
    g = gen(13)
    q, w = (torch.randn(1, 2, 3, 16, generator=g).to(cuda_dev).requires_grad_() for _ in range(2))
    pos, (f, _) = ints([4, 0, 9], cuda_dev), rfb_lib.rotary_frequencies(16, device=cuda_dev)
    y, none = rfb_lib.rfb_rotary(q, None, pos, f)
    assert none is None
    gq, = torch.autograd.grad(y, q, w, create_graph=True)
    z = torch.randn(1, 2, 3, 16, generator=g).to(cuda_dev)
    gw, = torch.autograd.grad(gq, w, z)
    assert torch.equal(gw, rfb_lib.rotary_fwd(z, None, pos, f)[0])
    a, b = rfb_lib.rfb_rotary(q, w, pos, f)
    ga, gb = torch.autograd.grad(b, (q, w), z)
    assert bool((ga == 0).all()) and torch.equal(gb, rfb_lib.rotary_bwd(z, None, pos, f)[0])


def test_rotary_before_attention_trains(rfb_lib, cuda_dev):
    """rfb_rotary feeds rfb_attention: the gradients reach the unrotated
    operands and are the inverse turn of the attention's own."""
    g = gen(12)
    q, k, v = (torch.randn(1, 2, 150, 32, generator=g).bfloat16().to(cuda_dev).requires_grad_()
               for _ in range(3))
    u, w = (torch.randn(1, 2, 150, 8, generator=g).bfloat16().to(cuda_dev) for _ in range(2))
    f, _ = rfb_lib.rotary_frequencies(32, device=cuda_dev)
    pos = torch.arange(150, dtype=torch.int32, device=cuda_dev)
    qr, kr = rfb_lib.rfb_rotary(q, k, pos, f)
    o = rfb_lib.rfb_attention(qr, kr, v, u, w)
    dout = torch.randn(o.shape, generator=g).bfloat16().to(cuda_dev)
    gq, gk, gv = torch.autograd.grad(o, (q, k, v), dout)
    qd, kd = qr.detach(), kr.detach()
    oo, lse = rfb_lib.attn_fwd(qd, kd, v.detach(), u, w)
    dq, dk, dv, _, _ = rfb_lib.attn_bwd(qd, kd, v.detach(), u, w, oo, lse, dout)
    iq, ik = rfb_lib.rotary_bwd(dq, dk, pos, f)
    assert torch.equal(oo, o)
    # the backward adds dQ in an order of its own: equal but for bf16 steps
    for a, b in ((gq, iq), (gk, ik), (gv, dv)):
        assert float((a.double() - b.double()).norm() / b.double().norm()) <= 2.0 ** -8


# -------------------------------------------------------------------- cache
def filled(rfb, dev, B, Hk, cap, d, r, seed, spread=0.0, mass=False):
    """A cache with random codes and scales; `spread` widens the scales (powers of two)."""
    g = gen(seed)
    c = rfb.Cache8.create(B, Hk, cap, d, r, mass=mass, device=dev)
    refs = {}
    for name in ("k", "v", "w"):
        codes, scales = getattr(c, name), getattr(c, name + "_scale")
        if codes is None:
            continue
        x = torch.randn(codes.shape, generator=g)
        e = torch.round(torch.randn(scales.shape, generator=g) * spread) - 6
        codes.copy_((x * 64).to(ref.E4M3))
        scales.copy_(torch.exp2(e))
        refs[name] = ref.Ref(codes, scales)
    if mass:
        c.mass.copy_(torch.rand(c.mass.shape, generator=g) ** 8)
    return c, refs


def check_cache(cache, refs, what=""):
    for name, rf in refs.items():
        got = getattr(cache, name).cpu().double()
        nan = torch.isnan(rf.c)
        assert torch.equal(torch.isnan(got), nan), f"{what} {name}: NaN codes differ"
        assert torch.equal(got[~nan], rf.c[~nan]), f"{what} {name}: codes differ"
        assert torch.equal(getattr(cache, name + "_scale").cpu().double(), rf.s), f"{what} {name} scales"


@pytest.mark.parametrize("d,r", [(32, 0), (64, 8), (128, 40), (64, 64), (32, 24)])
@pytest.mark.parametrize("n,starts,counts", [
    (1, [0, 31, 32, 63, 64, 95], None),
    (1, [5, 96, 97, 1000, -3, 2 ** 31 - 1], [1, 1, 1, 1, 1, 1]),     # at, behind the capacity
    (33, [0, 1, 31, 32, 60, 90], [33, 33, 2, 0, 33, 33]),
    (70, [0, 13, 64, 95, 32, 3], [70, 69, 64, 1, 200, -5]),
])
def test_append(rfb_lib, cuda_dev, d, r, n, starts, counts):
    B, Hk, cap = 6, 2, 96
    cache, refs = filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=d + r + n, spread=3.0, mass=True)
    mass = cache.mass.cpu().clone()
    g = gen(n)

    def rows(c):  # as a projection leaves them
        x = torch.randn(B, n, Hk, c, generator=g) * torch.exp2(torch.randint(-9, 6, (B, 1, Hk, 1),
                                                                          generator=g).float())
        return x.bfloat16()
    new = {"k": rows(d), "v": rows(d), "w": rows(r) if r else None}
    dev = {m: None if x is None else x.to(cuda_dev).transpose(1, 2) for m, x in new.items()}
    s, c = ints(starts, cuda_dev), None if counts is None else ints(counts, cuda_dev)
    for turn in range(2):  # the same rows again change nothing
        rfb_lib.cache_append(cache, dev["k"], dev["v"], dev["w"], start=s, counts=c)
        if turn == 0:
            cs = [n] * B if counts is None else [max(0, min(x, n)) for x in counts]
            for name, rf in refs.items():
                rf.append(new[name].transpose(1, 2), starts, cs)
            for b in range(B):
                lo = min(max(starts[b], 0), cap)
                mass[b, :, lo: min(lo + cs[b], cap)] = 0.0
        check_cache(cache, refs, f"turn {turn}")
        assert torch.equal(cache.mass.cpu(), mass)


def test_append_grows_a_block_token_by_token(rfb_lib, cuda_dev):
    """Rising magnitudes: each growth requantises what the block holds."""
    cache, refs = filled(rfb_lib, cuda_dev, 1, 1, 64, 64, 8, seed=5)
    g = gen(6)
    for t in range(40):
        x = {m: (torch.randn(1, 1, 1, c, generator=g) * 2.0 ** (t - 20)).bfloat16()
             for m, c in (("k", 64), ("v", 64), ("w", 8))}
        rfb_lib.cache_append(cache, *(x[m].to(cuda_dev) for m in "kvw"), start=ints([t], cuda_dev))
        for m, rf in refs.items():
            rf.append(x[m], [t], [1])
    check_cache(cache, refs)


def test_append_non_finite_and_extreme(rfb_lib, cuda_dev):
    """Infinities become the largest code, NaN stays NaN, neither sets the
    scale; zeros and values beyond the scales' range are held at their ends."""
    cache, refs = filled(rfb_lib, cuda_dev, 4, 1, 32, 64, 0, seed=8)
    x = torch.randn(4, 1, 3, 64, generator=gen(9)).bfloat16()
    x[0, 0, 1, 3], x[0, 0, 1, 4], x[0, 0, 2, 5] = float("inf"), float("-inf"), NAN
    x[1] = 0.0
    x[2, 0, 0, 0], x[2, 0, 1, 1] = 3.0e38, -3.0e38
    x[3] *= 2.0 ** -60
    rfb_lib.cache_append(cache, x.to(cuda_dev), x.to(cuda_dev), start=ints([0, 0, 7, 0], cuda_dev))
    for rf in refs.values():
        rf.append(x, [0, 0, 7, 0], [3] * 4)
    check_cache(cache, refs)
    assert float(cache.k[0, 0, 1, 3].float()) == 448.0 and math.isnan(float(cache.k[0, 0, 2, 5].float()))
    assert float(cache.k_scale[1, 0, 0]) == 2.0 ** -40


# ---------------------------------------------------------------- attention
def run_attn(rfb, dev, cache, refs, lengths, H, Nq, *, causal=True, scale=None, seed=0, mass=None,
             decay=1.0, q=None, u=None):
    g = gen(seed + 100)
    B, d, r = cache.B, cache.d, cache.r
    q = torch.randn(B, H, Nq, d, generator=g).bfloat16() if q is None else q
    if r and u is None:
        u = (torch.randn(B, H, Nq, r, generator=g) * r ** -0.5).bfloat16()
    s = d ** -0.5 if scale is None else scale
    kw = {}
    if mass is not None:
        kw = dict(mass=mass, mass_out=torch.full_like(mass, 123.0), decay=decay)
    o, lse = rfb.attn_fwd_cache(q.to(dev), u.to(dev) if r else None, cache, ints(lengths, dev), s,
                                causal=causal, **kw)
    v = {m: rf.values() for m, rf in refs.items()}
    ro, rl, rm, room = ref.attention(q, u if r else None, v["k"], v["v"], v.get("w"), lengths, s, causal,
                                     None if mass is None else mass, decay)
    ref.assert_within("o", o, ro, room[0])
    ref.assert_within("lse", lse, rl, room[1])
    if mass is not None:
        got = kw["mass_out"].cpu()
        for b, L in enumerate(lengths):
            L = min(max(L, 0), cache.cap)
            ref.assert_within("mass", got[b, :, :L], rm[b, :, :L], room[2][b, :, :L])
            assert bool((got[b, :, L:] == 123.0).all()), "mass behind the sequence was written"
    return o, lse


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("r", [0, 8, 16, 24, 40, 64])
def test_attention_channels_and_ranks(rfb_lib, cuda_dev, d, r):
    lengths = [0, 1, 2, 31, 32, 33, 63, 64, 95, 96]
    cache, refs = filled(rfb_lib, cuda_dev, len(lengths), 2, 96, d, r, seed=d * 100 + r)
    run_attn(rfb_lib, cuda_dev, cache, refs, lengths, 6, 1, mass=torch.rand(
        cache.B, 2, 96, generator=gen(1)).to(cuda_dev), seed=r)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk,Nq", [(1, 1, 1), (5, 1, 3), (8, 2, 4), (3, 3, 16), (4, 1, 17), (8, 4, 33),
                                     (16, 1, 5), (2, 1, 70)])
def test_attention_row_tiles(rfb_lib, cuda_dev, causal, H, Hk, Nq):
    """Row counts within, at and across the 16- and 64-row tiles; sequences
    shorter than the queries leave rows that see nothing."""
    lengths = [0, 3, 40, 200, 129, 16]
    cache, refs = filled(rfb_lib, cuda_dev, len(lengths), Hk, 224, 64, 16, seed=H + Nq)
    mass = torch.rand(cache.B, Hk, 224, generator=gen(2)).to(cuda_dev)
    o, lse = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, H, Nq, causal=causal, mass=mass, decay=0.75)
    assert bool((o[0] == 0).all()) and bool((lse[0] == float("-inf")).all())
    if causal and Nq > 3:
        assert bool((o[1, :, : Nq - 3] == 0).all()) and bool((lse[1, :, : Nq - 3] == float("-inf")).all())


@pytest.mark.parametrize("B,Hk,G,cap,top", [(1, 1, 1, 8192, 8191), (3, 2, 4, 4096, 4096),
                                            (40, 4, 1, 512, 500), (2, 8, 8, 2048, 2047)])
def test_attention_splits(rfb_lib, cuda_dev, B, Hk, G, cap, top):
    """Segments cut over many CTAs, and many segments a CTA."""
    lengths = [max(0, top - (top * b) // B) for b in range(B)]
    cache, refs = filled(rfb_lib, cuda_dev, B, Hk, cap, 64, 8, seed=B + cap)
    a = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, Hk * G, 1, seed=B)
    b = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, Hk * G, 1, seed=B)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the order of joins is fixed


@pytest.mark.parametrize("d,r", [(32, 0), (32, 16), (32, 32), (32, 64), (64, 0), (64, 16), (64, 32),
                                 (64, 64), (128, 0), (128, 16), (128, 32), (128, 64)])
@pytest.mark.parametrize("B,Hk,H,Nq,cap,lengths", [
    (3, 2, 4, 9, 512, [512, 77, 5]),          # few partials a segment, one of a single CTA
    (2, 1, 4, 40, 1024, [1000, 640]),         # the same, three row segments
    (1, 1, 2, 9, 2048, [2011]),               # many partials a segment
    (1, 1, 3, 50, 4096, [4095])])             # the same, three row segments
def test_attention_joins_of_many_rows(rfb_lib, cuda_dev, d, r, B, Hk, H, Nq, cap, lengths):
    """More than 8 rows a key head with weights kept, which need the joined LSE of every row."""
    cache, refs = filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=cap + r)
    mass = torch.rand(B, Hk, cap, generator=gen(3)).to(cuda_dev)
    a = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, H, Nq, mass=mass, decay=0.5, seed=r)
    b = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, H, Nq, mass=mass, decay=0.5, seed=r)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,r", [(32, 0), (32, 40), (64, 8), (64, 64), (128, 0), (128, 32)])
@pytest.mark.parametrize("B,Hk,H,Nq,cap,keep_mass", [
    (5, 2, 6, 1, 512, False),       # short contexts, some empty
    (5, 1, 4, 5, 256, False),       # 20 rows
    (4, 1, 2, 70, 128, False),      # several row segments, rows that see nothing
    (4, 1, 2, 70, 32, True),        # the same, one block
    (5, 2, 6, 1, 128, True),
    (130, 4, 4, 1, 160, True),      # more segments than CTAs at once
    (120, 4, 4, 1, 736, False)])    # the same, several blocks a warp
def test_attention_of_whole_segments(rfb_lib, cuda_dev, d, r, B, Hk, H, Nq, cap, keep_mass):
    """Segments that one CTA holds whole, without a join: every length of interest, none among them."""
    lengths = [(0, 1, cap, cap - 33, 31, cap // 2 + 1, 40)[b % 7] for b in range(B)]
    lengths = [max(0, min(n, cap)) for n in lengths]
    cache, refs = filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=cap + r)
    mass = torch.rand(B, Hk, cap, generator=gen(4)).to(cuda_dev) if keep_mass else None
    o, lse = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, H, Nq, mass=mass, seed=d)
    assert bool((o[0] == 0).all()) and bool((lse[0] == float("-inf")).all())
    size = rfb_lib.attn_cache_workspace_size(cache, H, Nq, keep_mass)
    ws = torch.empty(size + 64, dtype=torch.uint8, device=cuda_dev)[:size]
    q = torch.randn(B, H, Nq, d, generator=gen(5)).bfloat16().to(cuda_dev)
    u = torch.randn(B, H, Nq, r, generator=gen(6)).bfloat16().to(cuda_dev) if r else None
    L, out = ints(lengths, cuda_dev), torch.full_like(mass, 3.0) if keep_mass else None
    a = rfb_lib.attn_fwd_cache(q, u, cache, L, mass_out=out, workspace=ws)   # the size is enough
    b = rfb_lib.attn_fwd_cache(q, u, cache, L, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [32, 64, 128])
def test_attention_scales_far_apart(rfb_lib, cuda_dev, d):
    """Blocks whose scales differ by many powers of two, one of zeros."""
    cache, refs = filled(rfb_lib, cuda_dev, 2, 2, 256, d, 16, seed=31, spread=5.0)
    cache.v[:, :, 64:96] = torch.zeros((), dtype=torch.uint8, device=cuda_dev).view(ref.E4M3)
    cache.v_scale[:, :, 2] = 2.0 ** -40
    cache.v_scale[1, :, 4] = 2.0 ** 40
    cache.k_scale.clamp_(max=2.0 ** -5)
    refs = {m: ref.Ref(getattr(cache, m), getattr(cache, m + "_scale")) for m in "kvw"}
    run_attn(rfb_lib, cuda_dev, cache, refs, [256, 250], 4, 2, seed=3)


def test_attention_extreme_queries(rfb_lib, cuda_dev):
    """Rows of zeros, of tiny and of large queries; scores of +-300."""
    cache, refs = filled(rfb_lib, cuda_dev, 1, 1, 128, 64, 8, seed=41)
    q = torch.randn(1, 6, 1, 64, generator=gen(42))
    q[0, 0] = 0.0
    q[0, 1] *= 2.0 ** -70
    q[0, 2] *= 40.0
    q[0, 3, 0, 7] = 3000.0
    q[0, 4] *= 2.0 ** -30
    q[0, 4, 0, 0] = 1.0
    u = torch.randn(1, 6, 1, 8, generator=gen(43))
    u[0, 5] *= 30.0
    u[0, 0] = 0.0
    run_attn(rfb_lib, cuda_dev, cache, refs, [100], 6, 1, q=q.bfloat16(), u=u.bfloat16())


def test_attention_ignores_what_lies_behind(rfb_lib, cuda_dev):
    """NaN codes and scales behind the sequence change nothing."""
    lengths = [1, 30, 32, 33, 64, 77]
    cache, refs = filled(rfb_lib, cuda_dev, 6, 2, 128, 64, 8, seed=51)
    a = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, 4, 2, seed=5)
    bad = torch.full((), 0x7f, dtype=torch.uint8, device=cuda_dev).view(ref.E4M3)
    for b, L in enumerate(lengths):
        for t in (cache.k, cache.v, cache.w):
            t[b, :, L:] = bad
        for s in (cache.k_scale, cache.v_scale, cache.w_scale):
            s[b, :, (L + 31) // 32:] = NAN
    b = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, 4, 2, seed=5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("where", ["k", "v"])
def test_attention_nan_token_reaches_only_rows_that_see_it(rfb_lib, cuda_dev, where):
    """A NaN in a token that causal queries before it do not see."""
    cache, refs = filled(rfb_lib, cuda_dev, 1, 1, 96, 64, 0, seed=61)
    bad = torch.full((), 0x7f, dtype=torch.uint8, device=cuda_dev).view(ref.E4M3)
    getattr(cache, where)[0, 0, 70, 5] = bad
    refs = {m: ref.Ref(getattr(cache, m), getattr(cache, m + "_scale")) for m in "kv"}
    o, lse = run_attn(rfb_lib, cuda_dev, cache, refs, [75], 2, 12, seed=6)
    sees = torch.arange(12) >= 12 - (75 - 70)
    if where == "v":
        assert torch.equal(torch.isnan(o[0, 0, :, 5]).cpu(), sees)
        assert not bool(torch.isnan(o[0, 0, :, 6]).any())
    else:
        assert torch.equal(torch.isnan(lse[0, 1]).cpu(), sees)


def test_attention_mass_in_place_and_alone(rfb_lib, cuda_dev):
    cache, refs = filled(rfb_lib, cuda_dev, 2, 2, 160, 32, 0, seed=71, mass=True)
    q = torch.randn(2, 4, 3, 32, generator=gen(72)).bfloat16().to(cuda_dev)
    L = ints([150, 7], cuda_dev)
    start = cache.mass.clone()
    fresh = torch.full_like(start, 9.0)
    rfb_lib.attn_fwd_cache(q, None, cache, L, mass_out=fresh)          # mass None: zeros
    other = torch.full_like(start, 9.0)
    rfb_lib.attn_fwd_cache(q, None, cache, L, mass=start, mass_out=other, decay=0.5)
    rfb_lib.attn_fwd_cache(q, None, cache, L, mass=cache.mass, mass_out=cache.mass, decay=0.5)
    for b, n in ((0, 150), (1, 7)):
        assert torch.equal(cache.mass[b, :, :n], other[b, :, :n])
        assert torch.equal(cache.mass[b, :, n:], start[b, :, n:])
        # 6 query rows a key head, each with weights that add to 1 if it sees a token
        rows = 2 * min(3, n)
        assert torch.allclose(fresh[b, :, :n].sum(-1).cpu(), torch.full((2,), float(rows)), atol=1e-4)


# ----------------------------------------------------------------- eviction
def check_evict(rfb, dev, cache, refs, lengths, keep, recent, in_place):
    mass = cache.mass.cpu().clone()
    kept_ref, n_ref, blocks = ref.evict(refs, mass, lengths, keep, recent)
    before = {m: (getattr(cache, m).cpu().view(torch.uint8).clone(),
                  getattr(cache, m + "_scale").cpu().clone()) for m in refs}
    if in_place:
        to, back = cache, before
        mass_back = mass
    else:
        to = rfb.Cache8.create(cache.B, cache.Hk, keep + 40, cache.d, cache.r, mass=True, device=dev)
        for m in refs:
            getattr(to, m).copy_(torch.full((), 448.0).to(ref.E4M3))
        to.mass.fill_(77.0)
        back = {m: (getattr(to, m).cpu().view(torch.uint8).clone(),
                    getattr(to, m + "_scale").cpu().clone()) for m in refs}
        mass_back = to.mass.cpu().clone()
    n, kept = rfb.cache_evict(cache, ints(lengths, dev), keep, recent, out=None if in_place else to)
    assert torch.equal(n.cpu().long(), n_ref)
    assert torch.equal(kept.cpu().long(), kept_ref)
    got_mass = to.mass.cpu()
    for b in range(cache.B):
        m = int(n_ref[b])
        for h in range(cache.Hk):
            idx = kept_ref[b, h, :m]
            want = mass[b, h, idx]
            same = (got_mass[b, h, :m] == want) | (torch.isnan(got_mass[b, h, :m]) & torch.isnan(want))
            assert bool(same.all())
            assert torch.equal(got_mass[b, h, m:].nan_to_num(5.0), mass_back[b, h, m:].nan_to_num(5.0))
    for name in refs:
        codes, scales = getattr(to, name).cpu(), getattr(to, name + "_scale").cpu()
        for (b, h, j), (c, s) in blocks[name].items():
            rows = codes[b, h, j * 32: j * 32 + c.shape[0]].double()
            nan = torch.isnan(c)
            assert torch.equal(torch.isnan(rows), nan) and torch.equal(rows[~nan], c[~nan]), (name, b, h, j)
            assert float(scales[b, h, j]) == s, (name, b, h, j)
        for b in range(cache.B):
            m = int(n_ref[b])
            assert torch.equal(codes.view(torch.uint8)[b, :, m:], back[name][0][b, :, m:])
            nb = (m + 31) // 32
            assert torch.equal(scales[b, :, nb:], back[name][1][b, :, nb:])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("d,r", [(32, 0), (64, 8), (128, 24), (64, 64)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (33, 5), (64, 64), (200, 0), (288, 300)])
def test_evict(rfb_lib, cuda_dev, in_place, d, r, keep, recent):
    lengths = [0, 1, 32, 33, 64, 287, 288, 150]
    cache, refs = filled(rfb_lib, cuda_dev, len(lengths), 2, 288, d, r, seed=keep + d, spread=4.0,
                         mass=True)
    cache.mass[:, 1] = torch.round(cache.mass[:, 1] * 4)       # ties
    check_evict(rfb_lib, cuda_dev, cache, refs, lengths, keep, recent, in_place)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_long(rfb_lib, cuda_dev, in_place):
    """More rounds than one, lengths that do not fill the compaction's stretches."""
    cache, refs = filled(rfb_lib, cuda_dev, 3, 1, 5024, 64, 8, seed=81, spread=1.0, mass=True)
    cache.mass[1, 0, :4000] = 0.25
    check_evict(rfb_lib, cuda_dev, cache, refs, [5023, 4999, 1300], 2500, 100, in_place)


def test_evict_odd_masses(rfb_lib, cuda_dev):
    """Infinities, NaN, negative masses, both zeros, and NaN codes among the tokens."""
    cache, refs = filled(rfb_lib, cuda_dev, 2, 1, 64, 32, 0, seed=91, spread=2.0, mass=True)
    m = cache.mass
    m[0, 0, 3], m[0, 0, 5], m[0, 0, 9], m[0, 0, 10] = float("inf"), NAN, float("-inf"), -2.0
    m[0, 0, 20:30], m[0, 0, 30:40] = 0.0, -0.0
    m[1] = NAN
    cache.k.view(torch.uint8)[0, 0, 3, 4] = 0x7f
    refs = {n: ref.Ref(getattr(cache, n), getattr(cache, n + "_scale")) for n in "kv"}
    check_evict(rfb_lib, cuda_dev, cache, refs, [60, 50], 40, 3, True)


# ------------------------------------------------------ together, streams, graphs
def test_decode_loop(rfb_lib, cuda_dev):
    """A prompt, then single tokens with rotary positions, factors and masses,
    an eviction on the way: every step against the definitions on the cache's
    own values, which follow the definitions exactly."""
    B, H, Hk, d, r, cap = 3, 4, 2, 64, 8, 128
    g = gen(101)
    cache = rfb_lib.Cache8.create(B, Hk, cap, d, r, mass=True, device=cuda_dev)
    refs = {m: ref.Ref(getattr(cache, m), getattr(cache, m + "_scale")) for m in "kvw"}
    f, _ = rfb_lib.rotary_frequencies(d, device=cuda_dev)
    lengths, pos = [0] * B, [0] * B
    mass = torch.zeros(B, Hk, cap, dtype=torch.float64)
    # the kernel's masses follow the definition within the rooms of all steps so far
    room_m = torch.zeros_like(mass)
    for step, counts in enumerate([[50, 17, 32]] + [[1, 1, 1]] * 12 + [[4, 4, 4]] + [[1, 1, 1]] * 3):
        n = max(counts)
        q = torch.randn(B, n, H, d, generator=g).bfloat16().to(cuda_dev).transpose(1, 2)
        k = torch.randn(B, n, Hk, d, generator=g).bfloat16().to(cuda_dev).transpose(1, 2)
        v = torch.randn(B, n, Hk, d, generator=g).bfloat16().to(cuda_dev).transpose(1, 2)
        w = (torch.randn(B, n, Hk, r, generator=g) * 0.3).bfloat16().to(cuda_dev).transpose(1, 2)
        u = (torch.randn(B, H, n, r, generator=g) * 0.3).bfloat16().to(cuda_dev)
        at = ints([[p + i for i in range(n)] for p in pos], cuda_dev)
        qr, kr = rfb_lib.rotary_fwd(q, k, at, f)
        rfb_lib.cache_append(cache, kr, v, w, start=ints(lengths, cuda_dev), counts=ints(counts, cuda_dev))
        for m, x in (("k", kr), ("v", v), ("w", w)):
            refs[m].append(x, lengths, counts)
        check_cache(cache, refs, f"step {step}")
        for b in range(B):
            mass[b, :, lengths[b]: lengths[b] + counts[b]] = 0.0
            room_m[b, :, lengths[b]: lengths[b] + counts[b]] = 0.0
        lengths = [a + c for a, c in zip(lengths, counts)]
        pos = [a + c for a, c in zip(pos, counts)]
        if step == 0:
            continue  # a padded prompt: its attention is the framework's full forward
        o, lse = rfb_lib.attn_fwd_cache(qr, u, cache, ints(lengths, cuda_dev), mass=cache.mass,
                                        mass_out=cache.mass)
        val = {m: rf.values() for m, rf in refs.items()}
        ro, rl, mass, room = ref.attention(qr, u, val["k"], val["v"], val["w"], lengths, d ** -0.5,
                                           True, mass)
        room_m = room_m + room[2]
        ref.assert_within("o", o, ro, room[0])
        ref.assert_within("lse", lse, rl, room[1])
        ref.assert_within("mass", cache.mass, mass, room_m)
        if step == 9:
            keep, recent = 40, 8
            kept_ref, n_ref, blocks = ref.evict(refs, cache.mass, lengths, keep, recent)
            new, kept = rfb_lib.cache_evict(cache, ints(lengths, cuda_dev), keep, recent)
            assert torch.equal(kept.cpu().long(), kept_ref) and torch.equal(new.cpu().long(), n_ref)
            lengths = new.tolist()
            refs = {m: ref.Ref(getattr(cache, m), getattr(cache, m + "_scale")) for m in "kvw"}
            for name in refs:
                for (b, h, j), (c, s) in blocks[name].items():
                    assert torch.equal(refs[name].c[b, h, j * 32: j * 32 + c.shape[0]], c)
                    assert float(refs[name].s[b, h, j]) == s
            mass, room_m = cache.mass.cpu().double(), torch.zeros_like(mass)


def step_inputs(dev, B, H, Hk, d, r, seed):
    g = gen(seed)
    x = lambda h, c: torch.randn(B, h, 1, c, generator=g).bfloat16().to(dev)  # noqa: E731
    return dict(q=x(H, d), k=x(Hk, d), v=x(Hk, d), w=x(Hk, r), u=x(H, r))


def test_captured_step_follows_its_lengths(rfb_lib, cuda_dev):
    """A step captured once and replayed with growing lengths equals eager
    steps; two graphs with workspaces of their own replayed in turn."""
    B, H, Hk, d, r, cap = 2, 4, 2, 64, 8, 96
    f, _ = rfb_lib.rotary_frequencies(d, device=cuda_dev)
    caches = [filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=111, mass=True)[0] for _ in range(4)]
    x = step_inputs(cuda_dev, B, H, Hk, d, r, 112)

    def step(c, start, lengths):
        qr, kr = rfb_lib.rotary_fwd(x["q"], x["k"], start.view(B, 1), f)
        rfb_lib.cache_append(c, kr, x["v"], x["w"], start=start)
        return rfb_lib.attn_fwd_cache(qr, x["u"], c, lengths, mass=c.mass, mass_out=c.mass)
    graphs = []
    for c in caches[:2]:
        start, lengths = ints([30, 40], cuda_dev), ints([31, 41], cuda_dev)
        spare = filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=113, mass=True)[0]
        step(spare, start, lengths)  # loads the kernels
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = step(c, start, lengths)
        graphs.append((graph, start, lengths, o, lse))
    for i in range(3):
        for z, (graph, start, lengths, o, lse) in enumerate(graphs):
            graph.replay()
            eo, el = step(caches[2 + z], start, lengths)
            assert torch.equal(o, eo) and torch.equal(lse, el)
            start += 1
            lengths += 1
        for q in x.values():
            q.mul_(1.5)
    for a, b in ((0, 2), (1, 3)):
        for name in ("k", "v", "w", "k_scale", "v_scale", "w_scale", "mass"):
            s, t = getattr(caches[a], name), getattr(caches[b], name)
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8)), name


def test_captured_rotary_backward(rfb_lib, cuda_dev):
    q = torch.randn(1, 2, 33, 64, generator=gen(121)).bfloat16().to(cuda_dev)
    f, _ = rfb_lib.rotary_frequencies(64, device=cuda_dev)
    p = torch.arange(33, dtype=torch.int32, device=cuda_dev)
    want = rfb_lib.rotary_bwd(q, None, p, f)[0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rfb_lib.rotary_bwd(q, None, p, f)[0]
    graph.replay()
    assert torch.equal(got, want)


def test_empty_cache_and_empty_calls(rfb_lib, cuda_dev):
    """A cache without capacity, calls without sequences, rows or tokens."""
    for rows in (1, 3):
        c = rfb_lib.Cache8.create(2, 2, 0, 64, 8, mass=True, device=cuda_dev)
        q = torch.randn(2, 8, rows, 64, device=cuda_dev).bfloat16()
        u = torch.randn(2, 8, rows, 8, device=cuda_dev).bfloat16()
        o, lse = rfb_lib.attn_fwd_cache(q, u, c, ints([0, 5], cuda_dev), mass_out=c.mass)
        assert bool((o == 0).all()) and bool((lse == float("-inf")).all())
        x = torch.randn(2, 2, 1, 64, device=cuda_dev).bfloat16()
        rfb_lib.cache_append(c, x, x, x[..., :8].contiguous(), start=ints([0, 0], cuda_dev))
    c, _ = filled(rfb_lib, cuda_dev, 2, 2, 64, 64, 0, seed=3)
    before = c.k.view(torch.uint8).clone()
    x = torch.randn(2, 2, 0, 64, device=cuda_dev).bfloat16()
    rfb_lib.cache_append(c, x, x, start=ints([3, 3], cuda_dev))
    o, lse = rfb_lib.attn_fwd_cache(torch.zeros(2, 4, 0, 64, device=cuda_dev).bfloat16(), None, c,
                                    ints([3, 3], cuda_dev))
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    assert torch.equal(c.k.view(torch.uint8), before)
    e = rfb_lib.Cache8.create(0, 2, 64, 64, mass=True, device=cuda_dev)
    n, kept = rfb_lib.cache_evict(e, ints([], cuda_dev), 5)
    assert n.shape == (0,) and kept.shape == (0, 2, 5)


def test_offsets_past_32_bits(rfb_lib, cuda_dev):
    """The last sequence of a cache of more than 2^32 bytes a tensor."""
    B, cap, d = 66, 524288, 128
    assert (B - 1) * cap * d > 2 ** 32
    cache = rfb_lib.Cache8.create(B, 1, cap, d, mass=True, device=cuda_dev)
    small = rfb_lib.Cache8.create(1, 1, 4096, d, mass=True, device=cuda_dev)
    g = gen(151)
    k, v = (torch.randn(1, 1, 3000, d, generator=g).bfloat16().to(cuda_dev) for _ in range(2))
    q = torch.randn(1, 3, 1, d, generator=g).bfloat16().to(cuda_dev)
    rfb_lib.cache_append(small, k, v, start=ints([0], cuda_dev))
    o, lse = rfb_lib.attn_fwd_cache(q, None, small, ints([3000], cuda_dev), mass_out=small.mass)
    counts = ints([0] * (B - 1) + [3000], cuda_dev)
    zero = torch.zeros(B, dtype=torch.int32, device=cuda_dev)
    rfb_lib.cache_append(cache, k.expand(B, 1, 3000, d), v.expand(B, 1, 3000, d), start=zero,
                         counts=counts)
    ob, lb = rfb_lib.attn_fwd_cache(q.expand(B, 3, 1, d).contiguous(), None, cache, counts,
                                    mass_out=cache.mass)
    assert bool((ob[:-1] == 0).all()) and bool((lb[:-1] == float("-inf")).all())
    # the work is cut elsewhere: O a bf16 step apart at most, LSE and mass a few fp32 steps
    assert float((ob[-1].double() - o[0].double()).abs().max()) <= 2.0 ** -7 * float(o.abs().max())
    assert torch.allclose(lb[-1], lse[0], rtol=2.0 ** -21, atol=2.0 ** -20)
    assert torch.allclose(cache.mass[-1], small.mass[0, :, :1].new_zeros(1, cap).index_copy(
        1, torch.arange(3000, device=cuda_dev), small.mass[0, :, :3000]), rtol=2.0 ** -17, atol=2.0 ** -30)
    cache.mass[-1, 0, :3000] = small.mass[0, 0, :3000]  # the same bits, so the same choice
    n, kept = rfb_lib.cache_evict(cache, counts, 1000, 100)
    ns, ks = rfb_lib.cache_evict(small, ints([3000], cuda_dev), 1000, 100)
    assert n.tolist() == [0] * (B - 1) + [1000] and torch.equal(kept[-1], ks[0])
    assert torch.equal(cache.k[-1, :, :1000].view(torch.uint8), small.k[0, :, :1000].view(torch.uint8))
    assert torch.equal(cache.v[-1, :, :1000].view(torch.uint8), small.v[0, :, :1000].view(torch.uint8))


@pytest.mark.parametrize("Nq,sites", [(1, (71,)), (20, (70, 71)), (70, (70, 71))])
def test_waits_that_give_up(rfb_lib, cuda_dev, Nq, sites):
    """A wait of the attention's copy pipeline that gives up at once: the error
    word names its site, the call ends, and the next one is right.  Then a limit
    of 1 us, under which a call ends either way."""
    cache, refs = filled(rfb_lib, cuda_dev, 3, 2, 2048, 64, 8, seed=161)
    lengths = [2000, 1999, 700]
    want = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, 4, Nq, seed=7)
    torch.cuda.synchronize()
    assert rfb_lib.last_device_error() == 0
    for limit, site in [(0, s) for s in sites] + [(1, -1)]:
        try:
            rfb_lib.debug_set_wait_limit(limit, site)
            q = torch.randn(3, 4, Nq, 64, generator=gen(8)).bfloat16().to(cuda_dev)
            u = torch.randn(3, 4, Nq, 8, generator=gen(9)).bfloat16().to(cuda_dev)
            rfb_lib.attn_fwd_cache(q, u, cache, ints(lengths, cuda_dev))
            err = rfb_lib.last_device_error()
        finally:
            rfb_lib.debug_set_wait_limit(0, -1)
        assert err == (6 | site << 8) if site >= 0 else err & 0xff in (0, 6)
        again = run_attn(rfb_lib, cuda_dev, cache, refs, lengths, 4, Nq, seed=7)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
        assert rfb_lib.last_device_error() == 0


def test_nothing_outside_the_outputs(rfb_lib, cuda_dev):
    """Every output between canaries that no kernel writes."""
    def guarded(shape, dtype):
        n = math.prod(shape)
        raw = torch.full((n + 8192,), 77.0, dtype=dtype, device=cuda_dev) if dtype != torch.uint8 else \
            torch.full((n + 8192,), 77, dtype=dtype, device=cuda_dev)
        return raw, raw[4096:4096 + n].view(shape)

    def intact(raw):
        return bool((raw[:4096] == 77).all()) and bool((raw[-4096:] == 77).all())
    for d, r, H, Hk, Nq in [(64, 24, 6, 2, 1), (32, 8, 5, 1, 7), (128, 0, 4, 4, 1), (64, 64, 8, 1, 9)]:
        lengths = [97, 1, 160, 0]
        cache, refs = filled(rfb_lib, cuda_dev, 4, Hk, 160, d, r, seed=171, mass=True)
        q = torch.randn(4, H, Nq, d, generator=gen(172)).bfloat16().to(cuda_dev)
        u = torch.randn(4, H, Nq, r, generator=gen(173)).bfloat16().to(cuda_dev) if r else None
        ro, out = guarded((4, H, Nq, d), torch.bfloat16)
        rl, lse = guarded((4, H, Nq), torch.float32)
        rm, mass = guarded((4, Hk, 160), torch.float32)
        rw, ws = guarded((rfb_lib.attn_cache_workspace_size(cache, H, Nq, True),), torch.uint8)
        L = ints(lengths, cuda_dev)
        rfb_lib.attn_fwd_cache(q, u, cache, L, mass=cache.mass, mass_out=mass, out=out, lse=lse,
                               workspace=ws)
        o, l = rfb_lib.attn_fwd_cache(q, u, cache, L)
        assert all(intact(x) for x in (ro, rl, rm, rw))
        assert torch.equal(o, out) and torch.equal(l, lse)
        rq, qo = guarded((4, H, Nq, d), torch.bfloat16)
        f, _ = rfb_lib.rotary_frequencies(d // 2 - 2, device=cuda_dev)
        rfb_lib.rotary_fwd(q, None, ints(list(range(Nq)), cuda_dev), f, q_out=qo)
        assert intact(rq)


def test_other_stream(rfb_lib, cuda_dev):
    """Calls on a stream of the caller's, with tensors of the current one, and two at once."""
    B, H, Hk, d, r = 2, 4, 2, 64, 8
    ca, _ = filled(rfb_lib, cuda_dev, B, Hk, 2048, d, r, seed=131, mass=True)
    cb, _ = filled(rfb_lib, cuda_dev, B, Hk, 2048, d, r, seed=132, mass=True)
    x = step_inputs(cuda_dev, B, H, Hk, d, r, 133)
    L = ints([2000, 1500], cuda_dev)
    want = [rfb_lib.attn_fwd_cache(x["q"], x["u"], c, L) for c in (ca, cb)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = []
        for c, s in ((ca, s1), (cb, s2)):
            got.append(rfb_lib.attn_fwd_cache(x["q"], x["u"], c, L, stream=s))
        s1.synchronize()
        s2.synchronize()
        for (a, b), (o, lse) in zip(want, got):
            assert torch.equal(a, o) and torch.equal(b, lse)


def test_refusals(rfb_lib, cuda_dev):
    rfb = rfb_lib
    cache, _ = filled(rfb, cuda_dev, 2, 2, 64, 64, 8, seed=141, mass=True)
    bare, _ = filled(rfb, cuda_dev, 2, 2, 64, 64, 0, seed=142)
    x = step_inputs(cuda_dev, 2, 4, 2, 64, 8, 143)
    L = ints([3, 4], cuda_dev)
    f, _ = rfb.rotary_frequencies(64, device=cuda_dev)
    pos = ints([0], cuda_dev)
    cases = [
        (ValueError, "multiple of the cache", lambda: rfb.attn_fwd_cache(
            x["q"][:, :3].contiguous(), x["u"][:, :3].contiguous(), cache, L)),
        (ValueError, "contiguous", lambda: rfb.attn_fwd_cache(
            x["q"].transpose(0, 1).contiguous().transpose(0, 1), x["u"], cache, L)),
        (TypeError, "bfloat16", lambda: rfb.attn_fwd_cache(x["q"].float(), x["u"], cache, L)),
        (TypeError, "Tensor", lambda: rfb.attn_fwd_cache(x["q"], None, cache, L)),
        (ValueError, "no factors", lambda: rfb.attn_fwd_cache(x["q"], x["u"], bare, L)),
        (TypeError, "int32", lambda: rfb.attn_fwd_cache(x["q"], x["u"], cache, L.long())),
        (ValueError, "shape", lambda: rfb.attn_fwd_cache(x["q"], x["u"], cache, L[:1])),
        (ValueError, "mass_out", lambda: rfb.attn_fwd_cache(x["q"], x["u"], cache, L, mass=cache.mass)),
        (RuntimeError, "workspace", lambda: rfb.attn_fwd_cache(
            x["q"], x["u"], cache, L, workspace=torch.empty(16, dtype=torch.uint8, device=cuda_dev))),
        (RuntimeError, "status 1", lambda: rfb.attn_fwd_cache(x["q"], x["u"], cache, L, scale=0.0)),
        (ValueError, "shape", lambda: rfb.cache_append(cache, x["k"], x["v"][:, :1], x["w"], start=L)),
        (TypeError, "Tensor", lambda: rfb.cache_append(cache, x["k"], x["v"], start=L)),
        (ValueError, "no factors", lambda: rfb.cache_append(bare, x["k"], x["v"], x["w"], start=L)),
        (ValueError, "strides", lambda: rfb.cache_append(
            cache, torch.zeros(2, 2, 1, 66, device=cuda_dev).bfloat16()[..., :64], x["v"], x["w"], start=L)),
        (ValueError, "with mass", lambda: rfb.cache_evict(bare, L, 4)),
        (ValueError, "keep", lambda: rfb.cache_evict(cache, L, 0)),
        (ValueError, "keep", lambda: rfb.cache_evict(cache, L, 65)),
        (ValueError, "recent", lambda: rfb.cache_evict(cache, L, 4, -1)),
        (ValueError, "layout", lambda: rfb.rotary_fwd(x["q"], x["k"], pos, f, layout="other")),
        (TypeError, "float64", lambda: rfb.rotary_fwd(x["q"], x["k"], pos, f.float())),
        (ValueError, "pairs", lambda: rfb.rotary_fwd(x["w"], None, pos, f)),
        (ValueError, "channels", lambda: rfb.rotary_fwd(
            torch.zeros(2, 4, 1, 128, device=cuda_dev).bfloat16()[..., ::2], None, pos, f)),
        (ValueError, "positions", lambda: rfb.rotary_fwd(x["q"], None, pos[0], f)),
        (TypeError, "float16", lambda: rfb.rotary_fwd(x["q"].double(), None, pos, f)),
        (ValueError, "multiple of 32", lambda: rfb.Cache8(
            cache.k[:, :, :40].contiguous(), cache.v[:, :, :40].contiguous(), None, cache.k_scale,
            cache.v_scale, None)),
        (TypeError, "float8", lambda: rfb.Cache8(cache.k.view(torch.uint8), cache.v, None, cache.k_scale,
                                                 cache.v_scale, None)),
        (ValueError, "together", lambda: rfb.Cache8(cache.k, cache.v, cache.w, cache.k_scale,
                                                    cache.v_scale, None)),
    ]
    for err, match, call in cases:
        with pytest.raises(err, match=match):
            call()
    half = rfb.Cache8.create(2, 2, 64, 64, 8, mass=True, device=cuda_dev)
    mixed = rfb.Cache8(half.k, cache.v, half.w, half.k_scale, half.v_scale, half.w_scale, half.mass)
    with pytest.raises(RuntimeError, match="status 1"):
        rfb.cache_evict(cache, L, 4, out=mixed)     # in place for some tensors only
    torch.cuda.synchronize()


@pytest.mark.parametrize("H,Nq", [(2, 0), (0, 1)])
def test_attention_without_queries_decays_the_mass(rfb_lib, cuda_dev, H, Nq):
    cache, _ = filled(rfb_lib, cuda_dev, 4, 2, 224, 64, 8, seed=191, mass=True)
    lengths = [0, 1, 200, 500]
    q = torch.empty(4, H, Nq, 64, dtype=torch.bfloat16, device=cuda_dev)
    u = torch.empty(4, H, Nq, 8, dtype=torch.bfloat16, device=cuda_dev)
    mass = torch.rand(4, 2, 224, generator=gen(192)).to(cuda_dev)
    for before, decay in ((mass, 0.5), (None, 1.0)):
        got = torch.full_like(mass, 123.0)
        o, lse = rfb_lib.attn_fwd_cache(q, u, cache, ints(lengths, cuda_dev), mass=before, mass_out=got,
                                        decay=decay)
        assert o.shape == q.shape and lse.shape == q.shape[:3]
        for b, L in enumerate([0, 1, 200, 224]):
            want = mass[b, :, :L] * 0.5 if before is not None else torch.zeros_like(mass[b, :, :L])
            assert torch.equal(got[b, :, :L], want) and bool((got[b, :, L:] == 123.0).all())


def test_shared_memory_is_refused(rfb_lib, cuda_dev):
    """Outputs that lie in the inputs' memory; in place is for the mass and for eviction."""
    x = step_inputs(cuda_dev, 1, 2, 2, 64, 8, 201)
    pos, L = ints([3], cuda_dev), ints([40], cuda_dev)
    f, _ = rfb_lib.rotary_frequencies(64, device=cuda_dev)
    cache, _ = filled(rfb_lib, cuda_dev, 1, 1, 96, 64, 8, seed=202, mass=True)
    q2 = x["q"][:, :1].contiguous()
    both = torch.zeros(2 * 96, device=cuda_dev)

    def behind(name, n):  # a cache of 64 tokens within the other's 96
        return getattr(cache, name)[:, :, n:]
    part = rfb_lib.Cache8(behind("k", 32), behind("v", 32), behind("w", 32), behind("k_scale", 1),
                          behind("v_scale", 1), behind("w_scale", 1), behind("mass", 32))
    for call in (lambda: rfb_lib.rotary_fwd(x["q"], x["k"], pos, f, q_out=x["q"]),
                 lambda: rfb_lib.rotary_fwd(x["q"], x["k"], pos, f, q_out=x["k"]),
                 lambda: rfb_lib.rotary_fwd(x["q"], x["k"], pos, f, k_out=x["k"]),
                 lambda: rfb_lib.attn_fwd_cache(q2, x["u"][:, :1].contiguous(), cache, L, out=q2),
                 lambda: rfb_lib.attn_fwd_cache(
                     q2, x["u"][:, :1].contiguous(), cache, L, mass=both[:96].view(1, 1, 96),
                     mass_out=both[32:128].view(1, 1, 96)),
                 lambda: rfb_lib.cache_evict(cache, L, 8, out=part)):
        with pytest.raises(ValueError, match="share memory"):
            call()
    same = torch.zeros(1, 1, 96, device=cuda_dev)
    rfb_lib.attn_fwd_cache(q2, x["u"][:, :1].contiguous(), cache, L, mass=same, mass_out=same)
    # halves of one buffer are apart
    pair = torch.empty(2, *x["q"].shape, dtype=torch.bfloat16, device=cuda_dev)
    pair[0] = x["q"]
    a, _ = rfb_lib.rotary_fwd(pair[0], None, pos, f, q_out=pair[1])
    b, _ = rfb_lib.rotary_fwd(x["q"], None, pos, f)
    assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_copied_cache_is_its_own(rfb_lib, cuda_dev):
    """A deep copy or a pickled cache works on its own tensors, a copy on the same."""
    import copy
    import io
    cache, _ = filled(rfb_lib, cuda_dev, 1, 2, 64, 64, 8, seed=151, mass=True)
    x = step_inputs(cuda_dev, 1, 2, 2, 64, 8, 152)
    buf = io.BytesIO()
    torch.save(cache, buf)
    buf.seek(0)
    for other in (copy.deepcopy(cache), torch.load(buf, weights_only=False)):
        before = cache.k.view(torch.uint8).clone()
        rfb_lib.cache_append(other, x["k"], x["v"], x["w"], start=ints([5], cuda_dev))
        assert torch.equal(cache.k.view(torch.uint8), before)
        assert not torch.equal(other.k.view(torch.uint8), before)
    same = copy.copy(cache)
    assert same.k is cache.k and same.mass is cache.mass
    rfb_lib.cache_append(same, x["k"], x["v"], x["w"], start=ints([5], cuda_dev))
    assert not torch.equal(cache.k.view(torch.uint8), before)


def test_replaced_mass_and_other_stream_are_checked(rfb_lib, cuda_dev):
    cache, _ = filled(rfb_lib, cuda_dev, 2, 2, 64, 64, 0, seed=161, mass=True)
    x = step_inputs(cuda_dev, 2, 2, 2, 64, 8, 162)
    L = ints([3, 4], cuda_dev)

    class Elsewhere:
        device = torch.device("cuda", 77)
    for call in (lambda: rfb_lib.cache_append(cache, x["k"], x["v"], start=L, stream=Elsewhere()),
                 lambda: rfb_lib.attn_fwd_cache(x["q"], None, cache, L, stream=Elsewhere()),
                 lambda: rfb_lib.cache_evict(cache, L, 4, stream=Elsewhere())):
        with pytest.raises(ValueError, match="stream belongs to"):
            call()
    good = cache.mass
    for bad, err in ((good[:, :1].contiguous(), ValueError), (good.double(), TypeError),
                     (good.cpu(), ValueError), (good.transpose(1, 2), ValueError), (7, TypeError)):
        cache.mass = bad
        with pytest.raises(err, match="mass"):
            rfb_lib.cache_append(cache, x["k"], x["v"], start=L)
        with pytest.raises(err, match="mass"):
            rfb_lib.cache_evict(cache, L, 4)
    cache.mass = good
    rfb_lib.cache_append(cache, x["k"], x["v"], start=L)
    with pytest.raises(TypeError):
        rfb_lib.attn_fwd_cache(x["q"], None, cache, L, "a quarter")
    with pytest.raises(TypeError, match="Tensor"):
        rfb_lib.attn_fwd_cache(x["q"], None, cache, L, out=1)
    torch.cuda.synchronize()
