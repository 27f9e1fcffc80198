"""Serving operators on the GPU, beyond test_gpu_serving.py: calls that follow
one another without a pause, sizes and values at the ends of their ranges."""
import pytest
import torch

from tests import _serving_ref as ref
from tests.test_gpu_serving import filled, gen, ints, run_attn

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.mark.parametrize("d,r,H,Hk,Nq,cap", [
    (64, 8, 2, 1, 9, 2048),        # weights beside the join
    (128, 0, 4, 1, 5, 2048),
    (32, 32, 1, 1, 70, 4096),      # two row segments, many partials: weights behind the join
    (64, 64, 2, 2, 12, 256),       # a CTA a segment: weights from the final LSE
    (64, 16, 2, 1, 3, 2048),       # up to 8 rows: weights from the scores
])
def test_weights_of_just_appended_tokens(rfb_lib, cuda_dev, d, r, H, Hk, Nq, cap):
    """Append and attention with the weights kept, step behind step without a pause:
    every kernel of a step has to see what the kernels before it wrote."""
    B, steps, g = 2, 12, gen(d + Nq)
    cache, refs = filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=d + r)
    start = [cap - steps * Nq - 37, 45]
    new = [{"k": torch.randn(B, Hk, Nq, d, generator=g).bfloat16(),
            "v": torch.randn(B, Hk, Nq, d, generator=g).bfloat16(),
            "w": torch.randn(B, Hk, Nq, r, generator=g).bfloat16() if r else None,
            "q": torch.randn(B, H, Nq, d, generator=g).bfloat16(),
            "u": (torch.randn(B, H, Nq, r, generator=g) * r ** -0.5).bfloat16() if r else None}
           for _ in range(steps)]
    dev = [{n: None if t is None else t.to(cuda_dev) for n, t in x.items()} for x in new]
    at = [ints([s + i * Nq for s in start], cuda_dev) for i in range(steps + 1)]
    outs = [torch.full((B, Hk, cap), 9.0, device=cuda_dev) for _ in range(steps)]
    torch.cuda.synchronize()
    got = []
    for i, x in enumerate(dev):
        rfb_lib.cache_append(cache, x["k"], x["v"], x["w"], start=at[i])
        got.append(rfb_lib.attn_fwd_cache(x["q"], x["u"], cache, at[i + 1], mass_out=outs[i]))
    torch.cuda.synchronize()
    for i, x in enumerate(new):
        begin = [s + i * Nq for s in start]
        lengths = [s + Nq for s in begin]
        for m, rf in refs.items():
            rf.append(x[m], begin, [Nq] * B)
        val = {m: rf.values() for m, rf in refs.items()}
        o, lse, mass, room = ref.attention(x["q"], x["u"], val["k"], val["v"], val.get("w"), lengths,
                                           d ** -0.5, True, torch.zeros(B, Hk, cap))
        ref.assert_within(f"o {i}", got[i][0], o, room[0])
        ref.assert_within(f"lse {i}", got[i][1], lse, room[1])
        for b, L in enumerate(lengths):
            ref.assert_within(f"mass {i}", outs[i][b, :, :L], mass[b, :, :L], room[2][b, :, :L])


def evicted(cache, lengths, keep, recent):
    """The definition of eviction on whole tensors: kept [B, Hk, keep], and for the kept
    tokens codes (as values), scales and masses.  Values and scales are exact in fp32."""
    m = cache.mass.double()
    B, Hk, cap = m.shape
    t = torch.arange(cap, device=m.device)
    L = lengths.long().clamp(0, cap)
    n = L.clamp(max=keep)
    rec = n.clamp(max=recent)
    older = (t < (L - rec)[:, None])[:, None].expand(B, Hk, cap)
    # descending by mass among the older, NaN behind -inf, the lowest index first
    rank = torch.where(older, torch.where(torch.isnan(m), 1, 0), 2)
    order = torch.sort(torch.nan_to_num(m, nan=0.0, posinf=float("inf"), neginf=float("-inf")),
                       dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort(rank.gather(-1, order), dim=-1, stable=True).indices)
    place = torch.empty_like(order).scatter_(-1, order, t.expand(B, Hk, cap))
    stays = (older & (place < (n - rec)[:, None, None])) | (~older & (t < L[:, None])[:, None])
    kept = torch.sort(torch.where(stays, t, t + cap), dim=-1).values[..., :keep]
    kept = torch.where((torch.arange(keep, device=m.device) < n[:, None])[:, None], kept, -1)
    pad = -keep % 32
    src = torch.nn.functional.pad(kept, (0, pad), value=-1)
    live, at = src >= 0, src.clamp(min=0)
    same = ((src == torch.arange(keep + pad, device=m.device)) | ~live).view(B, Hk, -1, 32).all(-1)
    out = {}
    for name in ("k", "v"):
        codes, scales = getattr(cache, name), getattr(cache, name + "_scale")
        d = codes.shape[-1]
        x = codes.view(torch.uint8).gather(2, at[..., None].expand(-1, -1, -1, d)).view(ref.E4M3).float()
        x = torch.where(live[..., None], x * scales.gather(2, at // 32)[..., None], 0.0)
        top, e = torch.frexp(x.view(B, Hk, -1, 32 * d).abs().amax(-1))
        e = torch.where(top > 0.875, e - 8, e - 9)
        s = torch.exp2(torch.where(top > 0, e, -40).clamp(-40, 40).float())
        s = torch.where(same, scales[..., : s.shape[-1]], s)
        code = (x / s.repeat_interleave(32, -1)[..., None]).clamp(-448.0, 448.0).to(ref.E4M3).float()
        out[name] = (code, s)
    return kept, n, live, out, torch.where(live, cache.mass.gather(2, at), 0.0)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,Hk,cap,keep,recent", [
    (1, 1, 65536, 30000, 100),      # 8 CTAs a head, 8 keys a thread
    (1, 1, 131072, 777, 0),         # 16
    (1, 1, 262144, 200000, 3000),   # 32
    (1, 1, 300032, 100001, 77),     # more keys than a cluster holds
    (20, 1, 20000, 5000, 40),       # 4 CTAs a head, 8 keys
    (10, 4, 8192, 8000, 0),         # 2 CTAs a head
    (38, 2, 2048, 1000, 7),         # one CTA a head, 2 keys
    (19, 4, 7008, 3333, 50),        # 8
    (16, 8, 16000, 15000, 16),      # 16
    (25, 3, 30016, 1, 0),           # 32
    (75, 1, 32768, 20000, 20000)])  # 32, mostly recent tokens
def test_eviction_selections(rfb_lib, cuda_dev, in_place, B, Hk, cap, keep, recent):
    """Every way the selection is laid out: few tokens a thread and many, one CTA a head and
    clusters, masses with ties across their stretches, NaN, infinities and zeros of both signs."""
    cache, _ = filled(rfb_lib, cuda_dev, B, Hk, cap, 32, 0, seed=cap + B, spread=2.0, mass=True)
    g = gen(cap)
    m = cache.mass
    u = torch.rand(B, Hk, cap, generator=g).to(cuda_dev)
    m[u < 0.3] = 0.25                       # a third of all ties
    m[(u >= 0.3) & (u < 0.35)] = NAN
    m[(u >= 0.35) & (u < 0.36)] = float("inf")
    m[(u >= 0.36) & (u < 0.37)] = float("-inf")
    m[(u >= 0.37) & (u < 0.38)] = -0.0
    m[(u >= 0.38) & (u < 0.39)] = 0.0
    m[(u >= 0.39) & (u < 0.40)] *= -1.0
    if B * Hk > 2:
        m[0, -1] = NAN                      # one value for a whole head
        m[1, 0] = 0.5
    L = [cap, cap - 1, cap // 2 + 5, 33, 0, 1, cap // 3, keep, keep + 1, cap // 7]
    lengths = ints([L[b % len(L)] for b in range(B)], cuda_dev)
    kept, n, live, want, mass = evicted(cache, lengths, keep, recent)
    to = cache if in_place else rfb_lib.Cache8.create(B, Hk, keep, 32, mass=True, device=cuda_dev)
    before = to.mass.clone()
    got_n, got = rfb_lib.cache_evict(cache, lengths, keep, recent, out=None if in_place else to)
    assert torch.equal(got_n.long(), n) and torch.equal(got.long(), kept)
    rows = live.shape[-1]
    for name, (code, s) in want.items():
        c = getattr(to, name)[:, :, :rows].float()
        assert torch.equal(c[live], code[live]), name
        some = live.view(B, Hk, -1, 32).any(-1)
        assert torch.equal(getattr(to, name + "_scale")[..., : rows // 32][some], s[some]), name
    got_m = to.mass[..., :rows]
    assert torch.equal(got_m[live].nan_to_num(77.0), mass[live].nan_to_num(77.0))
    behind = torch.arange(to.cap, device=cuda_dev) >= n[:, None, None].expand(B, Hk, 1)
    assert torch.equal(to.mass[behind].nan_to_num(77.0), before[behind].nan_to_num(77.0))


@pytest.mark.parametrize("cap,L", [(128, 100), (4096, 4000)])
@pytest.mark.parametrize("Nq", [1, 9])
@pytest.mark.parametrize("power", [0, 60, 66, 67, 68, 80, 120, -60, -66, -68, -80, -100, -110])
def test_attention_queries_of_any_size(rfb_lib, cuda_dev, power, Nq, cap, L):
    """Queries around 2^power with a scale of 2^-power: ordinary scores, with weights."""
    cache, refs = filled(rfb_lib, cuda_dev, 1, 1, cap, 64, 8, seed=41)
    q = torch.randn(1, 4, Nq, 64, generator=gen(200 + power)) * 2.0 ** power
    run_attn(rfb_lib, cuda_dev, cache, refs, [L], 4, Nq, q=q.bfloat16(), scale=2.0 ** -power,
             mass=torch.zeros(1, 1, cap, device=cuda_dev))


@pytest.mark.parametrize("cap,L", [(128, 100), (4096, 4000)])
@pytest.mark.parametrize("Nq", [1, 9])
@pytest.mark.parametrize("power", [10, 16, 19, 21, 22, 23, 24, 25, 26, 27, 28, 30, 45, 80])
def test_attention_scores_of_any_size(rfb_lib, cuda_dev, power, Nq, cap, L):
    """Scores around 2^power, each sign first: past 2^24 a score less a constant
    rounds by more than the constant, and a weight may not leave fp16's range."""
    cache, refs = filled(rfb_lib, cuda_dev, 1, 1, cap, 64, 8, seed=41)
    q = torch.randn(1, 4, Nq, 64, generator=gen(power)) * 2.0 ** power
    u = torch.zeros(1, 4, Nq, 8)
    u[:, 1] = torch.randn(1, Nq, 8, generator=gen(power + 1)) * 2.0 ** power
    q[:, 1] = 0.0
    run_attn(rfb_lib, cuda_dev, cache, refs, [L], 4, Nq, q=q.bfloat16(), u=u.bfloat16())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("mass", [True, False])
@pytest.mark.parametrize("H,Hk,Nq,cap,d,r", [
    (2, 2, 5, 256, 64, 8),        # up to 8 rows, a CTA a segment
    (1, 1, 7, 4096, 32, 0),       # the same, many CTAs
    (4, 1, 40, 256, 64, 24),      # several row segments
    (2, 1, 9, 2048, 128, 64),     # weights beside the join
    (3, 1, 50, 4096, 64, 16)])    # weights behind it
def test_attention_of_a_padded_batch(rfb_lib, cuda_dev, H, Hk, Nq, cap, d, r, mass, causal):
    """Sequences with fewer queries than rows, appended and asked with the same counts:
    each as if it were alone, whatever lies in the rows behind its queries."""
    counts = [Nq, 1, Nq - 1, 0, Nq // 2, Nq + 3, -2]
    lengths = [cap - 3, 33, Nq - 1, 60, cap // 2, Nq, 20]
    B, g = len(counts), gen(cap + Nq)
    cache, refs = filled(rfb_lib, cuda_dev, B, Hk, cap, d, r, seed=Nq)
    n = [min(max(c, 0), Nq) for c in counts]
    new = {m: torch.randn(B, Hk, Nq, ch, generator=g).bfloat16() if ch else None
           for m, ch in (("k", d), ("v", d), ("w", r))}
    begin = [L - c for L, c in zip(lengths, n)]
    q = torch.randn(B, H, Nq, d, generator=g).bfloat16()
    u = (torch.randn(B, H, Nq, r, generator=g) * r ** -0.5).bfloat16() if r else None
    for b in range(B):      # what a padded batch holds there
        for t in (q, u):
            if t is not None:
                t[b, :, n[b]:] = NAN if b % 2 else 3.0e38
    c = ints(counts, cuda_dev)
    rfb_lib.cache_append(cache, *(t if t is None else t.to(cuda_dev) for t in new.values()),
                         start=ints(begin, cuda_dev), counts=c)
    for m, rf in refs.items():
        rf.append(new[m], begin, n)
    old = torch.rand(B, Hk, cap, generator=g)
    got_m = torch.full((B, Hk, cap), 123.0, device=cuda_dev)
    kw = dict(mass=old.to(cuda_dev), mass_out=got_m, decay=0.5) if mass else {}
    o, lse = rfb_lib.attn_fwd_cache(q.to(cuda_dev), u.to(cuda_dev) if r else None, cache,
                                    ints(lengths, cuda_dev), causal=causal, counts=c, **kw)
    val = {m: rf.values() for m, rf in refs.items()}
    for b in range(B):
        one = {m: v[b: b + 1] for m, v in val.items()}
        qs, us = q[b: b + 1, :, : n[b]], u[b: b + 1, :, : n[b]] if r else None
        ro, rl, rm, room = ref.attention(qs, us, one["k"], one["v"], one.get("w"), [lengths[b]],
                                         d ** -0.5, causal, old[b: b + 1], 0.5)
        ref.assert_within(f"o {b}", o[b: b + 1, :, : n[b]], ro, room[0])
        ref.assert_within(f"lse {b}", lse[b: b + 1, :, : n[b]], rl, room[1])
        assert bool((o[b, :, n[b]:] == 0).all()) and bool((lse[b, :, n[b]:] == float("-inf")).all())
        if mass:
            L = lengths[b]
            ref.assert_within(f"mass {b}", got_m[b: b + 1, :, :L], rm[:, :, :L], room[2][:, :, :L])
            assert bool((got_m[b, :, L:] == 123.0).all())


@pytest.mark.parametrize("causal", [True, False])
def test_padded_batch_with_nan_values(rfb_lib, cuda_dev, causal):
    """A NaN value reaches the queries that see its token and no padding row; full counts
    are the call without them, bit for bit."""
    cache, _ = filled(rfb_lib, cuda_dev, 2, 1, 96, 64, 0, seed=61)
    cache.v.view(torch.uint8)[:, 0, 40, 5] = 0x7f
    q = torch.randn(2, 2, 12, 64, generator=gen(62)).bfloat16().to(cuda_dev)
    L = ints([75, 42], cuda_dev)
    o, lse = rfb_lib.attn_fwd_cache(q, None, cache, L, causal=causal, counts=ints([12, 4], cuda_dev))
    assert bool(torch.isnan(o[0, :, :, 5]).all()) and not bool(torch.isnan(o[..., 6]).any())
    sees = torch.tensor([40 <= 42 - 4 + i if causal else True for i in range(4)])
    assert torch.equal(torch.isnan(o[1, 0, :4, 5]).cpu(), sees)
    assert bool((o[1, :, 4:] == 0).all()) and bool((lse[1, :, 4:] == float("-inf")).all())
    cache.v.view(torch.uint8)[:, 0, 40, 5] = 0
    a = rfb_lib.attn_fwd_cache(q, None, cache, L, causal=causal)
    b = rfb_lib.attn_fwd_cache(q, None, cache, L, causal=causal, counts=ints([12, 12], cuda_dev))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_counts_are_read_on_the_device_and_checked(rfb_lib, cuda_dev):
    cache, _ = filled(rfb_lib, cuda_dev, 2, 2, 64, 64, 0, seed=7)
    q = torch.randn(2, 4, 3, 64, generator=gen(8)).bfloat16().to(cuda_dev)
    L, c = ints([9, 30], cuda_dev), ints([3, 1], cuda_dev)
    for bad, err in ((c.long(), TypeError), (c[:1], ValueError), (c.cpu(), ValueError), (3, TypeError)):
        with pytest.raises(err, match="counts"):
            rfb_lib.attn_fwd_cache(q, None, cache, L, counts=bad)
    rfb_lib.attn_fwd_cache(q, None, cache, L, counts=c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = rfb_lib.attn_fwd_cache(q, None, cache, L, counts=c)
    for v in ([3, 1], [0, 2], [1, 3]):
        c.copy_(torch.tensor(v))
        graph.replay()
        eo, el = rfb_lib.attn_fwd_cache(q, None, cache, L, counts=c)
        assert torch.equal(o, eo) and torch.equal(lse, el)
        assert bool((lse[0, :, v[0]:] == float("-inf")).all()) and bool((lse[0, :, : v[0]] > -1e9).all())


@pytest.mark.parametrize("d,r,Nq,cap,L", [
    (64, 0, 1, 512, 512), (64, 8, 1, 4096, 4001), (128, 0, 1, 512, 77), (32, 16, 9, 512, 300),
    (64, 16, 9, 4096, 4096), (128, 64, 40, 512, 500), (64, 0, 70, 4096, 3999)])
def test_attention_weights_keep_fp32(rfb_lib, cuda_dev, d, r, Nq, cap, L):
    """Nearly equal weights on values that cancel: what is left shows each weight's rounding.

    A weight is off by its exponent's rounding (|x - m| < 16: 2^-21), the exponential's 2^-22
    and its two fp16 terms' 2^-22, a product by its sum's 2^-22; together below 2^-19 of
    sum p |v|, where one fp16 term would be off by 2^-12 a weight.  The common factor of a
    row and bf16 are relative to O."""
    g = gen(d + cap)
    cache = rfb_lib.Cache8.create(1, 1, cap, d, r, device=cuda_dev)
    k, v = torch.randn(cap, d, generator=g) * 64, torch.randn(cap // 2, d, generator=g) * 64
    cache.k.copy_(k.to(ref.E4M3)[None, None])
    cache.v.copy_(torch.stack((v, -v), 1).view(cap, d).to(ref.E4M3)[None, None])
    if r:
        cache.w.copy_((torch.randn(cap, r, generator=g) * 64).to(ref.E4M3)[None, None])
    val = {m: cache.values(m).cpu().double() for m in ("k", "v") + (("w",) if r else ())}
    q = (torch.randn(1, 2, Nq, d, generator=g) * 2.0 ** -20).bfloat16()
    u = (torch.randn(1, 2, Nq, r, generator=g) * 2.0 ** -20).bfloat16() if r else None
    o, _ = rfb_lib.attn_fwd_cache(q.to(cuda_dev), u.to(cuda_dev) if r else None, cache, ints([L], cuda_dev),
                                  1.0, causal=False)
    x = q.double() @ val["k"][0, 0, :L].T
    if r:
        x = x + u.double() @ val["w"][0, 0, :L].T
    assert float(x.abs().max()) < 2.0 ** -5     # so a score's own rounding is below 2^-23
    p = torch.softmax(x, -1)
    want = p @ val["v"][0, 0, :L]
    room = 2.0 ** -19 * (p @ val["v"][0, 0, :L].abs()) + (2.0 ** -8 + 2.0 ** -16) * want.abs()
    ref.assert_within("o", o, want, room)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("amplitude", [1.0, 1.25])
def test_rotary_angles_near_half_turns(rfb_lib, cuda_dev, inverse, amplitude):
    """Angles 2^-5 to 2^-16 off a half or whole turn: the sine is as small as that, and
    right to fp32's own steps, not to those of an angle of half a turn.

    Room: the sine's ulp and half, the rounding of the product with the amplitude and of
    the rotation (2^-24 each) make 2^-22 of the value; the angle in 64 bits is 2^-52 of
    itself off here and in the definition."""
    turns = torch.tensor([k / 2 + sign * (2.0 ** -e + j * 2.0 ** -29.7)
                          for k in (0, 1, 7, 101) for sign in (-1, 1) for e in (5, 9, 13, 16)
                          for j in range(8)], dtype=torch.float64)
    freqs = (turns * 2 * torch.pi / 7.0).abs()      # at position 7
    rot = 2 * freqs.numel()
    x = torch.zeros(1, 1, 2, rot)
    x[..., : rot // 2] = 1.0
    pos = torch.tensor([7, -7], dtype=torch.int32)
    turn = rfb_lib.rotary_bwd if inverse else rfb_lib.rotary_fwd
    y, _ = turn(x.to(cuda_dev), None, pos.to(cuda_dev), freqs.to(cuda_dev), amplitude=amplitude)
    want, _ = ref.rotary(x, pos, freqs, "half", amplitude, inverse=inverse)
    angle = pos.double()[None, None, :, None] * torch.cat((freqs, freqs))
    ref.assert_within("y", y, want, want.abs() * 2.0 ** -22 + angle.abs() * amplitude * 2.0 ** -51)


def test_views_of_single_sequences(rfb_lib, cuda_dev):
    """A cache and outputs that are views of one sequence each, whose scales, LSE and
    lengths lie at any 4-byte boundary, as the whole batch's calls."""
    B, H, Nq, cap, d, r = 3, 3, 1, 96, 64, 8
    names = ("k", "v", "w", "k_scale", "v_scale", "w_scale", "mass")
    whole, _ = filled(rfb_lib, cuda_dev, B, 1, cap, d, r, seed=7, mass=True)
    parts, _ = filled(rfb_lib, cuda_dev, B, 1, cap, d, r, seed=7, mass=True)
    g = gen(9)
    x = [torch.randn(B, 1, 2, c, generator=g).bfloat16().to(cuda_dev) for c in (d, d, r)]
    q, u = (torch.randn(B, H, Nq, c, generator=g).bfloat16().to(cuda_dev) for c in (d, r))
    start, lengths = ints([30, 63, 80], cuda_dev), ints([32, 65, 82], cuda_dev)
    rfb_lib.cache_append(whole, *x, start=start)
    o, lse = rfb_lib.attn_fwd_cache(q, u, whole, lengths, mass=whole.mass, mass_out=whole.mass)
    new, kept = rfb_lib.cache_evict(whole, lengths, 40, 5)
    got_lse = torch.zeros(B, H, Nq, device=cuda_dev)
    for b in range(B):
        s = slice(b, b + 1)
        one = rfb_lib.Cache8(*(getattr(parts, n)[s] for n in names))
        assert b == 0 or one.k_scale.data_ptr() % 16 and got_lse[s].data_ptr() % 16
        rfb_lib.cache_append(one, *(t[s] for t in x), start=start[s])
        ob, lb = rfb_lib.attn_fwd_cache(q[s], u[s], one, lengths[s], mass=one.mass, mass_out=one.mass,
                                        lse=got_lse[s])
        nb, kb = rfb_lib.cache_evict(one, lengths[s], 40, 5)
        assert torch.equal(ob, o[s]) and torch.equal(lb, lse[s])
        assert torch.equal(nb, new[s]) and torch.equal(kb, kept[s])
        empty = torch.empty(1, 3, 0, d, dtype=torch.bfloat16, device=cuda_dev)
        rfb_lib.attn_fwd_cache(empty, u[s, :, :0], one, lengths[s], mass=one.mass, mass_out=one.mass)
    for n in names:
        a, b = (getattr(c, n).view(torch.uint8) for c in (whole, parts))
        assert torch.equal(a, b), n
    assert torch.equal(got_lse, lse)


@pytest.mark.parametrize("need_q,need_k", [(True, True), (True, False), (False, True)])
def test_rotary_backward_turns_what_is_wanted(rfb_lib, cuda_dev, monkeypatch, need_q, need_k):
    """With q or k frozen the backward turns the other's gradient alone, to the same bits;
    gradients of gradients go the same way."""
    from rank_biased_window_b200 import serving
    g = gen(17)
    q, k, dq, dk = (torch.randn(2, h, 5, 32, generator=g).to(cuda_dev) for h in (4, 2, 4, 2))
    f, _ = rfb_lib.rotary_frequencies(32, device=cuda_dev)
    pos = ints(list(range(5)), cuda_dev)
    want = rfb_lib.rotary_bwd(dq, dk, pos, f)
    q.requires_grad_(need_q), k.requires_grad_(need_k)
    dq.requires_grad_(), dk.requires_grad_()
    qo, ko = rfb_lib.rfb_rotary(q, k, pos, f)
    turned, turn = [], serving.rotary_bwd
    monkeypatch.setattr(serving, "rotary_bwd", lambda a, b, *r, **kw: turned.append(
        [t is not None and t.shape[1] for t in (a, b)]) or turn(a, b, *r, **kw))
    inputs = [t for t, n in ((q, need_q), (k, need_k)) if n]
    got = torch.autograd.grad([qo, ko], inputs, [dq, dk], create_graph=True)
    assert turned == [[4, 2] if need_q and need_k else [4, False] if need_q else [2, False]]
    for a, b in zip(got, [w for w, n in zip(want, (need_q, need_k)) if n]):
        assert torch.equal(a, b)
    z = torch.randn(got[0].shape, generator=g).to(cuda_dev)
    back, = torch.autograd.grad(got[0], dq if need_q else dk, z)
    assert torch.equal(back, rfb_lib.rotary_fwd(z, None, pos, f)[0])
