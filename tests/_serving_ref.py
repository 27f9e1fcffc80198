"""Plain 64-bit definitions of the serving operators for their tests, on the
CPU, and the error bounds that the tests hold the kernels to.

Bounds count roundings: half a step of bf16 is 2^-8 of a value, of fp16 2^-11,
of fp32 2^-24.
"""
import math

import torch

BLOCK = 32
E4M3 = torch.float8_e4m3fn


def f64(t):
    return t.detach().cpu().double()


# ------------------------------------------------------------------- rotary
def rotary(x, positions, freqs, layout, amplitude=1.0, inverse=False):
    """x [B, H, N, d]; positions [B, N] or [N]; 64 bits throughout."""
    y = f64(x).contiguous().clone()
    B, H, N, d = y.shape
    pos = f64(positions).reshape(-1, N).expand(B, N)
    rot = 2 * freqs.numel()
    t = pos[:, None, :, None] * f64(freqs) * (-1.0 if inverse else 1.0)
    c, s = amplitude * torch.cos(t), amplitude * torch.sin(t)
    i = torch.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    x1, x2 = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    # what a sine or cosine that is 2^-22 off moves a value by
    room = torch.zeros_like(y)
    room[..., a] = room[..., b] = (x1.abs() + x2.abs()) * amplitude * 2.0 ** -21
    return y, room


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


# -------------------------------------------------------------------- cache
def scale_of(amax):
    """Smallest power of two with amax / scale <= 448, exponent in [-40, 40]."""
    s = 2.0 ** -40
    while amax > 448.0 * s and s < 2.0 ** 40:
        s *= 2.0
    return s


def to_codes(x, scale):
    """e4m3 values nearest x / scale (ties to even; beyond 448 the largest code)."""
    return (x / scale).clamp(-448.0, 448.0).float().to(E4M3)


class Ref:
    """One tensor of a cache in 64 bits: codes (as values) [B, H, cap, c] and scales."""

    def __init__(self, codes, scales):
        self.c, self.s = codes.cpu().double(), scales.cpu().double()

    def values(self):
        return self.c * self.s.repeat_interleave(BLOCK, 2)[..., None]

    def append(self, x, start, counts):
        B, H, cap, ch = self.c.shape
        x = f64(x)
        for b in range(B):
            s0 = min(max(int(start[b]), 0), cap)
            end = min(s0 + min(max(int(counts[b]), 0), x.shape[2]), cap)
            if end == s0:
                continue
            for h in range(H):
                for j in range(s0 // BLOCK, (end + BLOCK - 1) // BLOCK):
                    lo, hi = max(j * BLOCK, s0), min((j + 1) * BLOCK, end)
                    new = x[b, h, lo - s0: hi - s0]
                    fin = new[torch.isfinite(new)].abs()
                    s = scale_of(float(fin.max()) if fin.numel() else 0.0)
                    if lo > j * BLOCK:
                        was = float(self.s[b, h, j])
                        s = max(s, was)
                        if s != was:
                            old = self.c[b, h, j * BLOCK: lo]
                            self.c[b, h, j * BLOCK: lo] = to_codes(old * was, s).double()
                    self.s[b, h, j] = s
                    self.c[b, h, lo: hi] = to_codes(new, s).double()


def attention(q, u, k, v, w, lengths, scale, causal, mass=None, decay=1.0):
    """k, v, w: values [B, Hk, cap, c].  Returns o, lse, the new mass (or None) and
    the rooms of o, lse and mass."""
    q = f64(q)
    B, H, Nq, d = q.shape
    Hk, cap = k.shape[1], k.shape[2]
    G = H // Hk
    o = torch.zeros_like(q)
    lse = torch.full((B, H, Nq), float("-inf"), dtype=torch.float64)
    room_o, room_lse = torch.zeros_like(o), torch.zeros_like(lse)
    new_mass = None if mass is None else f64(mass).clone()
    room_m = None if mass is None else torch.zeros_like(new_mass)
    for b in range(B):
        L = min(max(int(lengths[b]), 0), cap)
        if L == 0:
            continue
        if mass is not None:
            new_mass[b, :, :L] *= decay
            room_m[b, :, :L] = new_mass[b, :, :L].abs() * 2.0 ** -23
        for h in range(H):
            hk = h // G
            kk, vv = k[b, hk, :L], v[b, hk, :L]
            x = scale * (q[b, h] @ kk.T)
            size = scale * (q[b, h].abs() @ kk.abs().T)
            if u is not None:
                uu, ww = f64(u)[b, h], w[b, hk, :L]
                x = x + uu @ ww.T
                size = size + uu.abs() @ ww.abs().T
            if causal:
                t = torch.arange(L)[None, :]
                x = x.masked_fill(t > L - Nq + torch.arange(Nq)[:, None], float("-inf"))
            some = (x > float("-inf")).any(-1)
            top = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(some, top, torch.zeros_like(top))[:, None])
            p[~some] = 0.0
            lse[b, h] = top
            seen = torch.where(x > float("-inf"), torch.ones_like(x), torch.zeros_like(x))
            # a weight of zero keeps a NaN out, a NaN weight does not
            pv = torch.where(p[..., None] == 0, torch.zeros((), dtype=x.dtype), p[..., None] * vv[None])
            o[b, h] = pv.sum(1)
            # a score in fp32: at most 12 accumulation steps and the two scalings, 2^-18 of the
            # sum of magnitudes; so a probability is off by twice that, by the exponential's
            # 2^-21 and by its rounding to fp16: half a step is 2^-11 of a normal value and 2^-25
            # below 2^-14; the kernel's weights are lifted by 2^11 at least, so the latter is 2^-36
            # of the largest weight (which matters where a small weight meets a large value)
            off = (torch.nan_to_num(size) * seen).amax(-1) * 2.0 ** -18
            a = pv.abs().sum(1)
            room_o[b, h] = (2.0 ** -11 + 2.0 ** -19 + 4 * off[:, None]) * a + 2.0 ** -8 * o[b, h].abs() \
                + 2.0 ** -36 * p.amax(-1)[:, None] * torch.nan_to_num(seen[..., None] * vv.abs()[None]).sum(1)
            room_lse[b, h] = 2 * off + 2.0 ** -20 + torch.nan_to_num(top.abs(), posinf=0.0) * 2.0 ** -22
            if mass is not None:
                new_mass[b, hk, :L] += p.sum(0)
                room_m[b, hk, :L] += p.sum(0) * 2.0 ** -18 + (p * (4 * off[:, None])).sum(0) \
                    + (p * torch.nan_to_num(top.abs(), posinf=0.0)[:, None]).sum(0) * 2.0 ** -21
    return o, lse, new_mass, (room_o, room_lse, room_m)


def evict(refs, mass, lengths, keep, recent):
    """refs: dict of Ref.  Returns kept [B, H, keep], lengths, moved refs' (values of
    codes, scales) per block as lists, and the moved mass, for entries < n."""
    mass = f64(mass)
    B, H, cap = mass.shape
    kept = torch.full((B, H, keep), -1, dtype=torch.int64)
    new_len = torch.zeros(B, dtype=torch.int64)
    out = {name: {} for name in refs}
    for b in range(B):
        L = min(max(int(lengths[b]), 0), cap)
        n = min(L, keep)
        rec = min(recent, n)
        new_len[b] = n
        for h in range(H):
            old = [(-math.inf, 1, t) if math.isnan(m) else (m, 0, t)
                   for t, m in enumerate(mass[b, h, : L - rec].tolist())]
            # largest first; among equals the lowest index; NaN behind -inf
            old.sort(key=lambda e: (-e[0], e[1], e[2]))
            idx = sorted(t for _, _, t in old[: n - rec]) + list(range(L - rec, L))
            kept[b, h, :n] = torch.tensor(idx, dtype=torch.int64)
            for name, ref in refs.items():
                for j in range((n + BLOCK - 1) // BLOCK):
                    src = idx[j * BLOCK: (j + 1) * BLOCK]
                    if src == list(range(j * BLOCK, j * BLOCK + len(src))):
                        out[name][b, h, j] = (ref.c[b, h, src], float(ref.s[b, h, j]))
                        continue
                    x = ref.c[b, h, src] * ref.s[b, h, [t // BLOCK for t in src]][:, None]
                    fin = x[torch.isfinite(x)].abs()
                    s = scale_of(float(fin.max()) if fin.numel() else 0.0)
                    out[name][b, h, j] = (to_codes(x, s).double(), s)
    return kept, new_len, out


def assert_within(name, got, ref, room, exact_where=None):
    """|got - ref| <= room; infinities and NaN in the same places."""
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    nan, inf = torch.isnan(ref), torch.isinf(ref)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaN in other places"
    assert torch.equal(got[inf], ref[inf]), f"{name}: infinities differ"
    fin = ~(nan | inf)
    over = ((got - ref).abs() - room)[fin]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{name}: {worst:.3e} beyond its room"
