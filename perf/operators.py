"""Workloads of the serving operators: rotary positions, the 8-bit key / value
cache (append, attention with the rank-factorised bias, eviction) and one
decode step of them together.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the package's entry points;
``exact`` is the operator's definition in 64 bits.

The cache holds e4m3 values with one scale per head and 32 tokens.  A scale is
a power of two, 2^ceil(log2(amax / 448)) with the exponent held in [-40, 40],
so that a value's code and its requantisation are the same in any precision.
"""
import math

import torch

own = False

BLOCK = 32          # tokens per scale
E4M3 = torch.float8_e4m3fn


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of 8 sequences: q and k of a decode step, latency
        dict(name="rotary_token", op="rotary", B=8, H=8, Hk=8, N=1, d=64, rot=64, layout="half",
             dtype="bf16", scaling="none", far=4096, train=False, strided=False),
        # training at the framework's 16384-token shape: q and k as the projection leaves them
        # ([B, N, H, d]), half of each head rotated, forward and backward
        dict(name="rotary_train", op="rotary", B=2, H=8, Hk=8, N=16384, d=64, rot=32,
             layout="interleaved", dtype="bf16", scaling="linear", far=0, train=True, strided=True),
        # a long prompt far behind the trained length, 32-bit values, shared key heads
        dict(name="rotary_far", op="rotary", B=1, H=12, Hk=4, N=4097, d=128, rot=128,
             layout="half", dtype="fp32", scaling="by_parts", far=1000000, train=False,
             strided=False),
        # one new token of 32 sequences into the cache, with its bias factor
        dict(name="append_token", op="append", B=32, Hk=8, n=1, d=64, r=32, cap=4096, start=3001),
        # four prompts of different length into an empty cache
        dict(name="append_prompt", op="append", B=4, Hk=8, n=4001, d=128, r=0, cap=4096, start=0),
        # one token, one sequence, a short context: latency
        dict(name="attn_token_short", op="attn", B=1, H=8, Hk=8, Nq=1, d=64, r=8, L=300, cap=512,
             ragged=False, mass=False),
        # a decode batch with shared key heads and lengths from 1/16 to all of 8192
        dict(name="attn_token", op="attn", B=16, H=32, Hk=8, Nq=1, d=128, r=0, L=8190, cap=8192,
             ragged=True, mass=False),
        # few sequences, a very long context, rank-32 bias factors
        dict(name="attn_long", op="attn", B=2, H=8, Hk=8, Nq=1, d=64, r=32, L=131000, cap=131072,
             ragged=False, mass=False),
        # a chunk of 16 tokens (a continued prompt, or drafted tokens) with attention weights kept
        dict(name="attn_chunk", op="attn", B=8, H=16, Hk=4, Nq=16, d=64, r=16, L=5003, cap=8192,
             ragged=True, mass=True),
        # one short sequence cut to half
        dict(name="evict_short", op="evict", B=1, Hk=8, d=64, r=8, L=1000, cap=1024, keep=512,
             recent=64, ragged=False),
        # a full batch cut to half its capacity
        dict(name="evict_batch", op="evict", B=8, Hk=8, d=128, r=0, L=16384, cap=16384, keep=8192,
             recent=512, ragged=True),
        # a decode step: positions, append, attention with weights kept
        dict(name="step", op="step", B=16, H=8, Hk=8, Nq=1, d=64, r=32, L=4097, cap=8192,
             ragged=True, mass=True, rot=64, layout="half", scaling="none"),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["rotary", "append", "attn", "attn", "evict", "step"])
    d = rng.choice([32, 64, 128])
    if op == "rotary":
        layout = rng.choice(["half", "interleaved"])
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 2, 3, 4])
        B = rng.randint(1, 8)
        rot = rng.choice([d, d, d // 2, 12, 16, 20])
        return dict(op=op, B=B, H=H, Hk=Hk, N=log(1, max(1, 150000 // (B * (H + Hk)))), d=d, rot=rot,
                    layout=layout, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    scaling=rng.choice(["none", "linear", "base", "by_parts"]),
                    far=rng.choice([0, 5000, 1000000]), train=rng.random() < 0.5,
                    strided=rng.random() < 0.5)
    r = rng.choice([0, 8, 16, 24, 32, 40, 64])
    if op == "append":
        B, Hk = log(1, 32), rng.choice([1, 2, 4, 8])
        n = log(1, min(4000, max(1, 120000 // (B * Hk))))
        start = rng.choice([0, rng.randint(1, 3000)])
        return dict(op=op, B=B, Hk=Hk, n=n, d=d, r=r, start=start,
                    cap=-(-(start + n + rng.randint(0, 100)) // BLOCK) * BLOCK)
    Hk = rng.choice([1, 2, 4, 8])
    if op == "evict":
        B = log(1, 16)
        L = log(2, max(2, min(16384, 400000 // (B * Hk))))
        keep = rng.randint(1, L + 20)
        return dict(op=op, B=B, Hk=Hk, d=d, r=r, L=L, cap=-(-max(L, keep) // BLOCK) * BLOCK,
                    keep=keep, recent=rng.randint(0, keep), ragged=rng.random() < 0.7)
    G = rng.choice([1, 1, 2, 4, 5, 8])
    Nq = rng.choice([1, 1, 1, 2, 5, 16, 33])
    B = log(1, 32)
    L = log(max(2, Nq), max(40, min(131072, 1000000 // (B * Hk * max(1, G * Nq // 16)))))
    c = dict(op=op, B=B, H=Hk * G, Hk=Hk, Nq=Nq, d=d, r=r, L=L,
             cap=-(-(L + rng.randint(0, 200)) // BLOCK) * BLOCK, ragged=rng.random() < 0.6,
             mass=rng.random() < 0.4)
    if op == "step":
        c.update(mass=True, rot=rng.choice([d, d // 2]), layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear"]))
    return c


def _lengths(case, L):
    """Tokens of each sequence: all L, or spread between about L / 16 and L."""
    B = case["B"]
    if not case.get("ragged") or B == 1:
        return [L] * B
    low = max(1, L // 16)
    return [L - (L - low) * ((5 * b) % B) // B for b in range(B)]


def _append_counts(case):
    """New tokens of each sequence: all n, or for prompts n less a sixteenth per sequence."""
    n = case["n"]
    return [max(1, n - (n * b) // (16 * case["B"])) if n > 1 else 1 for b in range(case["B"])]


def _append_starts(case):
    return [max(0, case["start"] - 7 * b) for b in range(case["B"])]


# ------------------------------------------------------------------ quantiser
def _pow2_scale(amax):
    """2^ceil(log2(amax / 448)), exponent in [-40, 40]; 448 = 0.875 2^9."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -40)).clamp(-40, 40)
    return torch.ldexp(torch.ones_like(amax), e)


def _to_code(x):
    return x.clamp(-448.0, 448.0).to(E4M3)


def _quantise(x):
    """x [B, H, cap, c] fp32 -> codes and scales [B, H, cap / 32]."""
    B, H, cap, c = x.shape
    t = x.view(B, H, cap // BLOCK, BLOCK * c)
    s = _pow2_scale(t.abs().amax(-1))
    return _to_code(t / s[..., None]).view(B, H, cap, c), s


def _values(codes, scales):
    B, H, cap, c = codes.shape
    return (codes.float().view(B, H, cap // BLOCK, BLOCK * c) * scales[..., None]).view(codes.shape)


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    op = case["op"]
    st = dict(case=case, op=op)
    if op in ("rotary", "step"):
        st["rot_args"] = (case["rot"], 10000.0, case["scaling"], 4.0, 4096)
        f, a = _frequencies(*st["rot_args"])
        st["freqs"], st["amplitude"] = f.to(dev), a
    if op == "rotary":
        dt = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)[case["dtype"]]
        B, N, d = case["B"], case["N"], case["d"]

        def act(H):
            if case["strided"]:
                return randn(B, N, H, d).to(dt).transpose(1, 2)
            return randn(B, H, N, d).to(dt)
        st["q"], st["k"] = act(case["H"]), act(case["Hk"])
        if case["train"]:
            st["dq"], st["dk"] = randn(B, case["H"], N, d).to(dt), randn(B, case["Hk"], N, d).to(dt)
        st["positions"] = ints([[case["far"] + 37 * b + i for i in range(N)] for b in range(B)])
        return st

    B, Hk, d, r, cap = case["B"], case["Hk"], case["d"], case["r"], case["cap"]

    def keys(n, c, spread):
        # activations: per-channel gains between 1/2 and about 3, slow drift along the tokens
        gain = torch.exp(0.5 * randn(1, Hk, 1, c)) * spread
        drift = torch.exp(0.3 * torch.sin(torch.arange(n, device=dev) / 50.0))[None, None, :, None]
        return randn(B, Hk, n, c) * gain * drift

    if op == "append" and case["start"] == 0:
        contents = [torch.zeros(B, Hk, cap, c, device=dev) for c in (d, d, r)]
    else:
        contents = [keys(cap, d, 1.0), keys(cap, d, 1.0), keys(cap, r, max(r, 1) ** -0.5)]
    for name, x in zip(("k8", "v8", "w8"), contents):
        if x.shape[-1]:
            st[name], st[name[0] + "s"] = _quantise(x)
        else:
            st[name] = st[name[0] + "s"] = None
    del contents
    # accumulated weights: heavy tailed, a fifth of the tokens never attended to
    u = torch.rand((B, Hk, cap), generator=g, device=dev)
    st["mass"] = torch.where(u < 0.2, torch.zeros_like(u), u ** 12 * 8)

    if op == "append":
        n = case["n"]
        st["start"], st["counts"] = ints(_append_starts(case)), ints(_append_counts(case))
    if op == "step":
        n = case["Nq"]
        st["lengths"] = ints(_lengths(case, case["L"]))
        st["start"] = (st["lengths"] - n).clamp(min=0)
        st["counts"] = ints([n] * B)
        st["positions"] = (st["start"][:, None] + torch.arange(n, device=dev, dtype=torch.int32)[None])
    if op in ("append", "step"):
        # as the projections leave them: [B, n, heads, channels]
        st["k"], st["v"] = (keys(n, d, 1.2).bfloat16().transpose(1, 2).contiguous().transpose(1, 2)
                            for _ in range(2))
        st["w"] = keys(n, r, r ** -0.5).bfloat16() if r else None
    if op in ("attn", "step"):
        H, Nq = case["H"], case["Nq"]
        st["lengths"] = ints(_lengths(case, case["L"]))
        st["q"] = randn(B, H, Nq, d).bfloat16()
        st["u"] = (randn(B, H, Nq, r) * r ** -0.5).bfloat16() if r else None
        st["mass_out"] = torch.zeros_like(st["mass"])
    if op == "evict":
        st["lengths"] = ints(_lengths(case, case["L"]))
        for name in ("k8", "v8", "w8", "ks", "vs", "ws", "mass"):
            t = st[name]
            st["new_" + name] = None if t is None else torch.zeros_like(t)
    if own:
        import rank_biased_window_b200 as rfb
        st["cache"] = rfb.Cache8(st["k8"], st["v8"], st["w8"], st["ks"], st["vs"], st["ws"],
                                 mass=st["mass"])
        if op == "evict":
            st["new_cache"] = rfb.Cache8(*(st["new_" + n] for n in ("k8", "v8", "w8", "ks", "vs", "ws")),
                                         mass=st["new_mass"])
    return st


def _frequencies(rot, base, scaling, factor, original):
    """Angular frequencies per position (fp64) and the amplitude of the rotation.

    none: base^(-2i / rot); linear: positions divided by the factor; base: the base raised to
    base factor^(rot / (rot - 2)), which stretches the slowest pair by the factor; by_parts: pairs
    that turn more than 32 times within the original length as they are, those that turn less than
    once divided by the factor, a ramp between, and the amplitude 0.1 ln(factor) + 1."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    a = 1.0
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        def pair(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        a = 0.1 * math.log(factor) + 1.0
    return f, a


# --------------------------------------------------------------- plain forms
def _rotate(x, positions, freqs, amplitude, layout, sign):
    rot = 2 * freqs.numel()
    ang = positions.double()[:, None, :, None] * freqs
    c, s = (torch.cos(ang) * amplitude).float(), (torch.sin(ang) * (amplitude * sign)).float()
    f = x.float()
    y = f.clone(memory_format=torch.contiguous_format)
    if layout == "half":
        a, b = f[..., : rot // 2], f[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    else:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y.to(x.dtype)


def _plain_rotary(st):
    layout, args = st["case"]["layout"], (st["positions"], st["freqs"], st["amplitude"])
    out = dict(q=_rotate(st["q"], *args, layout, 1.0), k=_rotate(st["k"], *args, layout, 1.0))
    if "dq" in st:
        out["gq"] = _rotate(st["dq"], *args, layout, -1.0)
        out["gk"] = _rotate(st["dk"], *args, layout, -1.0)
    return out


def _append_one(codes, scales, x, start, counts):
    """New rows x [B, H, n, c] into codes / scales, in place, block by block."""
    B, H, n, c = x.shape
    cap = codes.shape[2]
    nb = (n + BLOCK - 1) // BLOCK + 1
    blk = (start.long() // BLOCK)[:, None] + torch.arange(nb, device=x.device)       # [B, nb]
    t = (blk[..., None] * BLOCK + torch.arange(BLOCK, device=x.device))              # [B, nb, 32]
    i = t - start.long()[:, None, None]
    new = (i >= 0) & (i < counts.long()[:, None, None]) & (t < cap)
    old = (i < 0) & (t < cap)
    bi = torch.arange(B, device=x.device)[:, None, None]
    xs = x.float()[bi, :, i.clamp(0, n - 1)].permute(0, 3, 1, 2, 4)                  # [B, H, nb, 32, c]
    xs = torch.where(new[:, None, ..., None], xs, torch.zeros_like(xs))
    was = codes[bi, :, t.clamp(max=cap - 1)].permute(0, 3, 1, 2, 4).float()
    s_old = scales[bi[..., 0], :, blk.clamp(max=cap // BLOCK - 1)].permute(0, 2, 1)  # [B, H, nb]
    fin = torch.where(torch.isfinite(xs), xs.abs(), torch.zeros_like(xs))
    s = _pow2_scale(fin.amax((-1, -2)))
    s = torch.where(old.any(-1)[:, None], torch.maximum(s, s_old), s)
    touched = new.any(-1)[:, None].expand(B, H, nb)
    fresh = _to_code(xs / s[..., None, None]).float()
    again = _to_code(was * (s_old / s)[..., None, None]).float()
    res = torch.where(new[:, None, ..., None], fresh, torch.where(old[:, None, ..., None], again, was))
    b, h, k = touched.nonzero(as_tuple=True)
    scales[b, h, blk[b, k]] = s[b, h, k]
    b2, h2, k2, j2 = ((new | old)[:, None] & touched[..., None]).nonzero(as_tuple=True)
    codes[b2, h2, t[b2, k2, j2]] = res[b2, h2, k2, j2].to(E4M3)


def _plain_append(st, k, v, w):
    start, counts = st["start"], st["counts"]
    for name, x in (("k", k), ("v", v), ("w", w)):
        if x is not None:
            _append_one(st[name + "8"], st[name + "s"], x, start, counts)
    t = torch.arange(st["mass"].shape[2], device=start.device)
    new = (t >= start[:, None]) & (t < (start + counts)[:, None])
    st["mass"].masked_fill_(new[:, None], 0.0)
    return {n: st[n] for n in ("k8", "v8", "w8", "ks", "vs", "ws", "mass") if st[n] is not None}


def _plain_attn(st, q, want_mass):
    case = st["case"]
    B, H, Nq, d = q.shape
    Hk, G, cap = case["Hk"], case["H"] // case["Hk"], case["cap"]
    L = st["lengths"]
    k, v = _values(st["k8"], st["ks"]), _values(st["v8"], st["vs"])
    x = (q.float().view(B, Hk, G * Nq, d) @ k.transpose(2, 3)) * d ** -0.5
    if st["u"] is not None:
        x = x + st["u"].float().view(B, Hk, G * Nq, -1) @ _values(st["w8"], st["ws"]).transpose(2, 3)
    t = torch.arange(cap, device=q.device)
    i = torch.arange(Nq, device=q.device).repeat(G)
    sees = t[None, None] <= (L[:, None, None] - Nq + i[None, :, None])
    x = x.masked_fill(~sees[:, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    out = dict(o=(p @ v).to(q.dtype).view(B, H, Nq, d), lse=(m + torch.log(l)).view(B, H, Nq))
    if want_mass:
        inside = (t[None, :] < L[:, None])[:, None]
        st["mass_out"].copy_(torch.where(inside, st["mass"] + p.sum(2), st["mass_out"]))
        out["mass"] = st["mass_out"]
    return out


def _plain_evict(st):
    case, L = st["case"], st["lengths"].long()
    B, Hk, cap = st["mass"].shape
    keep = case["keep"]
    n = L.clamp(max=keep)
    rec = n.clamp(max=case["recent"])
    t = torch.arange(cap, device=L.device)
    older = (t[None] < (L - rec)[:, None])[:, None].expand(B, Hk, cap)
    key = torch.where(older, st["mass"].double(), torch.full((), float("-inf"), device=L.device,
                                                             dtype=torch.float64))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand(B, Hk, cap))
    stays = (older & (rank < (n - rec)[:, None, None])) | ((t[None] >= (L - rec)[:, None])
                                                           & (t[None] < L[:, None]))[:, None]
    first = torch.sort(torch.where(stays, t, t + cap), dim=-1).values[..., :keep]
    used = torch.arange(keep, device=L.device)[None] < n[:, None]                     # [B, keep]
    kept = torch.where(used[:, None], first, torch.full_like(first, -1))
    nb = -(-keep // BLOCK)
    pad = nb * BLOCK - keep
    src = torch.nn.functional.pad(kept, (0, pad), value=-1)                           # [B, Hk, nb 32]
    live = (src >= 0).view(B, Hk, nb, BLOCK)
    same = ((src == torch.arange(nb * BLOCK, device=L.device)) | (src < 0)).view(B, Hk, nb, BLOCK).all(-1)
    out = dict(kept=kept.int(), lengths=n.int())
    for name in ("k", "v", "w"):
        codes, scales = st[name + "8"], st[name + "s"]
        if codes is None:
            continue
        c = codes.shape[-1]
        at = src.clamp(min=0)
        x = torch.gather(codes.view(torch.uint8), 2, at[..., None].expand(-1, -1, -1, c)).view(E4M3).float()
        x = x * torch.gather(scales, 2, at // BLOCK)[..., None]
        x = torch.where(live.view(B, Hk, -1, 1), x, torch.zeros_like(x)).view(B, Hk, nb, BLOCK, c)
        s = _pow2_scale(x.abs().amax((-1, -2)))
        s = torch.where(same, scales[:, :, :nb], s)
        code = _to_code(x / s[..., None, None])
        nc, ns = st["new_" + name + "8"], st["new_" + name + "s"]
        full = live.reshape(B, Hk, -1, 1)
        m = nb * BLOCK
        nc[:, :, :m] = torch.where(full, code.view(B, Hk, m, c).float(), nc[:, :, :m].float()).to(E4M3)
        ns[:, :, :nb] = torch.where(live.any(-1), s, ns[:, :, :nb])
        out[name + "8"], out[name + "s"] = nc, ns
    nm = st["new_mass"]
    moved = torch.gather(st["mass"], 2, src.clamp(min=0))
    nm[:, :, : nb * BLOCK] = torch.where(src >= 0, moved, nm[:, :, : nb * BLOCK])
    out["mass"] = nm
    return out


def _plain_step(st):
    layout, args = st["case"]["layout"], (st["positions"], st["freqs"], st["amplitude"])
    q, k = _rotate(st["q"], *args, layout, 1.0), _rotate(st["k"], *args, layout, 1.0)
    _plain_append(st, k, st["v"], st["w"])
    return _plain_attn(st, q, True)


# ---------------------------------------------------------------------- runs
def _own_run(st):
    import rank_biased_window_b200 as rfb
    case, op = st["case"], st["op"]
    if op == "rotary":
        args = (st["positions"], st["freqs"])
        kw = dict(layout=case["layout"], amplitude=st["amplitude"])
        q, k = rfb.rotary_fwd(st["q"], st["k"], *args, **kw)
        out = dict(q=q, k=k)
        if "dq" in st:
            out["gq"], out["gk"] = rfb.rotary_bwd(st["dq"], st["dk"], *args, **kw)
        return out
    cache = st["cache"]
    if op == "append":
        rfb.cache_append(cache, st["k"], st["v"], st["w"], start=st["start"], counts=st["counts"])
        return {n: st[n] for n in ("k8", "v8", "w8", "ks", "vs", "ws", "mass") if st[n] is not None}
    if op == "attn":
        kw = dict(mass=st["mass"], mass_out=st["mass_out"]) if case["mass"] else {}
        o, lse = rfb.attn_fwd_cache(st["q"], st["u"], cache, st["lengths"], **kw)
        return dict(o=o, lse=lse, mass=st["mass_out"]) if case["mass"] else dict(o=o, lse=lse)
    if op == "evict":
        lengths, kept = rfb.cache_evict(cache, st["lengths"], case["keep"], case["recent"],
                                        out=st["new_cache"])
        out = dict(kept=kept, lengths=lengths, mass=st["new_mass"])
        for n in ("k8", "v8", "w8", "ks", "vs", "ws"):
            if st[n] is not None:
                out[n] = st["new_" + n]
        return out
    q, k = rfb.rotary_fwd(st["q"], st["k"], st["positions"], st["freqs"], layout=case["layout"],
                          amplitude=st["amplitude"])
    rfb.cache_append(cache, k, st["v"], st["w"], start=st["start"], counts=st["counts"])
    o, lse = rfb.attn_fwd_cache(q, st["u"], cache, st["lengths"], mass=st["mass"],
                                mass_out=st["mass_out"])
    return dict(o=o, lse=lse, mass=st["mass_out"])


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "rotary":
        return _plain_rotary(state)
    if op == "append":
        return _plain_append(state, state["k"], state["v"], state["w"])
    if op == "attn":
        return _plain_attn(state, state["q"], state["case"]["mass"])
    if op == "evict":
        return _plain_evict(state)
    return _plain_step(state)


# ---------------------------------------------------------------------- work
def work(case):
    op, d = case["op"], case["d"]
    if op == "rotary":
        rows = case["B"] * case["N"] * (case["H"] + case["Hk"])
        passes = 2 if case["train"] else 1
        size = 4 if case["dtype"] == "fp32" else 2
        return dict(bytes=passes * (2 * rows * d * size + 4 * case["B"] * case["N"]),
                    flops=passes * 3 * rows * case["rot"])
    B, Hk, r = case["B"], case["Hk"], case["r"]
    row = 2 * d + r                                 # bytes of a cached token, channels of a score
    scales = 4 * (3 if r else 2) / BLOCK
    total_bytes = total_flops = 0.0
    if op in ("append", "step"):
        n = sum(_append_counts(case)) if op == "append" else B * case["Nq"]
        total_bytes += n * Hk * (2 * row + row + 4 + scales)
        total_flops += n * Hk * 2 * row
    if op == "step":
        total_bytes += 2 * 2 * n * d * (case["H"] + Hk)
        total_flops += 3 * n * case["rot"] * (case["H"] + Hk)
    if op in ("attn", "step"):
        tokens, rows = sum(_lengths(case, case["L"])), case["H"] * case["Nq"]
        total_bytes += tokens * Hk * (row + scales + (8 if case["mass"] else 0))
        total_bytes += B * rows * (2 * (2 * d + r) + 4)
        total_flops += 2.0 * tokens * rows * row
    if op == "evict":
        L = _lengths(case, case["L"])
        n = sum(min(v, case["keep"]) for v in L)
        total_bytes += Hk * (4 * sum(L) + 2 * n * (row + scales) + 4 * n + 4 * B * case["keep"])
        total_flops += Hk * n * 2 * row
    return dict(bytes=total_bytes, flops=total_flops)


# ------------------------------------------------------- definitions, 64 bits
def _exact_rotate(x, positions, rot_args, layout, sign):
    """Each pair as a complex number times a exp(+-i pos f)."""
    freqs, a = _frequencies(*rot_args)
    rot = 2 * freqs.numel()
    ang = sign * positions.double()[:, None, :, None] * freqs.to(x.device)
    turn = torch.polar(torch.full_like(ang, a), ang)
    y = x.double().clone(memory_format=torch.contiguous_format)
    if layout == "half":
        z = torch.complex(y[..., : rot // 2].clone(), y[..., rot // 2: rot].clone()) * turn
        return torch.cat([z.real, z.imag, y[..., rot:]], -1)
    z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2)) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), y[..., rot:]], -1)


def _e4m3_table(device):
    """The non-negative finite e4m3 values in order of their codes 0..126."""
    code = torch.arange(127, device=device)
    e, m = code // 8, (code % 8).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.double() - 7))


def _round_e4m3(x):
    """Nearest table value, ties to the even code, magnitudes above 448 to 448."""
    table = _e4m3_table(x.device)
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(table, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - table[lo], table[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(x < 0, -1.0, 1.0) * torch.where(up, table[hi], table[lo])


def _exact_scale(amax):
    """The smallest power of two with amax / scale <= 448, exponent in [-40, 40]."""
    e = torch.arange(-40, 41, device=amax.device).double()
    fits = amax[..., None] <= 448.0 * torch.exp2(e)
    first = torch.where(fits.any(-1), fits.int().argmax(-1), torch.full_like(fits[..., 0].long(), 80))
    return torch.exp2(e[first])


def _exact_append(st, x, name):
    """One sequence, head and block at a time over [start / 32, end / 32]."""
    codes, scales = st[name + "8"].double(), st[name + "s"].double()
    B, H, cap, c = codes.shape
    for b in range(B):
        s0, n = int(st["start"][b]), int(st["counts"][b])
        n = min(n, cap - s0)
        lo, hi = s0 // BLOCK, -(-(s0 + n) // BLOCK)
        span = torch.zeros(H, (hi - lo) * BLOCK, c, dtype=torch.float64, device=codes.device)
        span[:, s0 - lo * BLOCK: s0 - lo * BLOCK + n] = x[b, :, :n].double()
        need = _exact_scale(span.view(H, hi - lo, -1).abs().amax(-1))
        if s0 % BLOCK:
            was = scales[b, :, lo].clone()
            need[:, 0] = torch.maximum(need[:, 0], was)
            ratio = (was / need[:, 0])[:, None, None]
            codes[b, :, lo * BLOCK: s0] = _round_e4m3(codes[b, :, lo * BLOCK: s0] * ratio)
        scales[b, :, lo:hi] = need
        code = _round_e4m3(span / need.repeat_interleave(BLOCK, 1)[..., None])
        codes[b, :, s0: s0 + n] = code[:, s0 - lo * BLOCK: s0 - lo * BLOCK + n]
    return codes, scales


def _exact_attn(st, q, cache, mass):
    """Softmax over the visible prefix of each sequence, one head at a time."""
    case = st["case"]
    B, H, Nq, d = q.shape
    G = case["H"] // case["Hk"]
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, Nq), float("-inf"), dtype=torch.float64, device=q.device)
    mo = st["mass_out"].double()
    for b in range(B):
        L = int(st["lengths"][b])
        for hk in range(case["Hk"]):
            def value(name):
                codes, scales = cache[name]
                return codes[b, hk, :L].double() * scales[b, hk].double().repeat_interleave(BLOCK)[:L, None]
            k, v = value("k"), value("v")
            w = value("w") if st["u"] is not None else None
            got = torch.zeros(L, dtype=torch.float64, device=q.device)
            for h in range(hk * G, hk * G + G):
                x = q[b, h].double() @ k.T / math.sqrt(d)
                if w is not None:
                    x = x + st["u"][b, h].double() @ w.T
                behind = torch.arange(L, device=q.device)[None] - torch.arange(Nq, device=q.device)[:, None]
                x[behind > L - Nq] = float("-inf")
                top = torch.logsumexp(x, -1)
                p = torch.exp(x - top[:, None])
                p[torch.isinf(top)] = 0.0
                o[b, h], lse[b, h] = p @ v, top
                got += p.sum(0)
            mo[b, hk, :L] = mass[b, hk, :L].double() + got
    out = dict(o=o, lse=lse)
    if case["mass"]:
        out["mass"] = mo
    return out


def _exact_evict(st):
    case = st["case"]
    keep = case["keep"]
    B, Hk, cap = st["mass"].shape
    dev = st["mass"].device
    kept = torch.full((B, Hk, keep), -1, dtype=torch.int32, device=dev)
    lengths = torch.zeros(B, dtype=torch.int32, device=dev)
    names = [n for n in ("k", "v", "w") if st[n + "8"] is not None]
    new = {n: (st["new_" + n + "8"].double(), st["new_" + n + "s"].double()) for n in names}
    nm = st["new_mass"].double()
    for b in range(B):
        L = int(st["lengths"][b])
        n = min(L, keep)
        rec = min(case["recent"], n)
        lengths[b] = n
        for h in range(Hk):
            m = st["mass"][b, h, : L - rec]
            best = torch.argsort(-m.double(), stable=True)[: n - rec]
            idx = torch.cat([best.sort().values, torch.arange(L - rec, L, device=dev)])
            kept[b, h, :n] = idx.int()
            nm[b, h, :n] = st["mass"][b, h, idx].double()
            nb = -(-n // BLOCK)
            stay = torch.ones(nb * BLOCK, dtype=torch.bool, device=dev)
            stay[:n] = idx == torch.arange(n, device=dev)
            stay = stay.view(nb, BLOCK).all(-1)
            for name in names:
                codes, scales = st[name + "8"][b, h], st[name + "s"][b, h].double()
                x = torch.zeros(nb * BLOCK, codes.shape[-1], dtype=torch.float64, device=dev)
                x[:n] = codes.view(torch.uint8)[idx].view(E4M3).double() * scales[idx // BLOCK][:, None]
                s = torch.where(stay, scales[:nb], _exact_scale(x.view(nb, -1).abs().amax(-1)))
                code = _round_e4m3(x / s.repeat_interleave(BLOCK)[:, None])
                new[name][0][b, h, :n] = code[:n]
                new[name][1][b, h, :nb] = s
    out = dict(kept=kept, lengths=lengths, mass=nm)
    for n in names:
        out[n + "8"], out[n + "s"] = new[n]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "step"):
        rot = (st["positions"], st["rot_args"], case["layout"])
    if op == "rotary":
        out = dict(q=_exact_rotate(st["q"], *rot, 1.0), k=_exact_rotate(st["k"], *rot, 1.0))
        if case["train"]:
            out["gq"] = _exact_rotate(st["dq"], *rot, -1.0)
            out["gk"] = _exact_rotate(st["dk"], *rot, -1.0)
        return out
    if op in ("append", "step"):
        k = st["k"]
        if op == "step":
            # the step's keys and queries are bf16 between the operators
            k = _exact_rotate(k, *rot, 1.0).to(torch.bfloat16)
        held = {n: _exact_append(st, x, n) for n, x in (("k", k), ("v", st["v"]), ("w", st["w"]))
                if x is not None}
        mass = st["mass"].double()
        for b in range(case["B"]):
            s0 = int(st["start"][b])
            mass[b, :, s0: s0 + int(st["counts"][b])] = 0.0
    if op == "append":
        out = {n + "8": c for n, (c, _) in held.items()}
        out.update({n + "s": s for n, (_, s) in held.items()}, mass=mass)
        return out
    if op == "attn":
        held = {n: (st[n + "8"], st[n + "s"]) for n in ("k", "v", "w") if st[n + "8"] is not None}
        return _exact_attn(st, st["q"], held, st["mass"])
    if op == "step":
        return _exact_attn(st, _exact_rotate(st["q"], *rot, 1.0).to(torch.bfloat16), held, mass)
    return _exact_evict(st)
