"""Serving operators on the GPU, beyond test_gpu_serving.py: calls that follow
one another without a pause, sizes and values at the ends of their ranges."""
import pytest
import torch

from tests import _serving_ref as ref
from tests.test_gpu_serving import filled, gen, ints

pytestmark = pytest.mark.gpu


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
