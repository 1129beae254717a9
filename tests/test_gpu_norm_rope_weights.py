"""The weights' gradients of attn_norm_rope_bwd, to a bound that a single token or head left out breaks (needs a GB300).

Tolerance, derived before the first run, from how the kernels add.  `blocks` = min(4 an SM, ceil(tokens / 4)) blocks of 4 warps take a token
a warp at a time, and 512 / d heads of it side by side: a thread's fp32 chain has ceil(tokens / (4 blocks)) tokens of
ceil(heads / (512 / d)) terms (k's a token's sum at a time, one more step each); then come 3 levels of a warp, 4 warps,
ceil(blocks / 32) blocks and 32 sums of those.  Each step is off by 2^-24 of the magnitudes so far.  Beside that a term, a
rotated gradient times a normed element, is off by 2^-17 of its magnitude (the squares' sum of 16 terms and 3 levels 19 * 2^-24, half of
it in the root; the angle 2^-24 of half a turn; sine, cosine, root and products 2^-24 to 2^-22 each).
"""
import numpy as np
import pytest
import torch

from tests import norm_rope_ref as ref
from tests.test_gpu_norm_rope import attn, draw, f64, tables_of, weight  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [  # B, S, H, Hkv, d, layout, axis dims, pairing, first position
    (1, 5003, 3, 1, 64, "bshd", (48,), "halves", -9),               # 3 tokens a warp, one part of the heads
    (3, 1201, 7, 2, 128, "bhsd", (64, 32), "adjacent", 3),          # 2, across batch entries
    (1, 1021, 17, 3, 64, "bshd", (64,), "halves", 0),               # 3 parts of the heads
    (2, 2433, 9, 5, 128, "bshd", (44, 42, 42), "halves", 7),        # one token over two a warp
    (1, 130, 12, 12, 128, "bshd", (128,), "adjacent", 0),           # fewer tokens than warps
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_S%d_H%d_%d_d%d_%s" % c[:6])
def test_every_token_and_head_counts(attn, case):  # noqa: F811
    B, S, H, Hkv, d, layout, dims, pairing, _ = case
    tables = tables_of(attn, case)
    to = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2).contiguous())
    x = [draw(B, S, h, d, seed=10 + h, scale=2) for h in (H, Hkv)]
    dy = [draw(B, S, h, d, seed=20 + h) for h in (H, Hkv)]
    w = [weight(d, "fp32", 5), weight(d, "fp32", 6)]
    back = attn.attn_norm_rope_bwd(*map(to, dy), *map(to, x), *w, *tables, layout=layout, pairing=pairing)
    assert attn.cache_device_status() == (0, 0)
    pos, freqs, axes = f64(tables[0]), f64(tables[1]), tables[2].cpu().numpy()
    tokens = B * S
    blocks = min(4 * torch.cuda.get_device_properties(0).multi_processor_count, -(-tokens // 4))
    for t in range(2):
        g, v, got, heads = f64(dy[t]), f64(x[t]), f64(back[2 + t]), x[t].shape[2]

        def sums(b, s, h):
            return ref.backward(g[b, s, h], v[b, s, h], f64(w[t]), 1e-6, pos[:, s], freqs, axes, pairing)[2:]
        every = slice(None)
        dw, mag = sums(every, every, every)
        chain = -(-tokens // (4 * blocks)) * (-(-heads // (512 // d)) + 1) + 3 + 4 + -(-blocks // 32) + 32
        tol = mag * (chain * 2.0 ** -24 + 2.0 ** -17)
        assert np.all(np.abs(got - dw) <= tol), float((np.abs(got - dw) - tol).max())
        # the bound sees a token or a head of one that is left out
        last = slice(S - 1, S)
        for part in ((slice(0, 1), slice(0, 1), every), (slice(B - 1, B), last, every), (slice(0, 1), slice(S // 2, S // 2 + 1), every),
                     (slice(B - 1, B), last, slice(heads - 1, heads))):
            assert np.any(np.abs(got - (dw - sums(*part)[0])) > tol), part
