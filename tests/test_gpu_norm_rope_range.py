"""Heads at the ends of bf16's range through attn_norm_rope, its gradient and the cache append (needs a GB300).

Documented: a head whose squares' sum overflows fp32 comes out zero, whatever the weights and angles; small heads come out right, also
those whose squares underflow.  Tolerances of test_gpu_norm_rope.py (half a bf16 step and 2^-18, 2^-17 of the terms); a bf16 result below 2^-126
is off by half a step there, 2^-134.
"""
import numpy as np
import pytest
import torch

from tests import norm_rope_ref as ref
from tests.test_gpu_norm_rope import attn, draw, f64  # noqa: F401

pytestmark = pytest.mark.gpu

H, S = 5, 70


def tables(attn, d):  # noqa: F811
    freqs, axes = attn.rope_freqs((d,))
    return torch.arange(S, dtype=torch.int32, device="cuda")[None], freqs, axes


def append(attn, x, w, t, pairing, eps):  # noqa: F811
    """Keys through the cache append."""
    kc, vc = (torch.full((S, 1, H, x.shape[2]), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    attn.attn_norm_rope_append(x, x, kc, vc, torch.arange(S, device="cuda"), k_weight=w, positions=t[0], freqs=t[1], axes=t[2], eps=eps,
                               pairing=pairing)
    return kc[:, 0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("weighted", [0.0, 1.0, 1e30])
def test_heads_near_the_largest_number_come_out_zero(attn, d, pairing, weighted):  # noqa: F811
    t = tables(attn, d)
    x, dy = draw(S, H, d, seed=1), draw(S, H, d, seed=2)
    w = (1.5 + torch.arange(d) / d).cuda() * weighted if weighted else None
    clean = attn.attn_norm_rope(x, None, w, None, *t, pairing=pairing)
    clean_dx, _ = attn.attn_norm_rope_bwd(dy, None, x, None, w, None, *t, pairing=pairing)
    x[::3, 2] = torch.where(x[::3, 2] < 0, -3.38e38, 3.38e38).to(torch.bfloat16)
    y = attn.attn_norm_rope(x, None, w, None, *t, pairing=pairing)
    dx, _ = attn.attn_norm_rope_bwd(dy, None, x, None, w, None, *t, pairing=pairing)
    big = torch.zeros((S, H), dtype=torch.bool, device="cuda")
    big[::3, 2] = True
    for got, want in ((y, clean), (append(attn, x, w, t, pairing, 1e-6), clean), (dx, clean_dx)):
        assert not got[big].any() and torch.equal(got[~big], want[~big])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_small_heads(attn, d, pairing, eps):  # noqa: F811
    """Sizes from 1 to 10^-38, next to each other in a warp; with eps = 0 all of them are normed to 1."""
    t = tables(attn, d)
    sizes = 10.0 ** -torch.linspace(0, 38, S * H).view(S, H)
    x = (torch.randn((S, H, d), generator=torch.Generator().manual_seed(1)) * sizes[torch.randperm(S), :, None]).to(torch.bfloat16).cuda()
    w = (1 + torch.arange(d) / d).cuda()
    dy = draw(S, H, d, seed=2, scale=2.0 ** -20)
    y = attn.attn_norm_rope(x, None, w, None, *t, eps=eps, pairing=pairing)
    dx, dw = attn.attn_norm_rope_bwd(dy, None, x, None, w, None, *t, eps=eps, pairing=pairing)
    assert torch.equal(append(attn, x, w, t, pairing, eps), y)
    pos, freqs, axes = f64(t[0]), f64(t[1]), t[2].cpu().numpy()
    eps = float(np.float32(eps))
    want, mag = ref.forward(f64(x), f64(w), eps, pos, freqs, axes, pairing)
    assert np.all(np.abs(f64(y) - want) <= np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -18 + 2.0 ** -134)
    want, mag, sums, sums_mag = ref.backward(f64(dy), f64(x), f64(w), eps, pos, freqs, axes, pairing)
    fits = np.abs(want) + mag * 2.0 ** -17 < 3e38                      # (1 / 10^-38 times a gradient may not)
    assert fits.mean() > 0.97
    err = np.abs(f64(dx) - want) - (np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -17 + 2.0 ** -134)
    assert np.all(err[fits] <= 0), float(err[fits].max())
    assert np.all(np.abs(f64(dw) - sums) <= sums_mag * (200 * 2.0 ** -24 + 2.0 ** -17))
