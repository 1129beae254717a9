"""Angles of attn_rope and attn_paged_append where they show: small ones beside a partner of zero, those of
fast pairs at far positions, and frequencies that are not finite (needs a GB300).

Tolerances.  An element x0 cos - x1 sin is rounded once to bf16, half a step, 2^-8 of itself.  Before that, in
fp32: the angle in half turns is rounded once (2^-24 of itself; at most pi 2^-25 rad), cosine and sine are off by
2^-23 of themselves at most, two products and their difference by 2^-24 each.  With one product zero all of
these are relative to the result, below 2^-21 together; in general they are below 2^-21 (|x0| + |x1|).  The
frequency's fraction of a turn is off by a unit of 2^-64 at most, which a position p multiplies: below
2^-32 turns, 2^-29 rad, of an angle of any size, and 2^-30 of the smallest angles below.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# 1 / 2 pi to 60 digits
TURN = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


def angle(position, freq):
    """position * freq in radians, whole turns taken off exactly, -pi .. pi."""
    turns = position * Fraction(freq) * TURN
    return float((turns - round(turns)) / TURN)


def rotated(positions, freqs):
    """Cosines and sines [tokens, pairs] in 64 bits."""
    a = np.array([[angle(p, f) for f in freqs] for p in positions])
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("base", [1e4, 5e5, 1e7, 1e9])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_small_angles_beside_a_partner_of_zero(attn, base, pairing):
    d, positions = 128, [0, 1, -1, 2, 3, -5, 7, 10, 33, 64, 100, 1000, -4095, 100000]
    freqs, axes = attn.rope_freqs((d,), base=base)
    pos = torch.tensor([positions], dtype=torch.int32, device="cuda")
    q = torch.zeros((1, len(positions), 2, d), dtype=torch.bfloat16, device="cuda")
    first, second = (slice(0, None, 2), slice(1, None, 2)) if pairing == "adjacent" else (slice(0, 64), slice(64, None))
    q[:, :, 0, first] = 1.0            # head 0: (1, 0), head 1: (0, 1.5)
    q[:, :, 1, second] = 1.5
    c, s = rotated(positions, freqs.tolist())
    want = np.zeros((len(positions), 2, d))
    want[:, 0, first], want[:, 0, second] = c, s
    want[:, 1, first], want[:, 1, second] = -1.5 * s, 1.5 * c
    back = want.copy()
    back[:, 0, second], back[:, 1, first] = -s, 1.5 * s
    kc, vc = (torch.empty((1, len(positions), 2, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = torch.tensor([0, len(positions)], dtype=torch.int32, device="cuda")
    attn.attn_paged_append(q[0], q[0], kc, vc, n, n[1:], torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                           positions=pos, freqs=freqs, axes=axes, pairing=pairing)
    for got, ref in ((attn.attn_rope(q, None, pos, freqs, axes, pairing=pairing), want), (kc, want),
                     (attn.attn_rope(q, None, pos, freqs, axes, pairing=pairing, inverse=True), back)):
        off = np.abs(got[0].float().cpu().numpy().astype(np.float64) - ref) - (2.0 ** -8 + 2.0 ** -21) * np.abs(ref)
        assert np.all(off <= 0), (float(off.max()), np.argwhere(off > 0)[:4])
    assert attn.cache_device_status() == (0, 0)


def test_far_positions_of_fast_pairs(attn):
    # a frequency's own error counts 2^31 times here; where the two products cancel the angle shows
    d, freqs = 64, [1.0, 0.7, 2.5, 17.0, 100.0, 3.3e4, -1e6, 1e-4]
    positions = [s * (2 ** 31 - 1 - 37 * i) for i in range(300) for s in (1, -1)] + [-2 ** 31, 2 ** 30, 10 ** 9 + 7]
    x = np.random.default_rng(5).integers(-60, 61, (len(positions), 8, len(freqs), 2)) / 64.0       # exact in bf16
    q = torch.zeros((1, len(positions), 8, d), dtype=torch.bfloat16, device="cuda")
    q[0, :, :, :2 * len(freqs)] = torch.as_tensor(x).flatten(2).to(torch.bfloat16)
    got = attn.attn_rope(q, None, torch.tensor([positions], dtype=torch.int32, device="cuda"),
                         torch.tensor(freqs, dtype=torch.float64, device="cuda"),
                         torch.zeros(len(freqs), dtype=torch.int32, device="cuda"))
    c, s = (t[:, None] for t in rotated(positions, freqs))
    ref = np.stack([x[..., 0] * c - x[..., 1] * s, x[..., 1] * c + x[..., 0] * s], -1)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * np.abs(x).sum(-1, keepdims=True)
    off = np.abs(got[0, :, :, :2 * len(freqs)].float().cpu().numpy().reshape(x.shape) - ref) - tol
    assert np.all(off <= 0), [float(off[:, :, p].max()) for p in range(len(freqs))]
    assert attn.cache_device_status() == (0, 0)


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_a_frequency_that_is_not_finite_makes_its_pair_nan(attn, pairing):
    # at position 0 too: 0 * inf has no value; the pair's zeros are NaN as well, the other pairs and the rest keep theirs
    d, odd = 64, {0: float("nan"), 3: float("inf"), 6: float("-inf")}
    freqs, axes = attn.rope_freqs((16, 16))
    positions = torch.tensor([[0, 1, -7, 2 ** 31 - 1], [0, 5, 6, 7]], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 4, 3, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q[0, 1, 1] = 0.0
    want = attn.attn_rope(q, None, positions, freqs, axes, pairing=pairing)
    hit = torch.zeros(d, dtype=torch.bool)
    for p, f in odd.items():
        freqs[p] = f
        for i in (2 * p, 2 * p + 1) if pairing == "adjacent" else (p, p + 16):
            hit[i] = True
    for inverse in (False, True):
        got = attn.attn_rope(q, None, positions, freqs, axes, pairing=pairing, inverse=inverse)
        assert torch.isnan(got[..., hit]).all() and not torch.isnan(got[..., ~hit]).any()
        if not inverse:
            assert torch.equal(got[..., ~hit], want[..., ~hit])
    assert attn.cache_device_status() == (0, 0)
