"""Which views attn_rope takes as inputs and outputs beside one another: refused where two of them share an
element, and only there, for slices of one buffer (CPU only; fake addresses that nothing reads)."""
import ctypes
import itertools

import numpy as np
import pytest

import bf16_attention_forward_gb300 as attn
from tests.test_cache_boundary import ALIAS, M, NO_DEVICE, fake_pointers, lib  # noqa: F401  (lib is a fixture)


def call(lib, B, S, d, q, k, qo, ko, Hq, Hk):
    """Each view: (offset in elements, strides of batch, token and head)."""
    a = attn.RopeArgs()
    for n, (at, st) in (("q", q), ("k", k), ("q_out", qo), ("k_out", ko)):
        setattr(a, n, M + 2 * at)
        getattr(a, n + "_stride")[:] = st
    a.B, a.S, a.H, a.Hkv, a.d = B, S, Hq, Hk, d
    a.positions, a.freqs, a.axes = M >> 2, M >> 3, M >> 4
    a.pos_axis_stride, a.pairs, a.num_axes = S, d // 2, 1
    return lib.attn_rope(ctypes.byref(a), None)


def in_place(lib, B, S, d, q, k, Hq, Hk):
    return call(lib, B, S, d, q, k, q, k, Hq, Hk)


@fake_pointers
@pytest.mark.parametrize("B", [1, 2, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_slices_of_a_buffer_in_place(lib, B, d):  # noqa: F811
    S, H, Hkv, W = 10, 4, 2, 8
    # bhsd: heads of one [B, H + 2 Hkv, S, d] buffer
    st = (W * S * d, d, S * d)
    assert in_place(lib, B, S, d, (0, st), (H * S * d, st), H, Hkv) == NO_DEVICE
    assert in_place(lib, B, S, d, (0, st), ((H - 1) * S * d, st), H, Hkv) == ALIAS
    # bshd: the first S tokens of a longer projection buffer, heads side by side
    room = 16
    st = (room * W * d, W * d, d)
    assert in_place(lib, B, S, d, (0, st), (H * d, st), H, Hkv) == NO_DEVICE
    assert in_place(lib, B, S, d, (0, st), ((H - 1) * d, st), H, Hkv) == ALIAS
    # token ranges and batch entries of one buffer
    assert in_place(lib, B, 6, d, (0, st), (6 * W * d, st), W, W) == NO_DEVICE
    assert in_place(lib, B, 6, d, (0, st), (5 * W * d, st), W, W) == ALIAS
    st2 = (2 * S * W * d, W * d, d)
    assert in_place(lib, B, S, d, (0, st2), (S * W * d, st2), W, W) == NO_DEVICE
    # every other head, the keys' batch stride unlike the queries' (one entry: it does not count)
    st = (S * W * d, W * d, 2 * d)
    assert in_place(lib, B, S, d, (0, st), (d, st), H, H) == NO_DEVICE
    assert in_place(lib, B, S, d, (0, st), (2 * d, st), H, Hkv) == ALIAS


@fake_pointers
def test_random_views_against_their_elements(lib):  # noqa: F811
    # every extent nests in the next larger stride, as slices of one buffer do; shifts of all kinds between the two
    rng = np.random.default_rng(7)
    d, seen = 64, {ALIAS: 0, NO_DEVICE: 0}
    for _ in range(3000):
        dims = [int(x) for x in rng.integers(1, 5, 3)]               # of the buffer: outer, middle, inner, in heads of d
        order = rng.permutation(3)                                   # which of batch, token, head lies outermost ...
        unit = [dims[1] * dims[2] * d, dims[2] * d, d]
        stride = [0, 0, 0]
        step = [int(x) for x in rng.integers(1, 3, 3)]
        most = [0, 0, 0]
        for place, x in enumerate(order):
            stride[x] = unit[place] * step[place]
            most[x] = -(-dims[place] // step[place])
        B, S = int(rng.integers(1, most[0] + 1)), int(rng.integers(1, most[1] + 1))
        Hq, Hk = (int(rng.integers(1, most[2] + 1)) for _ in range(2))

        def start(heads):
            at = 0
            for place, x in enumerate(order):
                n = (B, S, heads)[x]
                at += int(rng.integers(0, dims[place] - (n - 1) * step[place])) * unit[place]
            return at

        def elements(at, heads):
            return {at + b * stride[0] + s * stride[1] + h * stride[2]
                    for b, s, h in itertools.product(range(B), range(S), range(heads))}

        q, k = start(Hq), start(Hk)
        want = ALIAS if elements(q, Hq) & elements(k, Hk) else NO_DEVICE
        got = in_place(lib, B, S, d, (q, stride), (k, stride), Hq, Hk)
        assert got == want, (dims, order, step, B, S, Hq, Hk, q, k)
        seen[got] += 1
    assert min(seen.values()) > 200


@fake_pointers
def test_views_of_unlike_strides(lib):  # noqa: F811
    # a bhsd and a bshd view of one buffer
    S, H, d = 8, 2, 64
    a, b = (0, (2 * S * d, d, S * d)), (0, (2 * S * d, 2 * d, d))
    assert call(lib, 2, S, d, a, (M, b[1]), b, (2 * M, b[1]), H, H) == ALIAS
    assert call(lib, 2, S, d, a, (M, b[1]), (4 * S * d, b[1]), (2 * M, b[1]), H, H) == NO_DEVICE
