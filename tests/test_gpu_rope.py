"""Rotary positions with several axes (attn_rope, attn_rope_bwd) and their cache-writing form
(attn_paged_append) against plain fp64 arithmetic (needs a GB300).

Tolerance.  The kernel rotates in fp32 and rounds once to bf16: half a bf16 step, 2^-8 relative to
the result.  Angles are good to about 2^-24 of a turn's fraction and sine and cosine to a few
2^-24, so the fp32 part is below 2^-20 (|x0| + |x1|).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

CANARY = 0x7BAD


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


def status_ok(attn):
    assert attn.cache_device_status() == (0, 0)


def turned(x, positions, freqs, axes, pairing, sign=1.0):
    """fp64 rotation of x [..., tokens, heads, d] (any leading axes); positions [axes, ..., tokens].
    Returns (y, sum of the terms' magnitudes, mask of rotated elements)."""
    x = np.asarray(x, dtype=np.float64)
    y, mag = x.copy(), np.zeros_like(x)
    n = len(freqs)
    for p in range(n):
        i, j = (2 * p, 2 * p + 1) if pairing == "adjacent" else (p, p + n)
        # whole turns taken off in extended precision: far positions keep their fp64 angle
        angle = np.asarray(positions[axes[p]], dtype=np.longdouble) * np.longdouble(freqs[p])
        c, s = np.cos(angle).astype(np.float64)[..., None], sign * np.sin(angle).astype(np.float64)[..., None]
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., j] * c + x[..., i] * s
        mag[..., i] = mag[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, mag


def check(got, x, positions, freqs, axes, pairing, sign=1.0):
    ref, mag = turned(x.float().cpu().numpy(), positions.cpu().numpy(), freqs.cpu().numpy(), axes.cpu().numpy(),
                      pairing, sign)
    got = got.float().cpu().numpy().astype(np.float64)
    tol = np.abs(ref) * 2.0 ** -8 + mag * 2.0 ** -20
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))
    n = 2 * len(freqs)
    assert np.array_equal(got[..., n:], ref[..., n:])        # the rest passes through


def draw(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


CASES = [  # B, S, H, Hkv, d, layout, axis dims, pairing, first position
    (1, 1, 1, 1, 128, "bshd", (128,), "adjacent", 0),
    (2, 37, 4, 2, 64, "bhsd", (32, 16), "adjacent", 5),
    (1, 130, 12, 12, 128, "bshd", (44, 42, 42), "adjacent", 0),
    (3, 33, 5, 1, 128, "bshd", (32, 48, 48), "halves", -40),
    (2, 61, 6, 3, 64, "bhsd", (32,), "halves", 1000000),
    (1, 517, 32, 8, 128, "bshd", (128,), "halves", 2 ** 31 - 600),
    (1, 700, 1, 1, 64, "bshd", (2,), "adjacent", -2 ** 31),
    (2, 9, 71, 1, 128, "bhsd", (16, 16, 16, 16), "halves", 7),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_S%d_H%d_%d_d%d_%s_%s_%s" % (
    c[0], c[1], c[2], c[3], c[4], c[5], "x".join(map(str, c[6])), c[7]))
def test_rope_and_its_gradient(attn, case):
    B, S, H, Hkv, d, layout, dims, pairing, first = case
    freqs, axes = attn.rope_freqs(dims)
    g = torch.Generator().manual_seed(B * S)
    positions = torch.stack([(first + torch.arange(S, dtype=torch.int64) if a == 0 else
                              torch.randint(-50, 4000, (S,), generator=g)) for a in range(len(dims))])
    positions = positions.to(torch.int32).cuda()
    shape = (lambda n: (B, S, n, d)) if layout == "bshd" else (lambda n: (B, n, S, d))
    q, k = draw(*shape(H), seed=S), draw(*shape(Hkv), seed=S + 1)
    back = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2))
    qo, ko = attn.attn_rope(q, k, positions, freqs, axes, layout=layout, pairing=pairing)
    dq, dk = attn.attn_rope_bwd(q, k, positions, freqs, axes, layout=layout, pairing=pairing)
    status_ok(attn)
    for x, y, dx in ((q, qo, dq), (k, ko, dk)):
        assert y.is_contiguous() and y.shape == x.shape
        check(back(y), back(x), positions[:, None], freqs, axes, pairing)
        check(back(dx), back(x), positions[:, None], freqs, axes, pairing, sign=-1.0)
    only = attn.attn_rope(q, None, positions, freqs, axes, layout=layout, pairing=pairing)
    assert torch.equal(only.view(torch.int16), qo.view(torch.int16))


def test_gradient_against_differences(attn):
    # L = sum(G * rope(x)) is linear in x: L(x + e) - L(x - e) over 2 e is the gradient.  With x = 0 the
    # forward of one unit element gives a column of the rotation, whose dot product with G is that
    # element's gradient; bf16 rounding of the column, the gradient and nothing else (G is bf16).
    d, S = 64, 5
    freqs, axes = attn.rope_freqs((32, 32))
    positions = torch.tensor([[0, 3, 17, 100, 5000], [1, 0, 2, 9, 77]], dtype=torch.int32, device="cuda")
    G = draw(1, S, 1, d, seed=3)
    grad, _ = attn.attn_rope_bwd(G, G, positions, freqs, axes)
    unit = torch.eye(d, dtype=torch.bfloat16, device="cuda")[None, :, None, :].expand(S, d, 1, d).contiguous()
    cols, _ = attn.attn_rope(unit, unit, positions.T[:, :, None].expand(S, 2, d).permute(1, 0, 2).contiguous(), freqs, axes)
    for s in range(S):
        num = cols[s, :, 0].double() @ G[0, s, 0].double()
        # two rounded cosine/sine entries per column, each half a step off
        tol = 2.0 ** -8 * (cols[s, :, 0].double().abs() @ G[0, s, 0].double().abs()) + 2.0 ** -8 * num.abs() + 1e-5
        assert ((grad[0, s, 0].double() - num).abs() <= tol).all()


def test_positions_per_batch_and_packed(attn):
    B, S, H, d = 3, 20, 4, 128
    freqs, axes = attn.rope_freqs((64, 64), spectrum="shared")
    positions = torch.randint(0, 9999, (2, B, S), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    q = draw(B, S, H, d, seed=2)
    y = attn.attn_rope(q, None, positions, freqs, axes)
    check(y, q, positions, freqs, axes, "adjacent")
    packed = attn.attn_rope(q.flatten(0, 1), None, positions.flatten(1), freqs, axes)
    assert torch.equal(packed.view(torch.int16), y.flatten(0, 1).view(torch.int16))
    status_ok(attn)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_views_of_a_projection_and_in_place(attn, layout):
    B, S, H, Hkv, d = 2, 45, 6, 2, 128
    freqs, axes = attn.rope_freqs((128,))
    positions = torch.arange(S, dtype=torch.int32, device="cuda")[None]
    x = draw(B, S, H + 2 * Hkv, d, seed=4)
    keep = x.clone()
    view = lambda t, a, b: t[:, :, a:b] if layout == "bshd" else t[:, :, a:b].transpose(1, 2)  # noqa: E731
    q, k = view(x, 0, H), view(x, H, H + Hkv)
    want = attn.attn_rope(q.contiguous(), k.contiguous(), positions, freqs, axes, layout=layout)
    got = attn.attn_rope(q, k, positions, freqs, axes, layout=layout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(x, keep)
    qo, ko = attn.attn_rope(q, k, positions, freqs, axes, layout=layout, q_out=q, k_out=k)      # in place
    assert qo is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, :, H + Hkv:], keep[:, :, H + Hkv:])                                   # v untouched
    # one in place, the other to a tensor of its own
    x.copy_(keep)
    _, ko = attn.attn_rope(q, k, positions, freqs, axes, layout=layout, q_out=q)
    assert torch.equal(q, want[0]) and torch.equal(ko, want[1]) and torch.equal(k, view(keep, H, H + Hkv))
    status_ok(attn)


def test_one_token_a_sequence_in_place_and_a_shared_input(attn):
    B, H, Hkv, d = 3, 4, 2, 64
    freqs, axes = attn.rope_freqs((64,))
    positions = torch.tensor([[[5], [900], [77]]], dtype=torch.int32, device="cuda")       # [axes, B, 1]
    x = draw(B, 1, H + 2 * Hkv, d, seed=8)
    keep = x.clone()
    q, k = x[:, :, :H], x[:, :, H:H + Hkv]
    want = attn.attn_rope(q, k, positions, freqs, axes)
    check(want[0], keep[:, :, :H], positions, freqs, axes, "adjacent")
    attn.attn_rope(q, k, positions, freqs, axes, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, :, H + Hkv:], keep[:, :, H + Hkv:])
    # one row of queries for every sequence (a stride of zero)
    one = draw(1, 1, H, d, seed=9)
    got = attn.attn_rope(one.expand(B, 1, H, d), None, positions, freqs, axes)
    assert torch.equal(got, attn.attn_rope(one.expand(B, 1, H, d).contiguous(), None, positions, freqs, axes))
    status_ok(attn)


def test_what_the_binding_refuses(attn):
    freqs, axes = attn.rope_freqs((64,))
    q, k, pos = draw(1, 6, 4, 64), draw(1, 6, 2, 64), torch.zeros((1, 6), dtype=torch.int32, device="cuda")
    rope = attn.attn_rope
    for call, error in (
            (lambda: rope(q.float(), k, pos, freqs, axes), TypeError),
            (lambda: rope(q.cpu(), k, pos, freqs, axes), TypeError),
            (lambda: rope(q, k.cpu(), pos, freqs, axes), TypeError),
            (lambda: rope(q, k, pos.long(), freqs, axes), TypeError),
            (lambda: rope(q, k, pos, freqs.float(), axes), TypeError),
            (lambda: rope(q, k, pos, freqs, axes[:5]), ValueError),
            (lambda: rope(q, k, pos[:, :5], freqs, axes), ValueError),
            (lambda: rope(q, k[:, :5], pos, freqs, axes), ValueError),
            (lambda: rope(q, k, pos, freqs, axes, layout="sbhd"), ValueError),
            (lambda: rope(q, k, pos, freqs, axes, pairing="both"), ValueError),
            (lambda: rope(q, k, pos, freqs, axes, q_out=q[:, :5]), ValueError),
            (lambda: rope(q, None, pos, freqs, axes, k_out=k), ValueError),
            (lambda: rope(q.transpose(2, 3), k, pos, freqs, axes), ValueError),
            (lambda: rope(q, k, pos, freqs, axes, q_out=k.expand_as(k), k_out=q), ValueError),
            (lambda: rope(draw(1, 6, 4, 96), None, pos, freqs, axes), attn.AttnError),
            (lambda: rope(q, k, pos, torch.ones(40, dtype=torch.float64, device="cuda"),
                          torch.zeros(40, dtype=torch.int32, device="cuda")), attn.AttnError),
            (lambda: rope(q, k, pos, freqs[:12], axes[:12], pairing="halves"), attn.AttnError),
            (lambda: rope(q[:, :4], None, pos[:, :4], freqs, axes, q_out=q[:, 1:5]), attn.AttnError)):
        with pytest.raises(error):
            call()
    status_ok(attn)


def test_non_finite_elements_stay_in_their_pair_and_the_rest_keeps_its_bits(attn):
    freqs, axes = attn.rope_freqs((32,))
    q = torch.zeros((1, 3, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 1, 0, 4] = float("inf")
    q[0, 2, 0, 9] = float("nan")
    q[0, 0, 0, 40] = float("nan")
    q[0, 1, 0, 41] = -0.0
    q.view(torch.int16)[0, 2, 0, 63] = 0x7F81            # a signalling pattern passes through
    y = attn.attn_rope(q, None, torch.tensor([[1, 2, 3]], dtype=torch.int32, device="cuda"), freqs, axes)
    odd = ~torch.isfinite(y[0, :, 0, :32])
    assert odd[1].nonzero().flatten().tolist() == [4, 5] and odd[2].nonzero().flatten().tolist() == [8, 9]
    assert not odd[0].any()
    assert torch.equal(y[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))


def test_no_tokens(attn):
    freqs, axes = attn.rope_freqs((64,))
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert attn.attn_rope(q, None, torch.empty((1, 0), dtype=torch.int32, device="cuda"), freqs, axes).shape == q.shape


def test_an_axis_that_is_not_there_is_reported(attn):
    freqs, axes = attn.rope_freqs((32, 32))
    q = draw(1, 4, 2, 64)
    out = torch.full_like(q, 7.0)
    attn.attn_rope(q, None, torch.zeros((1, 4), dtype=torch.int32, device="cuda"), freqs, axes, q_out=out)
    assert attn.cache_device_status() == (1, 20)
    assert (out == 7.0).all()
    status_ok(attn)


# ------------------------------------------------------------------------------------- append
def filled(*shape):
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    t.view(torch.int16).fill_(CANARY)
    return t


APPEND = [  # new tokens, lengths with them, H, Hkv, d, page size, pairing or None
    ([1, 1, 1], [1, 130, 77], 4, 2, 128, 16, "halves"),
    ([5, 0, 33, 1], [5, 40, 100, 24], 3, 3, 64, 24, "adjacent"),
    ([200, 17], [333, 17], 16, 2, 128, 128, "halves"),
    ([7], [9], 1, 1, 64, 1, "adjacent"),
    ([3, 2], [10, 2], 2, 1, 128, 5, None),
    ([1] * 1500, list(range(1, 1501)), 1, 1, 64, 256, "halves"),      # offsets searched in global memory
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "n%d_H%d_%d_d%d_P%d_%s" % (
    len(c[0]), c[2], c[3], c[4], c[5], c[6]))
def test_append(attn, case):
    new, lens, H, Hkv, d, P, pairing = case
    B, lead, tail = len(new), 2, 3                        # rows in front of the first sequence, behind the last
    total = lead + sum(new) + tail
    cu = np.cumsum([lead] + new)
    most = -(-max(lens) // P)
    rng = np.random.default_rng(P)
    table = rng.permutation(B * most).reshape(B, most).astype(np.int32)
    x = draw(total, H + 2 * Hkv, d, seed=P)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    kc, vc, qo = filled(B * most, P, Hkv, d), filled(B * most, P, Hkv, d), filled(total, H, d)
    freqs, axes = attn.rope_freqs((32, 16, 16) if d == 64 else (64, 32, 32))
    positions = torch.as_tensor(rng.integers(0, 50000, (3, total)).astype(np.int32)).cuda()
    rot = dict(positions=positions, freqs=freqs, axes=axes, pairing=pairing) if pairing else {}
    got = attn.attn_paged_append(k, v, kc, vc, torch.as_tensor(cu.astype(np.int32)).cuda(),
                                 torch.as_tensor(np.asarray(lens, dtype=np.int32)).cuda(),
                                 torch.as_tensor(table).cuda(), q=q, q_out=qo, **rot)
    status_ok(attn)
    assert got is qo
    if pairing:
        qr, kr = attn.attn_rope(q, k, positions, freqs, axes, pairing=pairing)
        check(qr[None], q[None], positions[:, None], freqs, axes, pairing)
    else:
        qr, kr = q, k
    want_k, want_v, want_q = filled(*kc.shape), filled(*vc.shape), filled(*qo.shape)
    want_q[lead:lead + sum(new)] = qr[lead:lead + sum(new)]
    b = np.repeat(np.arange(B), new)
    at = np.concatenate([np.arange(n - m, n) for m, n in zip(new, lens)]).astype(np.int64)
    rows = torch.as_tensor(table[b, at // P].astype(np.int64) * P + at % P).cuda()
    want_k.view(-1, Hkv, d)[rows] = kr[lead:lead + sum(new)]
    want_v.view(-1, Hkv, d)[rows] = v[lead:lead + sum(new)]
    for g, w in ((kc, want_k), (vc, want_v), (qo, want_q)):
        assert torch.equal(g.view(torch.int16), w.view(torch.int16))


def test_append_slots_that_are_not_in_the_cache(attn):
    P, Hkv, d = 4, 2, 64
    kc, vc = filled(3, P, Hkv, d), filled(3, P, Hkv, d)
    k, v = draw(5, Hkv, d, seed=1), draw(5, Hkv, d, seed=2)
    # fine; a page of the table out of range; longer than the table; shorter than its new tokens; a negative page
    cu = torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 1, 9, 0, 1], dtype=torch.int32, device="cuda")
    table = torch.tensor([[1, 0], [3, 0], [0, 1], [0, 1], [-1, 0]], dtype=torch.int32, device="cuda")
    attn.attn_paged_append(k, v, kc, vc, cu, lens, table)
    assert attn.cache_device_status() == (1, 21)
    want = filled(3, P, Hkv, d)
    want[1, 1] = k[0]
    assert torch.equal(kc.view(torch.int16), want.view(torch.int16))
    status_ok(attn)


def test_offsets_that_decrease_write_inside_the_lengths_only(attn):
    P, Hkv, d = 4, 1, 64
    kc, vc = filled(4, P, Hkv, d), filled(4, P, Hkv, d)
    k, v = draw(6, Hkv, d, seed=1), draw(6, Hkv, d, seed=2)
    cu = torch.tensor([0, 3, 1, 6], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 2, 5], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 3], [1, 3], [2, 3]], dtype=torch.int32, device="cuda")
    attn.attn_paged_append(k, v, kc, vc, cu, lens, table)
    attn.cache_device_status()
    untouched = filled(1, Hkv, d)[0].view(torch.int16)
    for b, n in enumerate(lens.tolist()):
        for j in range(n, P):
            assert torch.equal(kc[b, j].view(torch.int16), untouched), (b, j)
    status_ok(attn)


def test_captured_and_replayed_on_another_stream(attn):
    freqs, axes = attn.rope_freqs((128,))
    q, k = draw(1, 50, 4, 128, seed=1), draw(1, 50, 2, 128, seed=2)
    positions = torch.arange(50, dtype=torch.int32, device="cuda")[None]
    want = attn.attn_rope(q, k, positions, freqs, axes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qs, ks = attn.attn_rope(q, k, positions, freqs, axes, stream=side)
    side.synchronize()
    assert torch.equal(qs, want[0]) and torch.equal(ks, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg, kg = attn.attn_rope(q, k, positions, freqs, axes)
    q.copy_(q.flip(1))
    want = attn.attn_rope(q, k, positions, freqs, axes)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qg, want[0]) and torch.equal(kg, want[1])
    status_ok(attn)
