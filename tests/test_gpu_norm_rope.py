"""Norms of queries and keys with their rotary positions (attn_norm_rope), the gradient and the form that writes the
cache, against plain fp64 arithmetic (needs a GB300).

Tolerances, derived before the first run.  Everything is computed in fp32 and rounded once to bf16: half a bf16
step, 2^-8 relative to the result.  The fp32 part: the squares' sum of 16 terms and 3 levels is good to 19 * 2^-24, its root
to half of that and 2 * 2^-24, four products and a sum behind it, sine and cosine a few 2^-24, the angle 2^-24 of half a
turn: below 2^-18 of the magnitudes of an element's terms in all.  The gradient has twice as many steps and
another sum over the head: 2^-17.  A weight's gradient is a sum whose longest chain in fp32 is of at most `rows` terms (a
thread's), 5 levels of a warp, 4 warps, and 38 + 32 sums of blocks: (rows + 80) * 2^-24 of the sum of magnitudes beside 2^-17.
"""
import ctypes

import numpy as np
import pytest
import torch

from tests import norm_rope_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def draw(*shape, seed=0, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()


def weight(d, kind, seed):
    if kind == "none":
        return None
    w = 1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))
    return w.to(torch.bfloat16 if kind == "bf16" else torch.float32).cuda()


def within(got, want, tol):
    got = f64(got)
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))


def check_forward(got, x, w, eps, tables, pairing):
    y, mag = ref.forward(f64(x), f64(w), eps, f64(tables[0]), f64(tables[1]), tables[2].cpu().numpy(), pairing)
    within(got, y, np.abs(y) * 2.0 ** -8 + mag * 2.0 ** -18)


def check_backward(got, got_w, dy, x, w, eps, tables, pairing):
    dx, mag, dw, w_mag = ref.backward(f64(dy), f64(x), f64(w), eps, f64(tables[0]), f64(tables[1]), tables[2].cpu().numpy(), pairing)
    within(got, dx, np.abs(dx) * 2.0 ** -8 + mag * 2.0 ** -17)
    if w is None:
        assert got_w is None
    else:
        assert got_w.dtype == torch.float32
        rows = x.numel() // x.shape[-1]
        within(got_w, dw, w_mag * ((rows + 80) * 2.0 ** -24 + 2.0 ** -17))


CASES = [  # B, S, H, Hkv, d, layout, axis dims, pairing, first position, weights, eps
    (1, 1, 1, 1, 128, "bshd", (128,), "adjacent", 0, "fp32", EPS),
    (2, 37, 4, 2, 64, "bhsd", (32, 16), "adjacent", 5, "bf16", EPS),
    (1, 130, 12, 12, 128, "bshd", (44, 42, 42), "adjacent", 0, "fp32", 1e-5),
    (3, 33, 5, 1, 128, "bshd", (32, 48, 48), "halves", -40, "bf16", EPS),
    (2, 61, 6, 3, 64, "bhsd", (32,), "halves", 1000000, "none", EPS),
    (1, 517, 32, 8, 128, "bshd", (128,), "halves", 2 ** 31 - 600, "bf16", 0.0),
    (1, 700, 1, 1, 64, "bshd", (2,), "adjacent", -2 ** 31, "fp32", 1.0),
    (2, 9, 71, 1, 128, "bhsd", (16, 16, 16, 16), "halves", 7, "fp32", EPS),
    (1, 1021, 17, 3, 64, "bshd", (64,), "halves", 0, "bf16", EPS),
    (1, 900, 13, 5, 128, "bshd", (64,), "adjacent", 0, "fp32", EPS),       # heads in two parts
    (3, 1201, 7, 2, 128, "bhsd", (64, 32), "adjacent", 3, "fp32", EPS),    # several tokens a warp, across batch entries
    (1, 5003, 3, 1, 64, "bshd", (48,), "halves", -9, "bf16", EPS),
]
ids = lambda c: "B%d_S%d_H%d_%d_d%d_%s_%s_%s_%s" % (*c[:6], "x".join(map(str, c[6])), c[7], c[9])      # noqa: E731


def tables_of(attn, case, per_batch=False):
    B, S, dims, first = case[0], case[1], case[6], case[8]
    freqs, axes = attn.rope_freqs(dims)
    g = torch.Generator().manual_seed(B * S)
    n = (B,) if per_batch else ()
    p = [(first + torch.arange(S).expand(*n, S) if a == 0 else torch.randint(-50, 4000, (*n, S), generator=g)) for a in range(len(dims))]
    return torch.stack(p).to(torch.int32).cuda(), freqs, axes


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward_and_gradient(attn, case):
    B, S, H, Hkv, d, layout, dims, pairing, first, kind, eps = case
    tables = tables_of(attn, case)
    to = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2).contiguous())
    x = [draw(B, S, H, d, seed=1, scale=3), draw(B, S, Hkv, d, seed=2, scale=0.1)]
    dy = [draw(B, S, H, d, seed=3), draw(B, S, Hkv, d, seed=4, scale=5)]
    w = [weight(d, kind, 5), weight(d, kind, 6)]
    out = attn.attn_norm_rope(to(x[0]), to(x[1]), *w, *tables, eps=eps, layout=layout, pairing=pairing)
    back = attn.attn_norm_rope_bwd(to(dy[0]), to(dy[1]), to(x[0]), to(x[1]), *w, *tables, eps=eps, layout=layout, pairing=pairing)
    again = attn.attn_norm_rope_bwd(to(dy[0]), to(dy[1]), to(x[0]), to(x[1]), *w, *tables, eps=eps, layout=layout, pairing=pairing)
    for t in range(2):
        check_forward(to(out[t]), x[t], w[t], eps, tables, pairing)
        check_backward(to(back[t]), back[2 + t], dy[t], x[t], w[t], eps, tables, pairing)
        assert torch.equal(back[t], again[t]) and (w[t] is None or torch.equal(back[2 + t], again[2 + t]))
    assert attn.cache_device_status() == (0, 0)


@pytest.mark.parametrize("d,layout,pairing", [(128, "bshd", "halves"), (64, "bhsd", "adjacent"), (128, "bhsd", "adjacent")])
def test_views_of_a_projection_in_place_and_positions_by_sequence(attn, d, layout, pairing):
    B, S, H, Hkv = 3, 45, 6, 2
    tables = tables_of(attn, (B, S, H, Hkv, d, layout, (d // 2,), pairing, 3), per_batch=True)
    w = [weight(d, "bf16", 1), weight(d, "bf16", 2)]
    to = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2))

    def cut(buffer):
        return [to(buffer[:, :, :H]), to(buffer[:, :, H:H + Hkv])]
    buf, grads = draw(B, S, H + 2 * Hkv, d, seed=3), draw(B, S, H + 2 * Hkv, d, seed=4)
    rest = buf[:, :, H + Hkv:].clone(), grads[:, :, H + Hkv:].clone()
    x, dy = [t.clone() for t in cut(buf)], [t.clone() for t in cut(grads)]
    q, k = cut(grads)                               # the gradients in place of the outputs'
    back = attn.attn_norm_rope_bwd(q, k, *cut(buf), *w, *tables, layout=layout, pairing=pairing, dq_out=q, dk_out=k)
    assert back[0] is q and back[1] is k
    q, k = cut(buf)
    out = attn.attn_norm_rope(q, k, *w, *tables, layout=layout, pairing=pairing, q_out=q, k_out=k)
    assert out[0] is q and out[1] is k
    for t in range(2):
        check_forward(to(out[t]), to(x[t]), w[t], EPS, tables, pairing)
        check_backward(to(back[t]), back[2 + t], to(dy[t]), to(x[t]), w[t], EPS, tables, pairing)
    assert torch.equal(buf[:, :, H + Hkv:], rest[0]) and torch.equal(grads[:, :, H + Hkv:], rest[1])


def test_packed_queries_alone_and_no_rotation(attn):
    x, dy, w = draw(321, 7, 128, seed=1), draw(321, 7, 128, seed=2), weight(128, "fp32", 3)
    none = (torch.zeros((1, 321)), torch.zeros(0, dtype=torch.float64), torch.zeros(0, dtype=torch.int32))
    check_forward(attn.attn_norm_rope(x, None, w), x, w, EPS, none, "adjacent")
    dx, dw = attn.attn_norm_rope_bwd(dy, None, x, None, w, pairing="halves")
    check_backward(dx, dw, dy, x, w, EPS, none, "adjacent")
    dx, dw = attn.attn_norm_rope_bwd(dy, None, x, None)
    check_backward(dx, dw, dy, x, None, EPS, none, "adjacent")


def test_gradient_against_differences_of_the_forward(attn):
    """Directional differences of the kernel's own forward, whose bf16 outputs are off by 2^-8 / sqrt(12)-ish of each element
    at random: a loss over n elements by their root sum of squares, four of those taken."""
    B, S, H, d = 1, 257, 8, 128
    tables = tables_of(attn, (B, S, H, 0, d, "bshd", (128,), "halves", 11))
    x, dy, w = draw(B, S, H, d, seed=1), draw(B, S, H, d, seed=2), weight(d, "fp32", 3)
    dx, dw = attn.attn_norm_rope_bwd(dy, None, x, None, w, None, *tables, pairing="halves")
    run = lambda x, w: attn.attn_norm_rope(x, None, w, None, *tables, pairing="halves").double()     # noqa: E731
    h = 0.25                                         # exact in bf16 steps of x; the norm's curvature is in the bound
    u = torch.sign(draw(B, S, H, d, seed=4).float()) * 2.0 ** -5
    up, down = (x.float() + u).to(torch.bfloat16), (x.float() - u).to(torch.bfloat16)
    step = (up.double() - down.double())
    diff = run(up, w) - run(down, w)
    got, want = float((diff * dy.double()).sum()), float((dx.double() * step).sum())
    noise = 4 * float(((run(x, w) * dy.double() * 2.0 ** -8) ** 2).sum().sqrt()) * 2 ** 0.5
    # third order: |u|^3 / 6 times third derivatives of n(x) (below 15 / size^3 with |x| about its size of 1): summed at random
    third = 4 * 15 / 6 * 2.0 ** -15 * 2 * float((dy.double() ** 2).sum().sqrt())
    assert abs(got - want) <= noise + third, (got, want, noise, third)
    v = torch.randn(d, generator=torch.Generator().manual_seed(5)).cuda() * h
    diff = run(x, w + v) - run(x, w - v)             # linear in the weights
    got, want = float((diff * dy.double()).sum()), float((dw.double() * 2 * v.double()).sum())
    noise = 4 * float(((run(x, w.abs() + v.abs()) * dy.double() * 2.0 ** -8) ** 2).sum().sqrt()) * 2 ** 0.5
    assert abs(got - want) <= noise, (got, want, noise)


def test_heads_of_zeros_infinities_and_nan(attn):
    x, dy, w = draw(5, 9, 64, seed=1), draw(5, 9, 64, seed=2), weight(64, "fp32", 3)
    clean, (_, dw_clean) = attn.attn_norm_rope(x, None, w), attn.attn_norm_rope_bwd(dy, None, x, None, w)
    x[1, 2] = 0
    x[2, 3, 7] = float("inf")
    x[3, 4, 8] = float("nan")
    x[4, 5] *= 2.0 ** 100                            # the squares' sum overflows
    y = attn.attn_norm_rope(x, None, w)
    dx, dw = attn.attn_norm_rope_bwd(dy, None, x, None, w)
    assert not y[1, 2].any()
    assert y[2, 3, 7].isnan() and not y[2, 3, :7].any() and y[3, 4].isnan().all() and not y[4, 5].any()
    keep = torch.ones((5, 9), dtype=torch.bool)
    keep[[1, 2, 3, 4], [2, 3, 4, 5]] = False
    assert torch.equal(y[keep.cuda()], clean[keep.cuda()]) and dw.isnan().all() and dw_clean.isfinite().all()
    assert dx[keep.cuda()].isfinite().all()
    # a head of zeros: its gradient is the weighted one over sqrt(eps)
    want = dy[1, 2].double() * w.double() / EPS ** 0.5
    assert torch.all((dx[1, 2].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -18))
    # infinite frequencies reach their pairs only
    pos, (freqs, axes) = torch.ones((1, 5), dtype=torch.int32, device="cuda"), attn.rope_freqs((32,))
    freqs[3] = float("inf")
    y = attn.attn_norm_rope(draw(5, 9, 64, seed=1), None, w, None, pos, freqs, axes)
    bad = y.isnan().all(0).all(0)
    assert bad.nonzero().flatten().tolist() == [6, 7] and int(y.isnan().sum()) == 2 * 45


def test_bad_axes_write_nothing(attn):
    x, dy, w = draw(40, 4, 128, seed=1), draw(40, 4, 128, seed=2), weight(128, "bf16", 3)
    freqs, axes = attn.rope_freqs((64, 64))
    pos = torch.zeros((1, 40), dtype=torch.int32, device="cuda")        # one axis, the table names two
    out, dw = torch.full_like(x, 7.0), torch.full((128,), 7.0, device="cuda")
    attn.attn_norm_rope(x, None, w, None, pos, freqs, axes, q_out=out)
    assert attn.cache_device_status() == (1, 20) and (out == 7).all()
    attn.attn_norm_rope_bwd(dy, None, x, None, w, None, pos, freqs, axes, dq_out=out, dq_weight=dw)
    assert attn.cache_device_status() == (1, 20) and (out == 7).all() and (dw == 7).all()


def test_no_tokens(attn):
    x, w = draw(0, 4, 128), weight(128, "fp32", 1)
    assert attn.attn_norm_rope(x, None, w).shape == x.shape
    dx, dw = attn.attn_norm_rope_bwd(x, None, x, None, w)
    assert dx.shape == x.shape and not dw.any()


def test_workspace_is_the_caller_s_and_outputs_stay_in_bounds(attn):
    B, S, H, Hkv, d = 1, 77, 3, 2, 64
    tables = tables_of(attn, (B, S, H, Hkv, d, "bshd", (64,), "halves", 0))
    x, dy = [draw(B, S, H, d, seed=1), draw(B, S, Hkv, d, seed=2)], [draw(B, S, H, d, seed=3), draw(B, S, Hkv, d, seed=4)]
    w = [weight(d, "fp32", 5), weight(d, "fp32", 6)]
    want = attn.attn_norm_rope_bwd(*dy, *x, *w, *tables, pairing="halves")
    a = attn.NormRopeBwdArgs()
    a.B, a.S, a.H, a.Hkv, a.d, a.k, a.num_axes = B, S, H, Hkv, d, 16, 1
    need = int(attn.load().attn_norm_rope_bwd_workspace_size(ctypes.byref(a)))
    assert need > 0
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    rooms = [torch.full((128 + n,), 3.0, dtype=t, device="cuda") for n, t in
             ((S * H * d, torch.bfloat16), (S * Hkv * d, torch.bfloat16), (d, torch.float32), (d, torch.float32))]
    outs = [rooms[0][64:-64].view(B, S, H, d), rooms[1][64:-64].view(B, S, Hkv, d), rooms[2][64:-64], rooms[3][64:-64]]
    got = attn.attn_norm_rope_bwd(*dy, *x, *w, *tables, pairing="halves", dq_out=outs[0], dk_out=outs[1], dq_weight=outs[2],
                                  dk_weight=outs[3], workspace=ws[:need])
    assert all(torch.equal(g, e) for g, e in zip(got, want))
    assert all((r[:64] == 3).all() and (r[-64:] == 3).all() for r in rooms) and (ws[need:] == 0xFF).all()
    with pytest.raises(attn.AttnError):
        attn.attn_norm_rope_bwd(*dy, *x, *w, *tables, pairing="halves", workspace=ws[:need - 16])


@pytest.mark.parametrize("d,page,pairing,kind,queries", [(128, 16, "halves", "bf16", True), (64, 7, "adjacent", "fp32", True),
                                                         (128, 1, "adjacent", "none", False)])
def test_append(attn, d, page, pairing, kind, queries):
    total, H, Hkv, pages = 93, 5, 3, 40 if page > 2 else 300
    g = torch.Generator().manual_seed(d + page)
    freqs, axes = attn.rope_freqs((d // 2,))
    pos = torch.randint(-5, 100000, (1, total), generator=g).to(torch.int32).cuda()
    x = draw(total, H + 2 * Hkv, d, seed=1, scale=2)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    w = [weight(d, kind, 2) if queries else None, weight(d, kind, 3)]
    kc, vc = draw(pages, page, Hkv, d, seed=4), draw(pages, page, Hkv, d, seed=5)
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.randperm(pages * page, generator=g)[:total]
    slots[[0, 50, 92]] = -1
    slots[[7, 33]] = torch.tensor([pages * page, -2])
    slots[9] = 2 ** 40
    room = torch.full((total, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    out = attn.attn_norm_rope_append(k, v, kc, vc, slots.cuda(), q=q if queries else None, q_out=room if queries else None,
                                     q_weight=w[0], k_weight=w[1], positions=pos, freqs=freqs, axes=axes, pairing=pairing)
    assert attn.cache_device_status() == (1, 24)
    tables = (pos, freqs, axes)
    put = (slots >= 0) & (slots < pages * page)
    got = kc.view(-1, Hkv, d)[slots[put].cuda()]
    check_forward(got, k[put.cuda()], w[1], EPS, (pos[:, put.cuda()], freqs, axes), pairing)
    assert torch.equal(vc.view(-1, Hkv, d)[slots[put].cuda()], v[put.cuda()])
    left = torch.ones(pages * page, dtype=torch.bool)
    left[slots[put]] = False
    assert torch.equal(kc.view(-1, Hkv, d)[left.cuda()], k0.view(-1, Hkv, d)[left.cuda()])
    assert torch.equal(vc.view(-1, Hkv, d)[left.cuda()], v0.view(-1, Hkv, d)[left.cuda()])
    if not queries:
        assert out is None
        return
    seen = (slots != -1).cuda()
    assert (out[~seen] == 9).all()
    check_forward(out[seen], q[seen], w[0], EPS, (tables[0][:, seen], freqs, axes), pairing)


def test_append_equals_the_norm_and_many_heads(attn):
    """Split over blocks by heads (few tokens) or not (many), the same bits as attn_norm_rope."""
    for total, H, Hkv in ((1, 40, 8), (3, 71, 5), (1500, 4, 1)):
        freqs, axes = attn.rope_freqs((44, 42, 42))
        pos = torch.randint(0, 999, (3, total), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        x, w = draw(total, H + 2 * Hkv, 128, seed=total), [weight(128, "bf16", 2), weight(128, "bf16", 3)]
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        kc, vc = (torch.zeros((total, 2, Hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        slots = torch.arange(total, device="cuda") * 2 + 1
        out = attn.attn_norm_rope_append(k, v, kc, vc, slots, q=q, q_weight=w[0], k_weight=w[1], positions=pos, freqs=freqs, axes=axes)
        want = attn.attn_norm_rope(q, k, *w, pos, freqs, axes)
        assert torch.equal(out, want[0]) and torch.equal(kc[:, 1], want[1]) and torch.equal(vc[:, 1], v)
        assert not kc[:, 0].any() and attn.cache_device_status() == (0, 0)


def test_captured(attn):
    """A graph of both directions, replayed on new data; eager calls between and after."""
    tables = tables_of(attn, (1, 50, 4, 2, 128, "bshd", (128,), "halves", 0))
    w = [weight(128, "fp32", 1), weight(128, "fp32", 2)]
    x, dy = [draw(1, 50, h, 128, seed=h) for h in (4, 2)], [draw(1, 50, h, 128, seed=9 + h) for h in (4, 2)]

    def step():
        return [*attn.attn_norm_rope(*x, *w, *tables, pairing="halves"),
                *attn.attn_norm_rope_bwd(*dy, *x, *w, *tables, pairing="halves")]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (20, 30):
        for t, h in zip(x + dy, (4, 2, 4, 2)):
            t.copy_(draw(1, 50, h, 128, seed=seed + h))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
