"""Attention of one new token over a paged cache (attn_paged_decode) against the fp64 oracle, and the
attention weights that it accumulates (needs a GB300).

Outputs go by the forward's criteria (tests/parity.py, lse as in the causal tests).  Weights: the
fp32 logit is off by at most 2 d 2^-24 A_i (A_i = max_j sum |q_i k_j| / sqrt(d)), which moves a weight by that
share of itself, the exponentials and their sum by 2^-18, and the fp32 sums by 2^-22.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tests import parity
from tests.test_gpu_canaries import guarded, guards_intact
from tests.test_gpu_causal_gqa import check_lse
from tests.test_gpu_paged import build_cache
from tests.test_gpu_varlen import lse_scale, offsets, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


def status_ok(attn):
    assert attn.cache_device_status() == (0, 0)


def cuda(x, dtype=np.int32):
    return torch.as_tensor(np.asarray(x, dtype=dtype)).cuda()


def reference_weights(q, k, cu_k, G):
    """fp64 softmax weights per key and K/V head, [Hkv, total_k], and their tolerance's relative part."""
    B, H, d = q.shape
    Hkv = H // G
    w, rel = np.zeros((Hkv, k.shape[0])), np.zeros((Hkv, k.shape[0]))
    qa, ka = q.float().numpy().astype(np.float64), k.float().numpy().astype(np.float64)
    for b in range(B):
        s = slice(int(cu_k[b]), int(cu_k[b + 1]))
        if s.stop == s.start:
            continue
        for h in range(H):
            x = ka[s, h // G] @ qa[b, h] / np.sqrt(d)
            a = np.max(np.abs(ka[s, h // G]) @ np.abs(qa[b, h])) / np.sqrt(d)
            e = np.exp(x - x.max())
            w[h // G, s] += e / e.sum()
            rel[h // G, s] = np.maximum(rel[h // G, s], 2 * d * 2.0 ** -24 * a + 2.0 ** -18)
    return w, rel


def run(attn, q, kc, vc, lens, table, **kw):
    o, lse = attn.attn_paged_decode(q.cuda(), kc.cuda(), vc.cuda(), cuda(lens), cuda(table), return_lse=True, **kw)
    torch.cuda.synchronize()
    return o, lse


def check(attn, lens, H, Hkv, d, P, mode="rtne", seed=0, weights=False, sigma=1.0):
    B = len(lens)
    q, k, v = packed(B, sum(lens), H, Hkv, d, seed=seed, sigma=sigma)
    kc, vc, table = build_cache(k, v, lens, P, seed=seed + 1)
    acc = None
    if weights:
        start = torch.rand((B, Hkv, table.shape[1] * P), generator=torch.Generator().manual_seed(seed))
        acc = start.cuda()
    o, lse = run(attn, q, kc, vc, lens, table, round=mode, weights=acc)
    status_ok(attn)
    cu = offsets([1] * B)
    ref = oracle.attention_varlen(q, k, v, cu, offsets(lens), mode, want_a=True, want_lse=True)
    ob = o.cpu().view(torch.int16).numpy().view(np.uint16)
    res = parity.compare(ob.reshape(-1, d), ref["o_bits"].reshape(-1, d), ref["a"].reshape(-1, d))
    assert res["ok"], res
    check_lse(lse.cpu().numpy().T.reshape(-1), ref["lse"].reshape(-1), lse_scale(q, k, cu, offsets(lens)).reshape(-1))
    if weights:
        w, rel = reference_weights(q, k, offsets(lens), H // Hkv)
        got, old, c = acc.cpu().numpy().astype(np.float64), start.numpy().astype(np.float64), offsets(lens)
        for b, n in enumerate(lens):
            ref_w = w[:, c[b]:c[b + 1]]
            tol = ref_w * rel[:, c[b]:c[b + 1]] + 2.0 ** -22 * (old[b, :, :n] + ref_w)
            assert np.all(np.abs(got[b, :, :n] - old[b, :, :n] - ref_w) <= tol)
            assert np.array_equal(got[b, :, n:], old[b, :, n:])
    return o, lse


CASES = [  # lens, H, Hkv, d, page size, mode
    ([1], 1, 1, 128, 16, "rtne"),
    ([513], 8, 2, 64, 16, "rtne"),
    ([1, 2, 15, 16, 17, 127, 128, 129, 255, 300], 4, 2, 128, 24, "rtne"),
    ([0, 700, 0, 3, 0], 4, 4, 128, 1, "rtna"),
    ([1023, 17, 400], 10, 2, 128, 64, "rtz"),
    ([640, 129], 32, 2, 64, 128, "rtne"),            # 16 query heads a K/V head
    ([300, 77], 27, 1, 128, 16, "rtne"),             # an odd group past 16
    ([200, 5], 71, 1, 64, 48, "rtne"),               # a group past 32: the keys are read for each 32 heads
    ([90, 260], 80, 2, 128, 256, "rtz"),
    ([3000], 8, 8, 128, 256, "rtne"),
    ([37] * 80, 6, 3, 64, 16, "rtne"),
    ([3, 0, 130, 1] * 500, 2, 2, 64, 8, "rtne"),     # more sequences than a block's threads
]


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "n%d_H%d_%d_d%d_P%d_%s" % (
    len(c[0]), c[1], c[2], c[3], c[4], c[5]))
def test_decode_matches_oracle(attn, case, weights):
    lens, H, Hkv, d, P, mode = case
    check(attn, lens, H, Hkv, d, P, mode, seed=100 + P, weights=weights)


def test_few_short_rows_and_their_neighbours_split(attn):
    # the same sequences with a table that has room for more keys: split rows against whole ones
    lens, P, d = [600, 1, 0, 129], 16, 128
    q, k, v = packed(4, sum(lens), 8, 2, d, seed=15)
    kc, vc, table = build_cache(k, v, lens, P, seed=16)
    wide = np.concatenate([table, np.full((4, 200), -5, dtype=table.dtype)], axis=1)
    a, b = run(attn, q, kc, vc, lens, table), run(attn, q, kc, vc, lens, wide)
    status_ok(attn)
    assert torch.isnan(a[0][2]).all() and torch.isnan(b[0][2]).all()
    assert torch.isneginf(a[1][2]).all() and torch.isneginf(b[1][2]).all()
    used = [0, 1, 3]
    # nearly equal values, each rounded by half a step (2^-8) at most
    assert ((a[0][used].float() - b[0][used].float()).abs() <= 2.0 ** -7 * b[0][used].float().abs() + 1e-5).all()
    assert torch.allclose(a[1][used], b[1][used], rtol=0, atol=1e-5)
    o = torch.full((4, 8, d), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = table.copy()
    bad[0, 3] = kc.shape[0]
    attn.attn_paged_decode(q.cuda(), kc.cuda(), vc.cuda(), cuda([600, -1, 0, table.shape[1] * P + 1]), cuda(bad), o=o)
    assert attn.cache_device_status() == (1, 22)
    assert (o[[0, 1, 3]] == 7.0).all() and torch.isnan(o[2]).all()


def test_peaked_rows(attn):
    # logits of deviation 16: the running maximum moves far, most weights underflow
    check(attn, [2000, 999], 8, 2, 128, 16, seed=7, weights=True, sigma=4.0)


def test_same_as_the_paged_forward_up_to_rounding(attn):
    lens, H, Hkv, d, P = [1000, 129, 1], 8, 2, 128, 128
    q, k, v = packed(3, sum(lens), H, Hkv, d, seed=5)
    kc, vc, table = build_cache(k, v, lens, P, seed=6)
    o, lse = run(attn, q, kc, vc, lens, table)
    of, lf = attn.attn_fwd_paged(q.cuda(), kc.cuda(), vc.cuda(), cuda(offsets([1] * 3)), cuda(lens), cuda(table),
                                 return_lse=True, causal=True, pack_heads=True)
    # both within the oracle's bound of 2^-8 A, A <= max |v|
    assert ((o.float() - of.float()).abs() <= 2.0 ** -7 * v.float().abs().max().item()).all()
    assert torch.allclose(lse.T, lf, rtol=0, atol=1e-3)
    status_ok(attn)


def test_repeats_bit_for_bit_and_reads_nothing_past_the_lengths(attn):
    lens, P = [700, 33, 260], 16
    q, k, v = packed(3, sum(lens), 8, 2, 128, seed=11)
    kc, vc, table = build_cache(k, v, lens, P, seed=12)                  # junk in every unused slot
    kz, vz, tz = build_cache(k, v, lens, P, seed=12, stale=False)
    w = torch.zeros((3, 2, table.shape[1] * P), device="cuda")
    w2 = torch.zeros_like(w)
    a = run(attn, q, kc, vc, lens, table, weights=w)
    b = run(attn, q, kz, vz, lens, tz, weights=w2)
    table = table.copy()
    for i, n in enumerate(lens):
        table[i, -(-n // P):] = -7                                       # entries past the last page are not read
    c = run(attn, q, kc, vc, lens, table)
    for x in (b, c):
        assert torch.equal(a[0].view(torch.int16), x[0].view(torch.int16))
        assert torch.equal(a[1], x[1])
    assert torch.equal(w, w2)
    status_ok(attn)


def test_non_finite_values_follow_the_forward(attn):
    lens, H, Hkv, d, P = [300, 300, 300, 300, 40], 4, 2, 128, 16
    q, k, v = packed(5, sum(lens), H, Hkv, d, seed=21)
    k[10, 0, 3] = float("nan")                     # sequence 0, K/V head 0: a NaN logit
    k[300 + 5] = 0
    k[300 + 5, 0, 0] = float("inf")                # +-inf logits by q's sign
    v[600 + 299, 1, 7] = float("inf")              # an infinite value with a positive weight
    v[600 + 12, 1, 7] = float("-inf")
    v[600 + 12, 1, 9] = float("-inf")
    k[900:1200] = 0
    k[900:1200, :, 0] = float("-inf")              # every logit infinite
    q[3, :, 0] = q[3, :, 0].abs() + 1
    kc, vc, table = build_cache(k, v, lens, P, seed=22)
    o, lse = run(attn, q, kc, vc, lens, table)
    status_ok(attn)
    cu = offsets([1] * 5)
    ref = oracle.attention_varlen(q, k, v, cu, offsets(lens), "rtne", want_a=True, want_lse=True)
    ob = o.cpu().view(torch.int16).numpy().view(np.uint16)
    res = parity.compare(ob.reshape(-1, d), ref["o_bits"].reshape(-1, d), ref["a"].reshape(-1, d))
    assert res["ok"] and res["n_nonfinite"] > 0, res
    got, want = lse.cpu().numpy().T.reshape(-1), ref["lse"].reshape(-1)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    assert np.allclose(got[fin], want[fin], rtol=0, atol=1e-3)


def test_tiny_weights_of_infinite_values(attn):
    # a key whose weight underflows still carries an infinite value, wherever its part of the row lies
    n, d = 4000, 128
    q, k, v = packed(1, n, 1, 1, d, seed=31)
    q[:] = 8.0
    k[:] = 0.0
    k[0] = 8.0                                      # logit 724, all others 0: weights of 2^-1000
    v[3999, 0, 5] = float("inf")
    v[1, 0, 6] = float("-inf")
    kc, vc, table = build_cache(k, v, [n], 16, seed=32)
    o, _ = run(attn, q, kc, vc, [n], table)
    assert o[0, 0, 5] == float("inf") and o[0, 0, 6] == float("-inf")
    keep = [x for x in range(d) if x not in (5, 6)]
    assert torch.equal(o[0, 0, keep].cpu(), v[0, 0, keep])
    status_ok(attn)


def test_a_lone_key_returns_its_value_in_every_mode(attn):
    q, k, v = packed(1, 1, 8, 2, 128, seed=41, sigma=3.0)
    kc, vc, table = build_cache(k, v, [1], 16, seed=42)
    for mode in ("rtne", "rtna", "rtz"):
        o, _ = run(attn, q, kc, vc, [1], table, round=mode)
        assert torch.equal(o[0].cpu(), v[0].repeat_interleave(4, 0))


def test_bad_lengths_and_pages_leave_their_sequences_alone(attn):
    lens, H, Hkv, d, P = [200, 260, 100, 40, 30], 4, 2, 128, 16
    q, k, v = packed(5, sum(lens), H, Hkv, d, seed=51)
    kc, vc, table = build_cache(k, v, lens, P, seed=52)
    good, gl = run(attn, q, kc, vc, lens, table)
    table, said = table.copy(), list(lens)
    table[1, 9] = kc.shape[0]                       # one page past the cache
    table[3, 0] = -1
    said[2] = table.shape[1] * P + 1                # longer than the table
    said[4] = -3
    o = torch.full((5, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, H), 9.0, device="cuda")
    w = torch.zeros((5, Hkv, table.shape[1] * P), device="cuda")
    attn.attn_paged_decode(q.cuda(), kc.cuda(), vc.cuda(), cuda(said), cuda(table), o=o, lse=lse, weights=w)
    assert attn.cache_device_status() == (1, 22)
    assert (o[1:] == 7.0).all() and (lse[1:] == 9.0).all() and not w[1:].any()
    # sequence 0's parts lie elsewhere than before: the same up to rounding
    assert ((o[0].float() - good[0].float()).abs() <= 2.0 ** -7 * v.float().abs().max().item()).all()
    assert torch.allclose(lse[0], gl[0], rtol=0, atol=1e-4)
    assert abs(w[0].sum().item() - H) < 1e-3        # each query head's weights sum to one
    status_ok(attn)


def test_shared_pages(attn):
    P, d = 16, 128
    q, k, v = packed(2, 40, 4, 2, d, seed=61)
    kc, vc, table = build_cache(k, v, [40], P, seed=62)
    both = np.concatenate([table, table])
    o, _ = run(attn, q, kc, vc, [40, 33], both)
    for b, n in enumerate([40, 33]):
        ref = oracle.attention_varlen(q[b:b + 1], k[:n], v[:n], offsets([1]), offsets([n]), "rtne", want_a=True)
        res = parity.compare(o[b].cpu().view(torch.int16).numpy().view(np.uint16).reshape(-1, d),
                             ref["o_bits"].reshape(-1, d), ref["a"].reshape(-1, d))
        assert res["ok"], res


def test_guards_and_workspace_contents(attn):
    lens, H, Hkv, d, P = [333, 900, 5], 10, 2, 128, 16
    q, k, v = packed(3, sum(lens), H, Hkv, d, seed=71)
    kc, vc, table = build_cache(k, v, lens, P, seed=72)
    want, wl = run(attn, q, kc, vc, lens, table)
    room = table.shape[1] * P
    a = attn.DecodeArgs()
    a.B, a.H, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d = 3, H, Hkv, kc.shape[0], P, table.shape[1], d
    a.weights = 16
    need = int(attn.load().attn_paged_decode_workspace_size(ctypes.byref(a)))
    ob, o = guarded(3 * H * d, "bf16")
    lb, lse = guarded(3 * H, "f32")
    wb, w = guarded(3 * Hkv * room, "f32")
    sb, ws = guarded(need, "ws")
    w.zero_()
    attn.attn_paged_decode(q.cuda(), kc.cuda(), vc.cuda(), cuda(lens), cuda(table), o=o.view(3, H, d),
                           lse=lse.view(3, H), weights=w.view(3, Hkv, room), workspace=ws)
    torch.cuda.synchronize()
    assert guards_intact(ob, "bf16") and guards_intact(lb, "f32") and guards_intact(wb, "f32") and guards_intact(sb, "ws")
    assert torch.equal(o.view(3, H, d).view(torch.int16), want.view(torch.int16)) and torch.equal(lse.view(3, H), wl)
    status_ok(attn)


def test_two_streams_with_workspaces_of_their_own_and_a_graph(attn):
    lens, P = [900, 333], 16
    q, k, v = packed(2, sum(lens), 8, 2, 128, seed=81)
    kc, vc, table = build_cache(k, v, lens, P, seed=82)
    dev = [q.cuda(), kc.cuda(), vc.cuda(), cuda(lens), cuda(table)]
    want, wl = attn.attn_paged_decode(*dev, return_lse=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        outs.append(attn.attn_paged_decode(*dev, return_lse=True, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
    graphs, kept = [], []
    for _ in range(2):                               # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(attn.attn_paged_decode(*dev, return_lse=True))
        graphs.append(g)
    dev[3].copy_(cuda([500, 1]))                     # the lengths are read at replay
    want, wl = attn.attn_paged_decode(*dev, return_lse=True)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, lse in kept:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
    status_ok(attn)


def test_what_the_binding_refuses(attn):
    q, k, v = packed(2, 20, 4, 2, 64, seed=91)
    kc, vc, table = build_cache(k, v, [10, 10], 16, seed=92)
    q, kc, vc, n, t = q.cuda(), kc.cuda(), vc.cuda(), cuda([10, 10]), cuda(table)
    room = table.shape[1] * 16
    w = torch.zeros((2, 2, room), device="cuda")
    call = attn.attn_paged_decode
    for f, error in (
            (lambda: call(q.float(), kc, vc, n, t), TypeError),
            (lambda: call(q[:1].contiguous(), kc, vc, n, t), ValueError),
            (lambda: call(q[:, :3].contiguous(), kc, vc, n, t), ValueError),
            (lambda: call(q[:, :, :32].contiguous(), kc, vc, n, t), ValueError),
            (lambda: call(q.transpose(0, 1), kc, vc, n, t), ValueError),
            (lambda: call(q, kc, vc[:1], n, t), ValueError),
            (lambda: call(q, kc, vc, n.long(), t), TypeError),
            (lambda: call(q, kc, vc, n, t, round="up"), ValueError),
            (lambda: call(q, kc, vc, n, t, weights=w[:, :1].contiguous()), ValueError),
            (lambda: call(q, kc, vc, n, t, lse=torch.zeros((4, 2), device="cuda")), ValueError),
            (lambda: call(q, kc, vc, n, t, o=q), attn.AttnError),
            (lambda: call(q, kc, vc, n, t, weights=w, workspace=torch.empty(64, device="cuda")), attn.AttnError)):
        with pytest.raises(error):
            f()
    status_ok(attn)
