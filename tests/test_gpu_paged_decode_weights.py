"""Accumulated weights of attn_paged_decode where four neighbouring ones are not a 16-byte access: tables with an odd
number of slots, weights that start at any fp32 (needs a GB300).  Tolerances as in the tests of the call."""
import numpy as np
import pytest
import torch

from tests.test_gpu_canaries import G, guarded, guards_intact
from tests.test_gpu_paged import build_cache
from tests.test_gpu_paged_decode import attn, check, cuda, reference_weights, run, status_ok  # noqa: F401  (a fixture)
from tests.test_gpu_varlen import offsets, packed

pytestmark = pytest.mark.gpu

CASES = [  # lens, H, Hkv, d, page size: rooms of 35, 1001, 903, 385, 651 and 702 slots
    ([35, 1, 0, 34, 17], 6, 3, 64, 5),
    ([1001, 1000, 3], 8, 2, 128, 7),
    ([903, 128, 129, 127, 899], 10, 2, 64, 3),
    ([381, 385], 27, 3, 128, 5),           # an odd group past the eight heads of a pass
    ([651, 650, 20], 80, 2, 64, 21),       # a group past 32
    ([700, 701], 4, 4, 128, 26),           # even, not a multiple of four
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "n%d_H%d_%d_d%d_P%d" % (len(c[0]), *c[1:]))
def test_odd_rooms(attn, case):  # noqa: F811
    lens, H, Hkv, d, P = case
    room = -(-max(lens) // P) * P
    assert room % 4
    check(attn, lens, H, Hkv, d, P, seed=P + H, weights=True)


@pytest.mark.parametrize("lead", [0, 1, 2, 3])
@pytest.mark.parametrize("case", [([500, 129, 1], 8, 2, 128, 16), ([1001, 700], 6, 3, 64, 7)],
                         ids=lambda c: "P%d" % c[4])
def test_weights_at_any_fp32(attn, case, lead):  # noqa: F811
    lens, H, Hkv, d, P = case
    B = len(lens)
    q, k, v = packed(B, sum(lens), H, Hkv, d, seed=P)
    kc, vc, table = build_cache(k, v, lens, P, seed=P + 1)
    shape = (B, Hkv, table.shape[1] * P)
    n = int(np.prod(shape))
    buf, view = guarded(n + 4, "f32")
    w = view[lead:lead + n].view(shape)
    assert (w.data_ptr() % 16) // 4 == lead
    start = torch.rand(shape, generator=torch.Generator().manual_seed(P))
    w.copy_(start)
    plain = torch.zeros(shape, device="cuda").copy_(start)
    o, lse = run(attn, q, kc, vc, lens, table, weights=w)
    o2, lse2 = run(attn, q, kc, vc, lens, table, weights=plain)
    status_ok(attn)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    assert torch.equal(w, plain)                   # the same sums, however they are loaded
    ends = torch.cat([view[:lead], view[lead + n:]]).view(torch.int32)
    assert guards_intact(buf, "f32") and bool((ends == buf.view(torch.int32)[0]).all()) and buf.numel() == n + 4 + 2 * G
    ref, rel = reference_weights(q, k, offsets(lens), H // Hkv)
    got, old, c = w.cpu().numpy().astype(np.float64), start.numpy().astype(np.float64), offsets(lens)
    for b, m in enumerate(lens):
        r = ref[:, c[b]:c[b + 1]]
        tol = r * rel[:, c[b]:c[b + 1]] + 2.0 ** -22 * (old[b, :, :m] + r)
        assert np.all(np.abs(got[b, :, :m] - old[b, :, :m] - r) <= tol)
        assert np.array_equal(got[b, :, m:], old[b, :, m:])


def test_a_refused_sequence_in_an_odd_room(attn):  # noqa: F811
    lens, H, Hkv, d, P = [700, 701, 300], 6, 2, 64, 7
    q, k, v = packed(3, sum(lens), H, Hkv, d, seed=1)
    kc, vc, table = build_cache(k, v, lens, P, seed=2)
    table = table.copy()
    table[1, 90] = -1
    w = torch.full((3, Hkv, table.shape[1] * P), 0.5, device="cuda")
    o = torch.full((3, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    attn.attn_paged_decode(q.cuda(), kc.cuda(), vc.cuda(), cuda(lens), cuda(table), o=o, weights=w)
    assert attn.cache_device_status() == (1, 22)
    assert (o[1] == 7.0).all() and (w[1] == 0.5).all() and (w[0, :, 700:] == 0.5).all() and (w[2, :, 300:] == 0.5).all()
    spent = w.double().sum((1, 2)) - 0.5 * Hkv * table.shape[1] * P
    assert ((spent[[0, 2]] - H).abs() < 1e-3).all()
    status_ok(attn)
