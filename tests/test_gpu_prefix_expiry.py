"""A wait that runs out in the shared prefix's kernel (needs a GB300).

The hook ATTN_TEST_WITHHOLD_O_READY makes the first CTA skip the signal that its first share's output accumulator of tile 0 is
complete, so that the wait for it expires under a 50 ms limit.  Nothing faults, traps or spins without a bound.  The
CTA then owes parts of some rows: those rows are not written, whatever the workspace held before; all others are as in a normal call, and the
device stays usable.
"""
import ctypes

import pytest
import torch

from tests.test_gpu_prefix_decode import Batch, alone, attn, draw  # noqa: F401

pytestmark = pytest.mark.gpu

WITHHOLD, TIMEOUT, SITE = 1, 8, 26


@pytest.mark.parametrize("own,H,Hkv,d,page,prefix", [
    ([5, 0, 200] * 8, 32, 8, 128, 16, 12000),        # one tile of rows, split over many CTAs
    ([5, 0, 200] * 8, 32, 8, 64, 16, 12000),
    ([5, 0, 90] * 20, 32, 4, 128, 48, 6000),         # two tiles
    ([5, 0, 9] * 300, 8, 2, 128, 16, 300),           # several shares a CTA
    ([5, 0, 9] * 300, 8, 2, 64, 16, 300),
])
def test_rows_that_an_expired_wait_cuts_off_are_not_written(attn, own, H, Hkv, d, page, prefix):  # noqa: F811
    x = Batch(own, H, Hkv, d, page, prefix, seed=len(own))
    assert not alone(x)
    B, G = len(own), H // Hkv
    a = attn.DecodeArgs()
    a.B, a.H, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d = B, H, Hkv, len(x.k), page, x.table.shape[1], d
    ws = torch.empty(int(attn.load().attn_paged_prefix_decode_workspace_size(ctypes.byref(a), prefix)), dtype=torch.uint8, device="cuda")
    want = x.call(attn, workspace=ws)
    q = x.q
    x.q = draw(B, H, d, seed=99)
    x.call(attn, workspace=ws)                       # (what the workspace holds when the wait runs out: another step's parts)
    x.q = q
    assert attn.cache_device_status() == (0, 0)
    o, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    x.call(attn, o=o, lse=lse, workspace=ws, wait_limit_ms=50, test_hooks=WITHHOLD)
    assert attn.cache_device_status() == (TIMEOUT, SITE)
    assert attn.cache_device_status() == (0, 0)                  # read and cleared
    kept = (o == 7).all(2) & (lse == 7)
    same = (o.view(torch.int16) == want[0].view(torch.int16)).all(2) & (lse == want[1])
    assert (kept | same).all()
    # tile 0 of the first CTA's first share: rows 0 .. 127 (sequence, head of the first group) of the first K/V head
    first = torch.zeros(B * G, dtype=torch.bool, device="cuda")
    first[:128] = True
    assert kept[:, :G][first.view(B, G)].all() and same.any()
    got = x.call(attn, workspace=ws)
    assert attn.cache_device_status() == (0, 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_wait_in_the_decoding_kernel_alone(attn):  # noqa: F811
    x = Batch([3, 4], 4, 2, 128, 16, 60)
    assert alone(x)
    want, got = x.call(attn), x.call(attn, wait_limit_ms=50, test_hooks=WITHHOLD)
    assert attn.cache_device_status() == (0, 0) and torch.equal(got[0], want[0])
    with pytest.raises(attn.AttnError):
        x.call(attn, test_hooks=2)
