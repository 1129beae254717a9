"""The weights of a shared prefix's keys (attn_paged_prefix_decode): as exact as in attn_paged_decode, whichever kernels the
batch's size sends a call to (needs a GB300).

Keys of two kinds: logit 0, weight 1, values v; and one other logit for each row, weight w in 1/2 .. 1, values -1, twice as many.
Column x has v = 1 + x / 64 (of 64 columns), so that for some columns the sum n (v - 2 w) all but vanishes, and what is left
shows w's own error, which is the same for every key: one bf16 part of w is off by up to 2^-9, and the sum by up to 2^-10 of the
sum of magnitudes A.

Tolerance, derived before the first run.  Two bf16 parts hold w to 2^-16; the logit is one product, exact in fp32, its
scaling 2^-23 of at most 1, the exponential 2^-22; sums of 2,500 products, 16 at a time, 160 * 2^-24 < 2^-16, and as much
for the weights' own sum: below 2^-14 A in all, beside the output's rounding, 2^-8 relative.  An offset that all logits
have (exact in fp32 too) changes no weight but by one factor for all, which the sum has as well.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


@pytest.mark.parametrize("offset", [0, 64, 128])       # up to 1,024 in base 2, and past it
@pytest.mark.parametrize("B,H,Hkv,d,prefix", [
    (4, 8, 8, 128, 600),             # the decoding kernel alone
    (16, 64, 8, 128, 2499),          # one tile of rows
    (16, 64, 8, 64, 2499),
    (40, 16, 4, 128, 1998),          # two
    (40, 16, 4, 64, 1998),
    (400, 8, 2, 128, 300),           # several blocks of them
    (400, 8, 2, 64, 300),
])
def test_weights_between_bf16_steps(attn, B, H, Hkv, d, prefix, offset):
    g = torch.Generator().manual_seed(B + d)
    page, n = 16, prefix // 3
    pages = -(-prefix // page) + B
    kind = torch.zeros(pages * page, dtype=torch.bool)                 # which keys weigh w; the prefix's slots are 0 .. prefix - 1
    kind[:prefix] = torch.randperm(prefix, generator=g) >= n
    k = torch.zeros((pages * page, Hkv, d), dtype=torch.bfloat16)
    k[kind, :, 0] = -1.0
    k[:, :, 1] = 64.0
    v = (1 + torch.arange(d) % 64 / 64.0).expand(pages * page, Hkv, d).to(torch.bfloat16).clone()
    v[kind] = -1.0
    q = torch.zeros((B, H, d), dtype=torch.bfloat16)
    q[:, :, 0] = (torch.rand((B, H), generator=g) * np.log(2) * d ** 0.5).to(torch.bfloat16)      # w = exp(-q / sqrt(d))
    q[:, :, 1] = offset
    table = torch.arange(pages - B, dtype=torch.int32).expand(B, -1).contiguous()
    lens = torch.full((B,), prefix, dtype=torch.int32)
    k, v = (t.view(pages, page, Hkv, d) for t in (k, v))
    o, lse = attn.attn_paged_prefix_decode(*(t.cuda() for t in (q, k, v, lens, table)), prefix, return_lse=True)
    assert attn.cache_device_status() == (0, 0)
    w = np.exp(-q[:, :, 0].double().numpy() / np.sqrt(d))[:, :, None]
    plus, minus = n * (1 + np.arange(d) % 64 / 64.0), (prefix - n) * w
    total = n + minus
    ref, A = (plus - minus) / total, (plus + minus) / total
    err = np.abs(o.cpu().double().numpy() - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * A)
    assert np.all(err <= 0), float((err / A).max())
    want = 64 * offset / np.sqrt(d) + np.log(total[:, :, 0])
    assert np.all(np.abs(lse.cpu().double().numpy() - want) <= 2.0 ** -14 * (1 + want))
    # a sequence's outputs hold what attn_paged_decode's do, to the sums' order
    want = attn.attn_paged_decode(*(t.cuda() for t in (q, k, v, lens, table)))
    assert np.all(np.abs(o.cpu().double().numpy() - want.cpu().double().numpy()) <= 2.0 ** -7 * np.abs(ref) + 2.0 ** -13 * A)
