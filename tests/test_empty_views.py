"""Dense tensors of no tokens, whose batch stride S * H * d is zero, through the C entries of the rotary calls: no two of their elements
share an address, since there are none (CPU only; fake addresses that nothing reads)."""
import ctypes

import pytest

import bf16_attention_forward_gb300 as attn
from tests.test_norm_reserve_boundary import M, NO_DEVICE, OK, back, fake_pointers, fill, lib, norm  # noqa: F401

DENSE = dict(S=0, B=3, q_stride=(0, 512, 128), q_out_stride=(0, 512, 128), k_stride=(0, 256, 128), k_out_stride=(0, 256, 128))


@fake_pointers
@pytest.mark.parametrize("kw", [dict(), dict(k=0), dict(q_out=M, k_out=3 * M)])
def test_no_tokens_in_dense_batches(lib, kw):  # noqa: F811
    assert lib.attn_norm_rope(ctypes.byref(norm(**DENSE, **kw)), None) == OK
    a = fill(attn.RopeArgs(), **{**dict(q=M, q_out=2 * M, k=3 * M, k_out=4 * M, positions=5 * M, freqs=6 * M, axes=7 * M, H=4, Hkv=2, d=128,
                                        pos_axis_stride=10, pairs=64, num_axes=1), **DENSE, **kw})
    assert lib.attn_rope(ctypes.byref(a), None) == OK
    b = dict(dq_stride=(0, 512, 128), dk_stride=(0, 256, 128))
    if "k" in kw:
        b.update(dk=0, dk_weight=0)
    b.update({n: v for n, v in kw.items() if n == "k"})
    assert lib.attn_norm_rope_bwd(ctypes.byref(back(**DENSE, **b)), None, 0, None) == NO_DEVICE
