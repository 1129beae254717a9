"""attn_norm_rope_bwd without tokens through the C entry (the binding ends before it): the weights' gradients are zero, and nothing
divides by the number of tokens (needs a GB300)."""
import ctypes

import pytest
import torch

from tests.test_gpu_norm_rope import attn, tables_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,k,weights", [(1, True, 2), (3, True, 1), (2, False, 1), (1, True, 0)])
def test_gradient_of_no_tokens(attn, d, B, k, weights):  # noqa: F811
    t = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    pos, freqs, axes = tables_of(attn, (1, 1, 1, 1, d, "bshd", (d,), "adjacent", 0))
    dw = torch.full((2, d + 64), 7.0, device="cuda")
    w = torch.ones(d, device="cuda")
    a = attn.NormRopeBwdArgs()
    at = [t[512 * i:].data_ptr() for i in range(6)]
    a.q, a.q_out, a.dq, a.q_weight = *at[:3], w.data_ptr()
    if k:
        a.k, a.k_out, a.dk, a.k_weight = *at[3:], w.data_ptr()
    a.positions, a.freqs, a.axes = pos.data_ptr(), freqs.data_ptr(), axes.data_ptr()
    a.B, a.S, a.H, a.Hkv, a.d, a.pairs, a.num_axes, a.eps = B, 0, 2, 1, d, d // 2, 1, 1e-6
    for s in ("q_stride", "q_out_stride", "k_stride", "k_out_stride", "dq_stride", "dk_stride"):
        setattr(a, s, (ctypes.c_int64 * 3)(2 * d, 2 * d, d))
    a.dq_weight, a.dk_weight = (dw[i, 32:].data_ptr() if weights > i else None for i in range(2))
    lib = attn.load()
    need = int(lib.attn_norm_rope_bwd_workspace_size(ctypes.byref(a)))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")         # (NaN, were it read)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.attn_norm_rope_bwd(ctypes.byref(a), ws.data_ptr(), need, stream) == 0
    assert attn.cache_device_status() == (0, 0) and not t.any()
    for i in range(2):
        assert (dw[i, :32] == 7).all() and (dw[i, 32 + d:] == 7).all()
        assert (dw[i, 32:32 + d] == (0 if weights > i else 7)).all()
