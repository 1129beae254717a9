"""Refusals of the calls around the paged cache, on the host: argument errors come back before
anything is launched (CPU only; the C entries get fake addresses that nothing reads)."""
import ctypes

import pytest
import torch

import bf16_attention_forward_gb300 as attn
from bf16_attention_forward_gb300 import build as libbuild

fake_pointers = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: only where no GPU is visible")
M = 1 << 24          # addresses this far apart do not meet in the cases below
OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS, NO_DEVICE, WORKSPACE = 0, 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return attn.load()


def fill(a, **kw):
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def rope(**kw):
    a = fill(attn.RopeArgs(), q=M, q_out=2 * M, k=3 * M, k_out=4 * M, positions=5 * M, freqs=6 * M, axes=7 * M,
             B=2, S=10, H=4, Hkv=2, d=128, q_stride=(5120, 512, 128), q_out_stride=(5120, 512, 128),
             k_stride=(2560, 256, 128), k_out_stride=(2560, 256, 128), pos_axis_stride=10, pairs=64, num_axes=1)
    return fill(a, **kw)


def append(**kw):
    a = fill(attn.AppendArgs(), k=M, v=2 * M, k_cache=3 * M, v_cache=4 * M, q=5 * M, q_out=6 * M, cu_seqlens_new=7 * M,
             seqlens_k=8 * M, block_table=9 * M, positions=10 * M, freqs=11 * M, axes=12 * M, B=2, H=4, Hkv=2, total=10,
             num_pages=8, page_size=16, max_pages=4, d=128, q_stride=(512, 128), k_stride=(256, 128),
             v_stride=(256, 128), pos_axis_stride=10, pairs=64, num_axes=1)
    return fill(a, **kw)


def decode(**kw):
    a = fill(attn.DecodeArgs(), q=M, k_cache=2 * M, v_cache=3 * M, o=4 * M, lse=5 * M, weights=6 * M, seqlens_k=7 * M,
             block_table=8 * M, B=2, H=8, Hkv=2, num_pages=8, page_size=16, max_pages=4, d=128)
    return fill(a, **kw)


def evict(**kw):
    a = fill(attn.EvictArgs(), k_cache=M, v_cache=2 * M, weights=3 * M, weights_out=4 * M, seqlens_k=5 * M,
             seqlens_out=6 * M, block_table=7 * M, B=2, Hkv=2, num_pages=8, page_size=16, max_pages=4, d=128, budget=32,
             sinks=4, recent=8)
    return fill(a, **kw)


ROPE = [
    (INVALID, [dict(q=0), dict(q_out=0), dict(k_out=0), dict(positions=0), dict(freqs=0), dict(axes=0), dict(B=0),
               dict(S=-1), dict(H=0), dict(Hkv=0), dict(pairs=0), dict(pairs=65), dict(num_axes=0), dict(pairing=2),
               dict(inverse=2), dict(q_stride=(5120, -512, 128)), dict(pos_axis_stride=-1),
               dict(q_stride=(1 << 41, 512, 128))]),
    (UNSUPPORTED, [dict(d=96), dict(pairing=1, pairs=20), dict(S=(1 << 30) + 1), dict(B=1 << 20, S=1 << 20)]),
    (MISALIGNED, [dict(q=M + 8), dict(k_out=4 * M + 2), dict(q_stride=(5120, 516, 128)), dict(freqs=6 * M + 4),
                  dict(positions=5 * M + 2)]),
    (ALIAS, [dict(q_out=M + 256), dict(k_out=2 * M), dict(k_out=M), dict(q_out=M, q_out_stride=(5120, 128, 1280)),
             dict(q_out_stride=(5120, 512, 64)), dict(q_out_stride=(512, 512, 128)), dict(q_out=3 * M)]),
    # columns of one projection's rows, in place or not, do not meet
    (NO_DEVICE, [dict(), dict(k=0), dict(q_out=M, k_out=3 * M), dict(S=1, q_stride=(512, 0, 128)), dict(S=1, q_stride=(512, 3, 128)), dict(B=1, q_stride=(7, 512, 128)),
                 dict(q=M, k=M + 1024, q_out=M, k_out=M + 1024, q_stride=(10240, 1024, 128), k_stride=(10240, 1024, 128),
                      q_out_stride=(10240, 1024, 128), k_out_stride=(10240, 1024, 128)),
                 dict(q_stride=(0, 512, 128)), dict(pairs=1), dict(pairing=1, pairs=8)]),
    (ALIAS, [dict(q=M, k=M + 768, q_out=M, k_out=M + 768, q_stride=(10240, 1024, 128), k_stride=(10240, 1024, 128),
                  q_out_stride=(10240, 1024, 128), k_out_stride=(10240, 1024, 128))]),
    (OK, [dict(S=0)]),
]
APPEND = [
    (INVALID, [dict(k=0), dict(v=0), dict(k_cache=0), dict(v_cache=0), dict(q_out=0), dict(cu_seqlens_new=0),
               dict(seqlens_k=0), dict(block_table=0), dict(positions=0), dict(B=0), dict(Hkv=0), dict(H=0),
               dict(total=-1), dict(num_pages=0), dict(page_size=0), dict(max_pages=0), dict(reserved=1),
               dict(pairs=-1), dict(num_axes=0), dict(k_stride=(-256, 128))]),
    (UNSUPPORTED, [dict(d=32), dict(num_pages=1 << 20, page_size=1 << 20), dict(pairing=1, pairs=12),
                   dict(max_pages=1 << 27)]),
    (MISALIGNED, [dict(k=M + 8), dict(v_cache=4 * M + 4), dict(q_stride=(516, 128)), dict(seqlens_k=8 * M + 1)]),
    (ALIAS, [dict(v_cache=3 * M), dict(k_cache=M), dict(q_out=M), dict(q_out=3 * M), dict(q_out=5 * M + 512)]),
    (NO_DEVICE, [dict(), dict(q=0), dict(pairs=0, positions=0, freqs=0, axes=0), dict(q_out=5 * M),
                 dict(page_size=1, max_pages=1)]),
    (OK, [dict(total=0)]),
]
DECODE = [
    (INVALID, [dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(o=0), dict(seqlens_k=0), dict(block_table=0), dict(B=0),
               dict(H=0), dict(Hkv=0), dict(H=7), dict(num_pages=0), dict(page_size=0), dict(max_pages=0),
               dict(round_mode=3), dict(round_mode=-1), dict(reserved=1)]),
    (UNSUPPORTED, [dict(d=256), dict(d=96), dict(num_pages=1 << 29, page_size=16), dict(B=1 << 29)]),
    (MISALIGNED, [dict(q=M + 2), dict(o=4 * M + 8), dict(lse=5 * M + 2), dict(weights=6 * M + 1), dict(seqlens_k=7 * M + 2)]),
    (ALIAS, [dict(o=M), dict(o=2 * M + 512), dict(lse=4 * M), dict(weights=4 * M + 64), dict(weights=3 * M),
             dict(lse=7 * M), dict(weights=8 * M)]),
    (NO_DEVICE, [dict(), dict(lse=0), dict(weights=0), dict(page_size=1), dict(H=142)]),
]
EVICT = [
    (INVALID, [dict(k_cache=0), dict(v_cache=0), dict(weights=0), dict(weights_out=0), dict(seqlens_k=0),
               dict(seqlens_out=0), dict(block_table=0), dict(B=0), dict(Hkv=0), dict(budget=0), dict(sinks=-1),
               dict(recent=-1), dict(sinks=30, recent=3), dict(page_size=0)]),
    (UNSUPPORTED, [dict(d=80), dict(budget=(1 << 30) + 1), dict(num_pages=1 << 29, page_size=16),
                   dict(num_pages=1 << 26, Hkv=16), dict(max_pages=1 << 25, Hkv=8)]),
    (MISALIGNED, [dict(k_cache=M + 8), dict(weights=3 * M + 2), dict(seqlens_out=6 * M + 1)]),
    (ALIAS, [dict(v_cache=M), dict(weights_out=3 * M + 64), dict(weights=M), dict(seqlens_out=5 * M + 4),
             dict(weights_out=2 * M)]),
    (WORKSPACE, [dict()]),
]


def cases(table):
    return [(want, kw) for want, kws in table for kw in kws]


def name(x):
    return "_".join("%s=%s" % i for i in x.items()).replace(" ", "") or "as_it_is" if isinstance(x, dict) else str(x)


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(ROPE), ids=name)
def test_rope(lib, want, kw):
    assert lib.attn_rope(ctypes.byref(rope(**kw)), None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(APPEND), ids=name)
def test_append(lib, want, kw):
    assert lib.attn_paged_append(ctypes.byref(append(**kw)), None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(DECODE), ids=name)
def test_decode(lib, want, kw):
    assert lib.attn_paged_decode(ctypes.byref(decode(**kw)), 16 * M, 1 << 20, None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(EVICT), ids=name)
def test_evict(lib, want, kw):
    assert lib.attn_paged_evict(ctypes.byref(evict(**kw)), None, 0, None) == want


@fake_pointers
def test_evict_workspace(lib):
    a = evict()
    need = lib.attn_paged_evict_workspace_size(ctypes.byref(a))
    assert need > 0
    assert lib.attn_paged_evict(ctypes.byref(a), 16 * M, need - 1, None) == WORKSPACE
    assert lib.attn_paged_evict(ctypes.byref(a), 16 * M + 8, need, None) == MISALIGNED
    assert lib.attn_paged_evict(ctypes.byref(a), 4 * M, need, None) == ALIAS
    assert lib.attn_paged_evict(ctypes.byref(a), 16 * M, need, None) == NO_DEVICE
    assert lib.attn_paged_evict_workspace_size(ctypes.byref(evict(budget=0))) == 0
    assert lib.attn_paged_decode_workspace_size(ctypes.byref(decode())) == 0      # no device to size it for


def test_null_arguments(lib):
    assert lib.attn_rope(None, None) == INVALID and lib.attn_paged_append(None, None) == INVALID
    assert lib.attn_paged_decode(None, None, 0, None) == INVALID
    assert lib.attn_paged_evict(None, None, 0, None) == INVALID


def test_rope_freqs():
    f, a = attn.rope_freqs((4, 2), base=100.0, device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == pytest.approx([1.0, 0.1, 1.0], rel=1e-15) and a.tolist() == [0, 0, 1]
    f, a = attn.rope_freqs((4, 2), base=8.0, spectrum="shared", scale=(1.0, 0.5), device="cpu")
    assert f.tolist() == pytest.approx([1.0, 0.5, 0.125], rel=1e-15)
    for bad in (dict(axis_dims=()), dict(axis_dims=(3,)), dict(axis_dims=(4,), spectrum="x"),
                dict(axis_dims=(4,), scale=(1, 2)), dict(axis_dims=(4,), base=0.0)):
        with pytest.raises(ValueError):
            attn.rope_freqs(device="cpu", **bad)


def test_binding_wants_cuda_tensors():
    t = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: attn.attn_rope(t, t, i, i, i), lambda: attn.attn_rope(None, None, i, i, i),
                 lambda: attn.attn_paged_append(t, t, c, c, i, i, i), lambda: attn.attn_paged_decode(t, c, c, i, i),
                 lambda: attn.attn_paged_evict(c, c, t, i, i, 1)):
        with pytest.raises(TypeError):
            call()
