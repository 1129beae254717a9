"""Refusals of the norms with positions, of attn_paged_reserve and of attn_paged_prefix_decode, on the host: argument errors come back before anything is
launched (CPU only; the C entries get fake addresses that nothing reads)."""
import ctypes

import pytest
import torch

import bf16_attention_forward_gb300 as attn
from bf16_attention_forward_gb300 import build as libbuild

fake_pointers = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: only where no GPU is visible")
M = 1 << 24          # addresses this far apart do not meet in the cases below
OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS, NO_DEVICE, WORKSPACE = 0, 1, 2, 3, 4, 5, 6
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return attn.load()


def fill(a, **kw):
    for n, v in kw.items():
        setattr(a, n, v)
    return a


FORWARD = dict(q=M, q_out=2 * M, k=3 * M, k_out=4 * M, q_weight=8 * M, k_weight=9 * M, positions=5 * M, freqs=6 * M, axes=7 * M,
               B=2, S=10, H=4, Hkv=2, d=128, q_stride=(5120, 512, 128), q_out_stride=(5120, 512, 128),
               k_stride=(2560, 256, 128), k_out_stride=(2560, 256, 128), pos_axis_stride=10, pairs=64, num_axes=1, eps=1e-6)


def norm(**kw):
    return fill(attn.NormRopeArgs(), **{**FORWARD, **kw})


def back(**kw):
    return fill(attn.NormRopeBwdArgs(), **{**FORWARD, **dict(dq=10 * M, dk=11 * M, dq_weight=12 * M, dk_weight=13 * M,
                                                             dq_stride=(5120, 512, 128), dk_stride=(2560, 256, 128)), **kw})


def append(**kw):
    a = fill(attn.NormAppendArgs(), k=M, v=2 * M, k_cache=3 * M, v_cache=4 * M, q=5 * M, q_out=6 * M, q_weight=7 * M,
             k_weight=8 * M, slots=9 * M, positions=10 * M, freqs=11 * M, axes=12 * M, H=4, Hkv=2, total=10, num_pages=8,
             page_size=16, d=128, q_stride=(512, 128), k_stride=(256, 128), v_stride=(256, 128), pos_axis_stride=10, pairs=64,
             num_axes=1, eps=1e-6)
    return fill(a, **kw)


def reserve(**kw):
    a = fill(attn.ReserveArgs(), seqlens_k=M, cu_seqlens_new=2 * M, block_table=3 * M, pages_held=4 * M, held_out=5 * M,
             shared_pages=6 * M, free_pages=7 * M, free_count=8 * M, count_out=9 * M, slots=10 * M, positions=11 * M, B=4,
             max_pages=8, page_size=16, capacity=64, total=20)
    return fill(a, **kw)


def prefix(**kw):
    a = fill(attn.DecodeArgs(), q=M, k_cache=2 * M, v_cache=3 * M, o=4 * M, lse=5 * M, seqlens_k=7 * M, block_table=8 * M,
             B=2, H=8, Hkv=2, num_pages=8, page_size=16, max_pages=4, d=128)
    return fill(a, **kw)


NORM = [
    (INVALID, [dict(q=0), dict(q_out=0), dict(k_out=0), dict(positions=0), dict(freqs=0), dict(axes=0), dict(B=0),
               dict(S=-1), dict(H=0), dict(Hkv=0), dict(pairs=-1), dict(pairs=65), dict(num_axes=0), dict(pairing=2),
               dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(weight_bf16=2), dict(reserved=1),
               dict(q_stride=(5120, -512, 128)), dict(pos_axis_stride=-1), dict(q_stride=(1 << 41, 512, 128))]),
    (UNSUPPORTED, [dict(d=96), dict(pairing=1, pairs=20), dict(S=(1 << 30) + 1), dict(B=1 << 20, S=1 << 20)]),
    (MISALIGNED, [dict(q=M + 8), dict(k_out=4 * M + 2), dict(q_stride=(5120, 516, 128)), dict(freqs=6 * M + 4),
                  dict(positions=5 * M + 2), dict(q_weight=8 * M + 2), dict(k_weight=9 * M + 1, weight_bf16=1)]),
    (ALIAS, [dict(q_out=M + 256), dict(k_out=2 * M), dict(k_out=M), dict(q_out=M, q_out_stride=(5120, 128, 1280)),
             dict(q_out_stride=(5120, 512, 64)), dict(q_out_stride=(512, 512, 128)), dict(q_out=3 * M), dict(q_weight=2 * M),
             dict(k_weight=4 * M + 512), dict(q_weight=4 * M, weight_bf16=1)]),
    (NO_DEVICE, [dict(), dict(k=0), dict(k=0, k_weight=0), dict(q_weight=0), dict(k_weight=9 * M + 2, weight_bf16=1), dict(eps=0.0),
                 dict(q_out=M, k_out=3 * M), dict(pairs=0, positions=0, freqs=0, axes=0), dict(pairs=0, pos_axis_stride=-1),
                 dict(q_stride=(0, 512, 128)), dict(pairs=1), dict(pairing=1, pairs=8), dict(q_weight=9 * M)]),
    (OK, [dict(S=0)]),
]
BACK = [
    (INVALID, [dict(dq=0), dict(dk=0), dict(k=0), dict(k=0, dk=0), dict(q=0), dict(q_out=0), dict(eps=NAN),
               dict(dq_stride=(5120, -512, 128)), dict(dk_stride=(-1, 256, 128))]),
    (UNSUPPORTED, [dict(d=32), dict(pairing=1, pairs=4)]),
    (MISALIGNED, [dict(dq=10 * M + 8), dict(dk=11 * M + 4), dict(dq_weight=12 * M + 2), dict(dk_stride=(2560, 260, 128)),
                  dict(q_out=2 * M + 8)]),
    (ALIAS, [dict(q_out=4 * M), dict(q_out_stride=(512, 512, 128)), dict(q_weight=2 * M), dict(q_out=M), dict(k_out=3 * M),
             dict(q_out=11 * M), dict(k_out=10 * M), dict(q_out=10 * M + 256), dict(q_out=3 * M), dict(dq_weight=M),
             dict(dk_weight=2 * M + 64), dict(dq_weight=8 * M), dict(dk_weight=12 * M + 256), dict(dk_weight=11 * M)]),
    (NO_DEVICE, [dict(), dict(q_out=10 * M, k_out=11 * M), dict(k=0, dk=0, dk_weight=0), dict(dq_weight=0), dict(S=0)]),
]
APPEND = [
    (INVALID, [dict(k=0), dict(v=0), dict(k_cache=0), dict(v_cache=0), dict(q_out=0), dict(slots=0), dict(positions=0),
               dict(Hkv=0), dict(H=0), dict(total=-1), dict(num_pages=0), dict(page_size=0), dict(reserved=1), dict(pairs=-1),
               dict(num_axes=0), dict(k_stride=(-256, 128)), dict(eps=-1.0), dict(eps=INF), dict(weight_bf16=-1)]),
    (UNSUPPORTED, [dict(d=32), dict(num_pages=1 << 20, page_size=1 << 20), dict(pairing=1, pairs=12), dict(total=(1 << 30) + 1)]),
    (MISALIGNED, [dict(k=M + 8), dict(v_cache=4 * M + 4), dict(q_stride=(516, 128)), dict(slots=9 * M + 4),
                  dict(q_weight=7 * M + 1)]),
    (ALIAS, [dict(v_cache=3 * M), dict(k_cache=M), dict(q_out=M), dict(q_out=3 * M), dict(q_out=5 * M + 512), dict(q=4 * M),
             dict(k_weight=3 * M), dict(q_weight=6 * M + 64)]),
    (NO_DEVICE, [dict(), dict(q=0), dict(pairs=0, positions=0, freqs=0, axes=0), dict(q_out=5 * M), dict(page_size=1),
                 dict(q_weight=0, k_weight=0)]),
    (OK, [dict(total=0)]),
]
RESERVE = [
    (INVALID, [dict(seqlens_k=0), dict(cu_seqlens_new=0), dict(block_table=0), dict(pages_held=0), dict(held_out=0),
               dict(free_pages=0), dict(free_count=0), dict(count_out=0), dict(slots=0), dict(B=0), dict(max_pages=0),
               dict(page_size=0), dict(capacity=0), dict(total=-1)]),
    (UNSUPPORTED, [dict(B=1 << 28), dict(max_pages=1 << 27), dict(capacity=(1 << 30) + 1), dict(total=(1 << 30) + 1)]),
    (MISALIGNED, [dict(seqlens_k=M + 2), dict(slots=10 * M + 4), dict(positions=11 * M + 1), dict(free_pages=7 * M + 3)]),
    (ALIAS, [dict(block_table=M), dict(held_out=4 * M + 4), dict(held_out=M), dict(count_out=7 * M + 8), dict(slots=3 * M),
             dict(positions=10 * M), dict(free_pages=3 * M + 64), dict(count_out=5 * M), dict(shared_pages=5 * M)]),
    (NO_DEVICE, [dict(), dict(held_out=4 * M, count_out=8 * M), dict(shared_pages=0), dict(positions=0), dict(total=0, slots=0),
                 dict(shared_pages=M), dict(page_size=1)]),
]


PREFIX = [
    (INVALID, [dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(o=0), dict(seqlens_k=0), dict(block_table=0), dict(B=0),
               dict(H=0), dict(Hkv=0), dict(H=7), dict(num_pages=0), dict(page_size=0), dict(max_pages=0), dict(round_mode=3),
               dict(reserved=1), dict(weights=6 * M), dict(n=0), dict(n=-1), dict(n=65)]),
    (UNSUPPORTED, [dict(d=256), dict(num_pages=1 << 29, page_size=16), dict(B=1 << 29)]),
    (MISALIGNED, [dict(q=M + 2), dict(o=4 * M + 8), dict(lse=5 * M + 2), dict(seqlens_k=7 * M + 2)]),
    (ALIAS, [dict(o=M), dict(o=2 * M + 512), dict(lse=4 * M), dict(lse=7 * M), dict(lse=8 * M)]),
    (NO_DEVICE, [dict(), dict(n=1), dict(n=64), dict(lse=0), dict(page_size=1, n=4), dict(H=142)]),
]


def cases(table):
    return [(want, kw) for want, kws in table for kw in kws]


def name(x):
    return "_".join("%s=%s" % i for i in x.items()).replace(" ", "") or "as_it_is" if isinstance(x, dict) else str(x)


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(NORM), ids=name)
def test_norm_rope(lib, want, kw):
    assert lib.attn_norm_rope(ctypes.byref(norm(**kw)), None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(BACK), ids=name)
def test_norm_rope_bwd(lib, want, kw):
    assert lib.attn_norm_rope_bwd(ctypes.byref(back(**kw)), 16 * M, 1 << 20, None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(APPEND), ids=name)
def test_norm_rope_append(lib, want, kw):
    assert lib.attn_norm_rope_append(ctypes.byref(append(**kw)), None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(RESERVE), ids=name)
def test_paged_reserve(lib, want, kw):
    assert lib.attn_paged_reserve(ctypes.byref(reserve(**kw)), None) == want


@fake_pointers
@pytest.mark.parametrize("want,kw", cases(PREFIX), ids=name)
def test_paged_prefix_decode(lib, want, kw):
    kw = dict(kw)
    n = kw.pop("n", 20)
    assert lib.attn_paged_prefix_decode(ctypes.byref(prefix(**kw)), n, 16 * M, 1 << 20, None) == want


@fake_pointers
def test_sizes_without_a_device(lib):
    assert lib.attn_paged_prefix_decode_workspace_size(ctypes.byref(prefix()), 20) == 0
    assert lib.attn_norm_rope_bwd_workspace_size(ctypes.byref(back())) == 0


def test_null_arguments(lib):
    assert lib.attn_norm_rope(None, None) == INVALID and lib.attn_norm_rope_append(None, None) == INVALID
    assert lib.attn_norm_rope_bwd(None, None, 0, None) == INVALID and lib.attn_paged_reserve(None, None) == INVALID
    assert lib.attn_norm_rope_bwd_workspace_size(None) == 0
    assert lib.attn_paged_prefix_decode(None, 1, None, 0, None) == INVALID
    assert lib.attn_paged_prefix_decode_workspace_size(None, 1) == 0


def test_argument_structures_have_the_abi_s_sizes():
    """The binding packs the arguments by itself: 8-byte fields first, no holes."""
    assert ctypes.sizeof(attn.NormRopeArgs) == 8 * (9 + 5 + 12 + 2) + 4 * 6
    assert ctypes.sizeof(attn.NormRopeBwdArgs) == ctypes.sizeof(attn.NormRopeArgs) + 8 * (4 + 6)
    assert ctypes.sizeof(attn.NormAppendArgs) == 8 * (12 + 6 + 6 + 1) + 4 * 6
    assert ctypes.sizeof(attn.ReserveArgs) == 8 * (11 + 5)


def test_binding_wants_cuda_tensors():
    t = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    c = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    i, j = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)
    for call in (lambda: attn.attn_norm_rope(t, t), lambda: attn.attn_norm_rope(None, None),
                 lambda: attn.attn_norm_rope_bwd(t, t, t, t), lambda: attn.attn_norm_rope_append(t, t, c, c, i.long()),
                 lambda: attn.attn_paged_reserve(i, i, j, i, i, i, 16),
                 lambda: attn.attn_paged_prefix_decode(t, c, c, i, j, 1)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: attn.attn_norm_rope(t, t, layout="x"), lambda: attn.attn_norm_rope(t, t, pairing="x")):
        with pytest.raises(ValueError):
            call()
