"""attn_paged_evict's ways through its kernels (needs a GB300): one CTA or a cluster a row, 512 or 1024 threads, rows moved
by the select kernel itself or over the list; by the numbers of rows and slots on a 152-SM part.  Values are copied, so
everything has to be equal, refused sequences and guards included."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_gpu_canaries import guarded, guards_intact
from tests.test_gpu_paged_evict import attn, expect, near, odd, status_ok, ties  # noqa: F401  (attn is a fixture)

pytestmark = pytest.mark.gpu


def cache(lens, most, P, Hkv, d, seed):
    """Pages for the used table entries only (the others name no page); bits of their own in every (slot, head)."""
    rng = np.random.default_rng(seed)
    used = [-(-n // P) for n in lens]
    pages = sum(used) + 2
    ids = rng.permutation(pages)
    table = np.full((len(lens), most), -9, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    g = torch.Generator().manual_seed(seed)
    bits = torch.randint(-2 ** 15, 2 ** 15, (2, pages, P, Hkv, d), generator=g, dtype=torch.int16)
    return bits[0].view(torch.bfloat16), bits[1].view(torch.bfloat16), table


def exponential(rng, shape):
    return rng.exponential(1.0, shape).astype(np.float32)


def device(x, dtype=np.int32):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=dtype)).cuda()


def compare(k, v, w, n, want):
    ek, ev, ew, en = want
    assert n.tolist() == en
    assert torch.equal(k.cpu().view(torch.int16), ek.view(k.shape)) and torch.equal(v.cpu().view(torch.int16), ev.view(v.shape))
    assert np.array_equal(w.cpu().numpy().reshape(ew.shape).view(np.int32), ew.view(np.int32))


def run(attn, lens, most, P, Hkv, d, budget, sinks, recent, seed, weights=exponential, inplace=True):  # noqa: F811
    kc, vc, table = cache(lens, most, P, Hkv, d, seed)
    w = weights(np.random.default_rng(seed + 1), (len(lens), Hkv, most * P))
    ek, ev, ew, en = expect(kc, vc, table, w, lens, budget, sinks, recent)
    k, v, wd, ld = kc.cuda(), vc.cuda(), device(w, np.float32), device(lens)
    out = {} if inplace else {"weights_out": torch.full_like(wd, -5.0), "seqlens_out": torch.full_like(ld, -5)}
    got = attn.attn_paged_evict(k, v, wd, ld, device(table), budget, sinks=sinks, recent=recent, **out)
    status_ok(attn)
    if not inplace:
        assert ld.tolist() == list(lens) and np.array_equal(wd.cpu().numpy().view(np.int32), w.view(np.int32))
        for b, n in enumerate(lens):
            ew[b, :, n:] = -5.0
    compare(k, v, wd if inplace else out["weights_out"], got, (ek, ev, ew, en))


RAGGED = [2560, 0, 1, 1000, 1001, 2559, 400, 401, 1255, 2000]
PATHS = {   # lens, max pages, page size, Hkv, budget, sinks, recent
    "1024_threads_own_moves": (RAGGED, 20, 128, 8, 400, 4, 200),           # keep 196
    "1024_threads_own_moves_few_over": (RAGGED, 20, 128, 8, 2400, 4, 200),  # 160 over at most
    "1024_threads_list": (RAGGED, 20, 128, 8, 1000, 4, 100),
    "1024_threads_list_wide_recent": (RAGGED, 20, 128, 8, 1000, 4, 900),    # few moves, a long recent block that overlaps
    "1024_threads_all_registers": ([16384, 16383, 9000] + [40] * 77, 64, 256, 1, 4096, 16, 512),
    "512_threads_list": ([1900, 700, 2048], 16, 128, 2, 600, 4, 100),
    "512_threads_own_moves": ([1900, 700, 2048], 16, 128, 2, 300, 50, 100),
    "cluster_of_2": ([4096, 700, 3000], 32, 128, 2, 600, 4, 100),
    "cluster_of_4_d": ([8192, 8191], 32, 256, 2, 1200, 4, 300),
    "own_moves_at_their_most": ([1024, 600], 64, 16, 2, 512, 0, 256),       # keep 256, recent 256
    "one_past_their_most": ([1024, 600], 64, 16, 2, 513, 0, 256),
    "recent_one_past": ([1024, 600], 64, 16, 2, 512, 0, 257),
}


@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "out"])
@pytest.mark.parametrize("weights", [exponential, ties, odd, near], ids=lambda f: f.__name__)
@pytest.mark.parametrize("path", PATHS)
def test_paths(attn, path, weights, inplace):  # noqa: F811
    lens, most, P, Hkv, budget, sinks, recent = PATHS[path]
    run(attn, lens, most, P, Hkv, 64, budget, sinks, recent, seed=len(path), weights=weights, inplace=inplace)


@pytest.mark.parametrize("path", ["1024_threads_own_moves", "512_threads_list", "cluster_of_2"])
def test_paths_with_longer_heads(attn, path):  # noqa: F811
    lens, most, P, Hkv, budget, sinks, recent = PATHS[path]
    run(attn, lens, most, P, Hkv, 128, budget, sinks, recent, seed=3)


REFUSED = {     # max pages, page size, budget, sinks, recent
    "own_moves": (64, 16, 200, 4, 8),
    "list": (64, 16, 400, 4, 8),
    "list_cluster": (256, 16, 400, 4, 8),
    "list_recent": (64, 16, 400, 4, 300),
}


@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "out"])
@pytest.mark.parametrize("path", REFUSED)
def test_refused_sequences_beside_cut_ones(attn, path, inplace):  # noqa: F811
    most, P, budget, sinks, recent = REFUSED[path]
    lens, Hkv, d = [1000, 800, 900, 20, 700, 950, 1024, budget, 0], 2, 64
    kc, vc, table = cache(lens, most, P, Hkv, d, 5)
    w = np.random.default_rng(6).random((len(lens), Hkv, most * P)).astype(np.float32)
    table, said = table.copy(), list(lens)
    table[1, 49] = kc.shape[0]                 # its last page is not in the cache
    table[2, 1] = table[3, 0]                  # shared with a sequence that is not cut
    said[4] = most * P + 1
    table[5, 2] = table[5, 40]                 # twice in one sequence
    stay = (1, 2, 4, 5)
    ek, ev, ew, _ = expect(kc, vc, table, w, [0 if b in stay else n for b, n in enumerate(lens)], budget, sinks, recent)
    en = [said[b] if b in stay else min(n, budget) for b, n in enumerate(lens)]
    k, v, wd, ld = kc.cuda(), vc.cuda(), device(w, np.float32), device(said)
    out = {} if inplace else {"weights_out": torch.full_like(wd, -5.0), "seqlens_out": torch.full_like(ld, -5)}
    got = attn.attn_paged_evict(k, v, wd, ld, device(table), budget, sinks=sinks, recent=recent, **out)
    assert attn.cache_device_status() == (1, 23)
    if not inplace:
        assert ld.tolist() == said and np.array_equal(wd.cpu().numpy(), w)
        for b, n in enumerate(lens):
            ew[b, :, 0 if b in stay else n:] = -5.0
    compare(k, v, wd if inplace else out["weights_out"], got, (ek, ev, ew, en))
    status_ok(attn)


def evict_args(attn, kc, table, P, budget, sinks, recent):  # noqa: F811
    a = attn.EvictArgs()
    a.B, a.max_pages = table.shape
    a.Hkv, a.num_pages, a.page_size, a.d = kc.shape[2], kc.shape[0], P, kc.shape[3]
    a.budget, a.sinks, a.recent = budget, sinks, recent
    return a


@pytest.mark.parametrize("path", ["512_threads_list", "cluster_of_2", "1024_threads_own_moves", "1024_threads_list"])
def test_guards(attn, path):  # noqa: F811
    lens, most, P, Hkv, budget, sinks, recent = PATHS[path]
    kc, vc, table = cache(lens, most, P, Hkv, 64, 7)
    w = np.random.default_rng(8).random((len(lens), Hkv, most * P)).astype(np.float32)
    want = expect(kc, vc, table, w, lens, budget, sinks, recent)
    a = evict_args(attn, kc, table, P, budget, sinks, recent)
    need = int(attn.load().attn_paged_evict_workspace_size(ctypes.byref(a)))
    kb, k = guarded(kc.numel(), "bf16")
    vb, v = guarded(vc.numel(), "bf16")
    wb, wd = guarded(w.size, "f32")
    sb, ws = guarded(need, "ws")
    k.view(torch.int16).copy_(kc.flatten().view(torch.int16))
    v.view(torch.int16).copy_(vc.flatten().view(torch.int16))
    wd.copy_(torch.as_tensor(w).flatten())
    ld = device(lens)
    attn.attn_paged_evict(k.view(kc.shape), v.view(vc.shape), wd.view(w.shape), ld, device(table), budget, sinks=sinks,
                          recent=recent, workspace=ws)
    torch.cuda.synchronize()
    for buf, kind in ((kb, "bf16"), (vb, "bf16"), (wb, "f32"), (sb, "ws")):
        assert guards_intact(buf, kind)
    compare(k, v, wd, ld, want)
    status_ok(attn)


def test_the_table_s_room_changes_nothing(attn):  # noqa: F811
    # lengths and budget alike, tables of 64, 128 and 2048 pages: own moves, the list, the list and clusters
    lens, P, Hkv, d, budget, sinks, recent = [1030, 1024, 900, 1001], 16, 2, 128, 1000, 4, 128
    kc, vc, table = cache(lens, 65, P, Hkv, d, 9)
    w = np.random.default_rng(10).exponential(1.0, (4, Hkv, 65 * P)).astype(np.float32)
    out = []
    for most in (65, 128, 2048):
        wide, ww = np.full((4, most), -9), np.full((4, Hkv, most * P), 3.0)
        wide[:, :65], ww[:, :, :65 * P] = table, w
        k, v, n, wd = kc.cuda(), vc.cuda(), device(lens), device(ww, np.float32)
        attn.attn_paged_evict(k, v, wd, n, device(wide), budget, sinks=sinks, recent=recent)
        assert most == 65 or (wd[:, :, 65 * P:] == 3.0).all()
        out.append((k.view(torch.int16), v.view(torch.int16), n, wd[:, :, :65 * P].contiguous()))
    for other in out[1:]:
        assert all(torch.equal(x, y) for x, y in zip(out[0], other))
    status_ok(attn)


@pytest.mark.parametrize("path", ["512_threads_own_moves", "512_threads_list", "cluster_of_2"])
def test_two_streams_with_workspaces_of_their_own_and_a_graph(attn, path):  # noqa: F811
    lens, most, P, Hkv, budget, sinks, recent = PATHS[path]
    kc, vc, table = cache(lens, most, P, Hkv, 64, 11)
    w = np.random.default_rng(12).random((len(lens), Hkv, most * P)).astype(np.float32)
    want = expect(kc, vc, table, w, lens, budget, sinks, recent)
    first = [kc.cuda(), vc.cuda(), device(w, np.float32), device(lens)]
    t = device(table)
    states = [[x.clone() for x in first] for _ in range(6)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, (k, v, wd, n) in enumerate(states):
        attn.attn_paged_evict(k, v, wd, n, t, budget, sinks=sinks, recent=recent, stream=streams[i % 2])
    torch.cuda.synchronize()
    for k, v, wd, n in states:
        compare(k, v, wd, n, want)
    graphs = []
    for state in states[:2]:                         # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attn.attn_paged_evict(*state, t, budget, sinks=sinks, recent=recent)
        graphs.append(g)
    for _ in range(3):
        for state in states[:2]:
            for x, y in zip(state, first):
                x.copy_(y)
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for k, v, wd, n in states[:2]:
            compare(k, v, wd, n, want)
    status_ok(attn)
