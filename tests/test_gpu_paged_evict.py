"""Eviction from a paged cache by accumulated weight (attn_paged_evict) against the rule written out
on the CPU: values are copied, so everything has to be equal (needs a GB300)."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_gpu_canaries import guarded, guards_intact

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


def sources(w, n, budget, sinks, recent):
    """Slot whose key each of the first min(n, budget) slots holds after the call."""
    if n <= budget:
        return list(range(n))
    rank = lambda j: (np.isnan(w[j]), -w[j] if not np.isnan(w[j]) else 0.0, j)  # noqa: E731
    best = sorted(range(sinks, n - recent), key=rank)[:budget - sinks - recent]
    kept = set(range(sinks)) | set(best)
    late = iter(sorted(j for j in kept if j >= budget - recent))
    return [j if j in kept else next(late) for j in range(budget - recent)] + list(range(n - recent, n))


def cache(lens, most, P, Hkv, d, seed):
    """Every (slot, head) of the cache holds bits of its own."""
    rng = np.random.default_rng(seed)
    pages = len(lens) * most + 2
    table = rng.permutation(pages)[:len(lens) * most].reshape(len(lens), most).astype(np.int32)
    bits = torch.as_tensor(rng.integers(-2 ** 15, 2 ** 15, (2, pages, P, Hkv, d)).astype(np.int16))
    return bits[0].view(torch.bfloat16), bits[1].view(torch.bfloat16), table


def expect(kc, vc, table, w, lens, budget, sinks, recent):
    P, Hkv = kc.shape[1:3]
    k, v, out = kc.clone().view(torch.int16), vc.clone().view(torch.int16), w.copy()
    new = list(lens)
    at = lambda b, j: table[b, np.asarray(j) // P].astype(np.int64) * P + np.asarray(j) % P  # noqa: E731
    for b, n in enumerate(lens):
        new[b] = min(n, budget)
        for h in range(Hkv):
            src = sources(w[b, h], n, budget, sinks, recent)
            if n > budget:
                to, rows = torch.as_tensor(at(b, np.arange(budget))), torch.as_tensor(at(b, src))
                for c in (k, v):
                    flat = c.view(-1, Hkv, c.shape[-1])
                    flat[to, h] = flat[rows, h]
                out[b, h, :budget] = w[b, h, src]
                out[b, h, budget:n] = 0
    return k, v, out, new


def run(attn, lens, most, P, Hkv, d, budget, sinks, recent, seed=0, weights=None, inplace=True):
    kc, vc, table = cache(lens, most, P, Hkv, d, seed)
    rng = np.random.default_rng(seed + 1)
    w = rng.exponential(1.0, (len(lens), Hkv, most * P)).astype(np.float32) if weights is None else weights(rng, (len(lens), Hkv, most * P))
    ek, ev, ew, en = expect(kc, vc, table, w, lens, budget, sinks, recent)
    k, v, wd = kc.cuda(), vc.cuda(), torch.as_tensor(w).cuda()
    ld = torch.as_tensor(np.asarray(lens, dtype=np.int32)).cuda()
    kw = {} if inplace else {"weights_out": torch.full_like(wd, -5.0), "seqlens_out": torch.full_like(ld, -5)}
    got = attn.attn_paged_evict(k, v, wd, ld, torch.as_tensor(table).cuda(), budget, sinks=sinks, recent=recent, **kw)
    status_ok(attn)
    assert got.tolist() == en
    assert torch.equal(k.cpu().view(torch.int16), ek) and torch.equal(v.cpu().view(torch.int16), ev)
    new = (wd if inplace else kw["weights_out"]).cpu().numpy().view(np.int32)
    if not inplace:
        assert ld.tolist() == list(lens) and np.array_equal(wd.cpu().numpy().view(np.int32), w.view(np.int32))
        for b, n in enumerate(lens):
            ew[b, :, n:] = -5.0
    assert np.array_equal(new, ew.view(np.int32))


CASES = [  # lens, max pages, page size, Hkv, d, budget, sinks, recent
    ([100], 8, 16, 2, 128, 99, 4, 16),                       # one key over
    ([100, 300, 64, 65], 20, 16, 2, 64, 64, 4, 16),
    ([1, 0, 257, 256], 300, 1, 3, 128, 100, 0, 0),           # pages of one slot, no protected ones
    ([333, 200, 1000], 40, 25, 1, 128, 150, 10, 140),        # nothing but sinks and recent
    ([500, 480], 4, 128, 2, 64, 128, 0, 128),                # only the recent
    ([500, 480], 4, 128, 2, 64, 128, 128, 0),                # only the sinks
    ([600, 513], 40, 16, 8, 128, 512, 4, 500),               # a recent block that overlaps its target
    ([5000, 4097, 3000], 20, 256, 1, 128, 1500, 7, 1001),    # over 1024 slots a pass, odd blocks
    ([700] * 40, 6, 128, 4, 64, 256, 4, 32),                 # more heads than SMs
    ([9], 3, 4, 1, 64, 1, 0, 0),
    ([9], 3, 4, 1, 64, 1, 0, 1),
    ([9], 3, 4, 1, 64, 40, 3, 7),                            # a budget past the table
]


@pytest.mark.parametrize("inplace", [True, False], ids=["inplace", "out"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "n%s_P%d_H%d_d%d_%d_%d_%d" % (
    "_".join(map(str, c[0][:3])), c[2], c[3], c[4], c[5], c[6], c[7]))
def test_evict(attn, case, inplace):
    run(attn, *case, seed=sum(case[0]), inplace=inplace)


def ties(rng, shape):
    return rng.integers(0, 3, shape).astype(np.float32)


def zeros(rng, shape):
    return np.where(rng.random(shape) < 0.5, np.float32(0.0), np.float32(-0.0)).astype(np.float32)


def odd(rng, shape):
    w = rng.standard_normal(shape).astype(np.float32)
    pick = rng.integers(0, 8, shape)
    for i, x in enumerate((np.nan, np.inf, -np.inf, 1e-45, -1e-45)):
        w[pick == i] = x
    w.view(np.uint32)[pick == 5] = 0xFFC00001             # a NaN with the sign bit
    return w


def rising(rng, shape):
    return np.broadcast_to(np.arange(shape[-1], dtype=np.float32), shape).copy()


def falling(rng, shape):
    return -rising(rng, shape)


@pytest.mark.parametrize("weights", [ties, zeros, odd, rising, falling], ids=lambda f: f.__name__)
@pytest.mark.parametrize("protected", [(4, 30), (0, 0), (50, 3)])
def test_weights_of_every_kind(attn, weights, protected):
    run(attn, [400, 1300, 130], 11, 128, 2, 64, 129, *protected, seed=3, weights=weights)


def spread(rng, shape):
    return (rng.standard_normal(shape) * 10.0 ** rng.integers(-30, 30, shape)).astype(np.float32)


def near(rng, shape):
    return (1.0 + rng.random(shape) / 16).astype(np.float32)      # all in one bin of the upper bits


@pytest.mark.parametrize("weights", [ties, zeros, odd, spread, near], ids=lambda f: f.__name__)
@pytest.mark.parametrize("n", [9000, 40000, 140000, 300000])
def test_long_caches(attn, n, weights):
    # a few CTAs a head that hold the keys; 300,000 slots are more than sixteen hold
    run(attn, [n, n // 3], -(-n // 512), 512, 1, 64, n // 4, 5, n // 9, seed=n, weights=weights, inplace=n != 40000)


def test_again_and_again(attn):
    # a cache that grows by a chunk and is cut, with the recent window kept in order at the end
    P, Hkv, d, budget, recent, chunk, most = 16, 2, 64, 100, 20, 17, 8
    kc, vc, table = cache([0], most, P, Hkv, d, 9)
    k, v, t = kc.cuda(), vc.cuda(), torch.as_tensor(table).cuda()
    w, lens = torch.zeros((1, Hkv, most * P), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rng, made = np.random.default_rng(4), 0
    for _ in range(25):
        n = lens.item()
        for j in range(n, n + chunk):                        # token number in every element of its key
            k[table[0, j // P], j % P] = v[table[0, j // P], j % P] = float(made % 256)
            made += 1
        lens += chunk
        w[:, :, :n + chunk] += torch.as_tensor(rng.random((1, Hkv, n + chunk)).astype(np.float32)).cuda()
        attn.attn_paged_evict(k, v, w, lens, t, budget, sinks=2, recent=recent)
        now = lens.item()
        assert now == min(n + chunk, budget) and not w[:, :, now:].any()
        for c in (k, v):
            flat = c[t[0].long()].flatten(0, 1)[:now, :, 0].float().cpu().numpy()
            tail = min(recent, now)
            assert np.array_equal(flat[now - tail:], np.repeat(np.arange(made - tail, made) % 256, Hkv).reshape(-1, Hkv))
            assert np.array_equal(flat[:2], [[0] * Hkv, [1] * Hkv])
    status_ok(attn)


def test_bad_and_shared_sequences_stay(attn):
    lens, most, P, Hkv, d = [100, 120, 110, 20, 115, 90, 128], 8, 16, 2, 64
    kc, vc, table = cache(lens, most, P, Hkv, d, 5)
    w = np.random.default_rng(6).random((7, Hkv, most * P)).astype(np.float32)
    table, said = table.copy(), list(lens)
    table[1, 3] = kc.shape[0]              # not in the cache
    table[2, 1] = table[3, 0]              # shared with a sequence that is not cut
    said[4] = most * P + 1
    table[5, 2] = table[5, 4]              # twice in one sequence
    ok = [0, 6]
    cut = [n if b in ok else 0 for b, n in enumerate(lens)]
    ek, ev, ew, en = expect(kc, vc, table, w, cut, 64, 4, 8)
    en = [64 if b in ok else n for b, n in enumerate(said)]
    k, v, wd = kc.cuda(), vc.cuda(), torch.as_tensor(w).cuda()
    ld = torch.as_tensor(np.asarray(said, dtype=np.int32)).cuda()
    attn.attn_paged_evict(k, v, wd, ld, torch.as_tensor(table).cuda(), 64, sinks=4, recent=8)
    assert attn.cache_device_status() == (1, 23)
    assert ld.tolist() == en
    assert torch.equal(k.cpu().view(torch.int16), ek) and torch.equal(v.cpu().view(torch.int16), ev)
    assert np.array_equal(wd.cpu().numpy(), ew)
    # pages shared among sequences that fit are nobody's trouble
    attn.attn_paged_evict(k, v, wd, ld.clamp_(max=64), torch.as_tensor(table).cuda().clamp_(0, kc.shape[0] - 1), 64)
    status_ok(attn)


def test_refused_sequences_leave_the_outputs_of_their_own_alone(attn):
    kc, vc, table = cache([100, 110, 30], 8, 16, 2, 64, 15)
    table = table.copy()
    table[1, 2] = kc.shape[0] + 5
    w = torch.rand((3, 2, 128), generator=torch.Generator().manual_seed(1)).cuda()
    wo, lo = torch.full_like(w, -5.0), torch.full((3,), -5, dtype=torch.int32, device="cuda")
    k, v, lens = kc.cuda(), vc.cuda(), torch.tensor([100, 110, 30], dtype=torch.int32, device="cuda")
    keep = [t.clone() for t in (k, v, w, lens)]
    for recent in (8, 0):              # (the second time the kept rows have moved already; the refused ones never)
        attn.attn_paged_evict(k, v, w, lens, torch.as_tensor(table).cuda(), 64, sinks=4, recent=recent, weights_out=wo,
                              seqlens_out=lo)
        assert attn.cache_device_status() == (1, 23)
        assert lo.tolist() == [64, 110, 30] and torch.equal(w, keep[2]) and torch.equal(lens, keep[3])
        assert (wo[1] == -5.0).all() and torch.equal(wo[2, :, :30], w[2, :, :30]) and (wo[2, :, 30:] == -5.0).all()
        own = [p for p in table[1] if p < kc.shape[0]]
        for t, old in ((k, keep[0]), (v, keep[1])):
            assert torch.equal(t[own].view(torch.int16), old[own].view(torch.int16))


def test_what_the_binding_refuses(attn):
    kc, vc, table = cache([20], 2, 16, 2, 64, 3)
    k, v, t = kc.cuda(), vc.cuda(), torch.as_tensor(table).cuda()
    w, n = torch.zeros((1, 2, 32), device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    evict = attn.attn_paged_evict
    for call, error in (
            (lambda: evict(k, v[:2], w, n, t, 8), ValueError),
            (lambda: evict(k, v, w[:, :, :31].contiguous(), n, t, 8), ValueError),
            (lambda: evict(k, v, w.half(), n, t, 8), TypeError),
            (lambda: evict(k, v, w, n.long(), t, 8), TypeError),
            (lambda: evict(k, v, w, torch.cat([n, n]), t, 8), ValueError),
            (lambda: evict(k, v, w, n, t, 8, seqlens_out=torch.cat([n, n])), ValueError),
            (lambda: evict(k.transpose(1, 2), v.transpose(1, 2), w, n, t, 8), ValueError),
            (lambda: evict(k, k, w, n, t, 8), attn.AttnError),
            (lambda: evict(k, v, w, n, t, 0), attn.AttnError),
            (lambda: evict(k, v, w, n, t, 8, sinks=5, recent=4), attn.AttnError),
            (lambda: evict(k, v, w, n, t, 8, workspace=torch.empty(16, device="cuda")), attn.AttnError)):
        with pytest.raises(error):
            call()
    assert n.item() == 20
    status_ok(attn)


def test_guards(attn):
    lens, most, P, Hkv, d, budget = [300, 77], 20, 16, 3, 64, 100
    kc, vc, table = cache(lens, most, P, Hkv, d, 7)
    w = np.random.default_rng(8).random((2, Hkv, most * P)).astype(np.float32)
    ek, ev, ew, en = expect(kc, vc, table, w, lens, budget, 4, 30)
    a = attn.EvictArgs()
    a.B, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d = 2, Hkv, kc.shape[0], P, most, d
    a.budget, a.sinks, a.recent = budget, 4, 30
    need = int(attn.load().attn_paged_evict_workspace_size(ctypes.byref(a)))
    kb, k = guarded(kc.numel(), "bf16")
    vb, v = guarded(vc.numel(), "bf16")
    wb, wd = guarded(w.size, "f32")
    sb, ws = guarded(need, "ws")
    k.copy_(kc.flatten()), v.copy_(vc.flatten()), wd.copy_(torch.as_tensor(w).flatten())
    k.view(torch.int16).copy_(kc.flatten().view(torch.int16))
    v.view(torch.int16).copy_(vc.flatten().view(torch.int16))
    ld = torch.as_tensor(np.asarray(lens, dtype=np.int32)).cuda()
    attn.attn_paged_evict(k.view(kc.shape), v.view(vc.shape), wd.view(2, Hkv, most * P), ld,
                          torch.as_tensor(table).cuda(), budget, sinks=4, recent=30, workspace=ws)
    torch.cuda.synchronize()
    for buf, kind in ((kb, "bf16"), (vb, "bf16"), (wb, "f32"), (sb, "ws")):
        assert guards_intact(buf, kind)
    assert torch.equal(k.cpu().view(torch.int16).view(kc.shape), ek.view(kc.shape))
    assert torch.equal(v.cpu().view(torch.int16).view(vc.shape), ev.view(vc.shape))
    assert np.array_equal(wd.cpu().numpy().reshape(w.shape), ew) and ld.tolist() == en
    status_ok(attn)
