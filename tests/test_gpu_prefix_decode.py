"""Attention of one new token per sequence behind a prefix that the batch shares (attn_paged_prefix_decode) against plain
fp64 attention over each sequence's keys (needs a GB300).

Tolerance, derived before the first run.  With A = sum_j w_j |v_j| / l (the softmax weights' sum of magnitudes): each weight of the
prefix is rounded to bf16, 2^-8 relative, the own keys' to 2^-15; fp32 logits off by d * 2^-24 of their magnitudes (below
2^-13 here), exponentials, sums and joins below 2^-13 together; the output's rounding is 2^-8 relative (RTNE, RTNA), 2^-7
(RTZ).  So |o - ref| <= 2^-8 |ref| + (2^-8 + 2^-12) A.  The log-sum-exp takes the unrounded weights: 2^-14 (1 + |lse|) + 2^-12.
"""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN_BITS = 0x7FC0


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


def draw(*shape, seed=0, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16).cuda()


class Batch:
    """Sequences of `own` keys behind a prefix; the table's other rows name no page that only the prefix uses."""

    def __init__(self, own, H, Hkv, d, page, prefix, seed=0, scale=1.0, spare=1, hidden=-7):
        B = len(own)
        self.H, self.Hkv, self.d, self.page, self.prefix = H, Hkv, d, page, prefix
        lens = [prefix + n for n in own]
        cut, most = prefix // page, -(-max(lens) // page) + spare
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(cut + B * (most - cut) + 3, generator=g).to(torch.int32)
        table = torch.full((B, most), hidden, dtype=torch.int32)
        table[0, :cut] = order[:cut]
        table[:, cut:] = order[cut:cut + B * (most - cut)].view(B, most - cut)
        for b, n in enumerate(lens):
            table[b, max(-(-n // page), -(-prefix // page) if b == 0 else 0):] = hidden     # nothing behind the last page
        self.table, self.lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.k, self.v = draw(len(order), page, Hkv, d, seed=seed + 1), draw(len(order), page, Hkv, d, seed=seed + 2)
        self.q = draw(B, H, d, seed=seed + 3, scale=scale)

    def keys(self, b):
        """Keys and values of sequence b, in order, fp64 [keys, Hkv, d]."""
        n, page = int(self.lens[b]), self.page
        j = torch.arange(n)
        t = self.table.cpu()
        row = torch.where(j < self.prefix, t[0, j // page], t[b, j // page]).long() * page + j % page
        return [c.cpu().flatten(0, 1)[row].double().numpy() for c in (self.k, self.v)]

    def reference(self, b):
        k, v = self.keys(b)
        G, q = self.H // self.Hkv, self.q[b].cpu().double().numpy()
        o, lse, A = np.empty((self.H, self.d)), np.empty(self.H), np.empty((self.H, self.d))
        for h in range(self.H):
            x = k[:, h // G] @ q[h] / np.sqrt(self.d)
            m = x.max()
            w = np.exp(x - m)
            o[h], A[h] = w @ v[:, h // G] / w.sum(), w @ np.abs(v[:, h // G]) / w.sum()
            lse[h] = m + np.log(w.sum())
        return o, lse, A

    def call(self, attn, **kw):
        return attn.attn_paged_prefix_decode(self.q, self.k, self.v, self.lens, self.table, self.prefix, return_lse=True, **kw)

    def check(self, got, rows=None, out=2.0 ** -8):
        o, lse = (x.cpu().double().numpy() for x in got)
        for b in range(len(self.lens)) if rows is None else rows:
            ref, ref_lse, A = self.reference(b)
            err = np.abs(o[b] - ref) - (out * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A)
            assert np.all(err <= 0), (b, float(err.max()))
            assert np.all(np.abs(lse[b] - ref_lse) <= 2.0 ** -14 * (1 + np.abs(ref_lse)) + 2.0 ** -12), b


def alone(x):
    """Whether the rule sends a call to the decoding kernel alone: by sequences * K/V heads * (tiles of the prefix + 2) against 17 an SM
    (2,584 on 152)."""
    group, B = x.H // x.Hkv, len(x.lens)
    rows = B * x.Hkv * -(-group // (8 if group <= 8 else 16 if group <= 16 else 32))
    return B == 1 or rows * (-(-x.prefix // 128) + 2) <= 17 * torch.cuda.get_device_properties(0).multi_processor_count


# "few" cases go to the decoding kernel alone, "many" to the shared prefix's kernels
FEW = [  # own keys, H, Hkv, d, page, prefix
    ([1], 8, 8, 128, 16, 1),
    ([0], 4, 2, 64, 16, 40),
    ([9], 4, 2, 64, 16, 40000),                      # one sequence shares with nobody
    ([0, 0, 0], 6, 2, 128, 32, 64),                  # no sequence has a key of its own
    ([5, 0, 300, 1, 129], 8, 2, 128, 16, 127),
    ([3, 77, 128], 24, 3, 64, 7, 129),
    ([7] * 9, 71, 1, 64, 100, 777),
    ([2000, 1, 4000], 8, 8, 64, 16, 90),
]
MANY = [
    ([2, 0, 40, 1] * 32, 8, 8, 128, 16, 1),          # 128 rows against one key
    ([1] * 128, 8, 8, 64, 7, 129),
    ([0] * 128, 8, 8, 128, 24, 257),                 # no own keys; an odd number of tiles
    ([3, 300] * 9, 64, 8, 128, 100, 2100),
    ([5] * 15, 64, 8, 128, 1, 2500),                 # a page a key
    ([1, 2, 0], 8, 8, 128, 512, 14000),              # three rows of many parts
    ([64, 1] * 22, 12, 12, 128, 3, 300),
    ([2, 300] * 16 + [9], 32, 8, 128, 256, 1000),    # 132 rows: two tiles of them
    ([1, 40, 0, 17] * 13, 40, 8, 128, 24, 2500),     # 260: a second block of rows
    ([7] * 60, 71, 1, 64, 100, 3000),
    ([11, 500] * 7, 142, 2, 128, 64, 6000),
    ([300, 1] * 150, 4, 1, 64, 16, 900),
    ([1, 0, 130] * 300, 3, 1, 128, 48, 1),
    ([0, 3] * 220, 8, 2, 128, 128, 128),             # whole tiles only
    ([0, 1, 0, 0, 90] * 340, 2, 1, 64, 16, 200),     # more sequences than a block has threads
    ([0] * 1500 + [33] * 3, 5, 1, 128, 8, 77),       # only the last ones have keys of their own
]
CASES = FEW + MANY


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_H%d_%d_d%d_p%d_%d" % (len(c[0]), *c[1:]))
def test_against_plain_attention(attn, case):
    x = Batch(*case, seed=len(case[0]) + case[5], scale=2.0)
    assert alone(x) == (case in FEW)
    got = x.call(attn)
    assert attn.cache_device_status() == (0, 0)
    B = len(case[0])
    x.check(got, rows=sorted({0, 1, 2, B // 2, B - 2, B - 1, *range(0, B, max(1, B // 12))} & set(range(B))))
    assert got[0].isfinite().all() and got[1].isfinite().all()
    again = x.call(attn)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(attn, seed):
    g = np.random.default_rng(seed)
    Hkv, G, d = int(g.integers(1, 9)), int(g.integers(1, 12)), int(g.choice([64, 128]))
    B, page = int(g.integers(1, 80)) if seed % 2 else int(g.integers(150, 400)), int(g.choice([1, 3, 8, 16, 48, 128, 300]))
    own = g.integers(0, int(g.choice([2, 40, 400])), B).tolist()
    x = Batch(own, Hkv * G, Hkv, d, page, int(g.integers(1, 1500)), seed=100 + seed, scale=float(g.choice([0.1, 1, 4])))
    x.check(x.call(attn), rows=sorted(set(g.integers(0, B, 6).tolist())))
    assert attn.cache_device_status() == (0, 0)


@pytest.mark.parametrize("times", [1, 40])
@pytest.mark.parametrize("mode", ["rtna", "rtz"])
def test_rounding_modes(attn, mode, times):
    x = Batch([10, 90, 3] * times, 16, 4, 128, 16, 2000, seed=4)
    assert alone(x) == (times == 1)
    near, other = x.call(attn), x.call(attn, round=mode)
    x.check(other, rows=[0, 1, 2], out=2.0 ** -8 if mode == "rtna" else 2.0 ** -7)
    step = (other[0].view(torch.int16).int() - near[0].view(torch.int16).int()).abs()
    assert step.max() <= 1 and torch.equal(near[1], other[1])


@pytest.mark.parametrize("times", [1, 10])
def test_equals_the_plain_decoding_call_where_pages_are_shared(attn, times):
    """The same caches through attn_paged_decode, whose rows name the prefix's pages too."""
    x = Batch([40, 0, 200, 7] * times, 32, 8, 128, 16, 960, seed=9, scale=2.0)
    assert alone(x) == (times == 1)
    got = x.call(attn)
    table = x.table.clone()
    table[:, :60] = table[0, :60]
    want = attn.attn_paged_decode(x.q, x.k, x.v, x.lens, table, return_lse=True)
    assert (got[0].float() - want[0].float()).norm() <= 2.0 ** -7 * want[0].float().norm()
    assert (got[1] - want[1]).abs().max() <= 1e-4
    # rows that name the shared pages change nothing, nor do other sequences
    assert torch.equal(attn.attn_paged_prefix_decode(x.q, x.k, x.v, x.lens, table, 960), got[0])


@pytest.mark.parametrize("rows", [4, 700])
def test_non_finite_keys_and_values(attn, rows):
    """Of the prefix and of own keys, as in attn_paged_decode: the same classes of outputs."""
    x = Batch([50, 3, 0, 20] * (rows // 4) + [8] * (rows % 4), 8, 1, 128, 16, 160, seed=rows)
    assert alone(x) == (rows == 4)
    k, v = x.k.flatten(0, 1), x.v.flatten(0, 1)
    page = x.table[0].cpu()

    def slot(b, j):
        t = page if j < x.prefix else x.table[b].cpu()
        return int(t[j // 16]) * 16 + j % 16
    table = x.table.clone()
    table[:, :10] = table[0, :10]
    cases = [(k, 0, 5, float("nan")), (k, 0, 130, float("inf")), (k, 0, 131, float("-inf")), (v, 0, 7, float("inf")),
             (v, 0, 9, float("nan")), (k, 1, 161, float("nan")), (v, 1, 162, float("-inf")), (k, 0, 170, float("inf"))]
    for c, b, j, value in cases:
        at = slot(b, j)
        kept = c[at].clone()
        c[at, :, 3] = value
        got, want = x.call(attn), attn.attn_paged_decode(x.q, x.k, x.v, x.lens, table, return_lse=True)
        for a, w in zip(got, want):
            assert torch.equal(a.isnan(), w.isnan()) and torch.equal(a.isinf(), w.isinf())
            assert torch.equal(a[a.isinf()], w[w.isinf()])
        assert set(got[0][got[0].isnan()].view(torch.int16).tolist()) <= {NAN_BITS}
        c[at] = kept


@pytest.mark.parametrize("times", [1, 350])
def test_infinite_values_under_vanishing_weights(attn, times):
    """A finite logit weighs something, however small: an infinite value stays infinite."""
    x = Batch([3, 20] * times, 4, 1, 64, 16, 200, seed=5)
    assert alone(x) == (times == 1)
    x.q.fill_(4.0)
    k, v = x.k.flatten(0, 1), x.v.flatten(0, 1)
    k[int(x.table[0, 2]) * 16 + 1] = 64.0            # stands far out: every other weight underflows
    k[int(x.table[0, 3]) * 16 + 2] = -64.0
    v[int(x.table[0, 3]) * 16 + 2, 0, 5] = float("inf")
    got = x.call(attn)[0]
    assert torch.isposinf(got[:, :, 5]).all() and got[:, :, :5].isfinite().all()


@pytest.mark.parametrize("times", [1, 120])
def test_all_logits_minus_infinity(attn, times):
    x = Batch([3, 0, 20] * times, 4, 2, 128, 16, 150, seed=5)
    assert alone(x) == (times == 1)
    x.q.fill_(1.0)
    x.k.fill_(float("-inf"))
    o, lse = x.call(attn)
    assert o.isnan().all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("B,prefix", [(5, 96), (100, 2000)])
def test_sequences_that_have_ended(attn, B, prefix):
    x = Batch([30, 4, 200, 9, 1] + [3] * (B - 5), 8, 2, 128, 16, prefix, seed=2)
    assert alone(x) == (B == 5)
    x.lens[[0, 3]] = 0
    o, lse = x.call(attn)
    assert attn.cache_device_status() == (0, 0)
    assert (o[[0, 3]].view(torch.int16) == NAN_BITS).all() and torch.isneginf(lse[[0, 3]]).all()
    x.check((o, lse), rows=[1, 2, 4])


def many(own, H, Hkv, d, page, prefix, seed=0):
    """A batch that is too large for the decoding kernel alone."""
    return Batch(own + [2] * 95, H, Hkv, d, page, prefix, seed=seed)


def far(own, H, Hkv, d, page, prefix, seed=0):
    """One tile of rows behind a long prefix."""
    return Batch(own + [2] * 25, H, Hkv, d, page, 6 * prefix, seed=seed)


@pytest.mark.parametrize("make", [Batch, many, far])
def test_bad_lengths_and_pages_leave_their_rows(attn, make):
    def run(x, **kw):
        o, lse = torch.full_like(x.q, 7.0), torch.full((len(x.lens), x.H), 7.0, device="cuda")
        x.call(attn, o=o, lse=lse)
        return o, lse
    x = make([30, 4, 200, 9, 0], 8, 2, 128, 16, 5 * 16 if make is Batch else 2000, seed=2)
    assert alone(x) == (make is Batch)
    room = x.table.shape[1] * 16
    for length in (x.prefix - 1, -1, 1, room + 1, 2 ** 31 - 1):
        kept = int(x.lens[2])
        x.lens[2] = length
        o, lse = run(x)
        assert attn.cache_device_status() == (1, 22) and (o[2] == 7).all() and (lse[2] == 7).all()
        x.lens[2] = kept
        x.check((o, lse), rows=[0, 1, 3, 4])
    for page in (-1, len(x.k), 2 ** 31 - 1):
        at = x.prefix // 16 + 2
        kept = int(x.table[2, at])
        x.table[2, at] = page
        o, lse = run(x)
        assert attn.cache_device_status() == (1, 22) and (o[2] == 7).all() and (lse[2] == 7).all()
        x.table[2, at] = kept
        x.check((o, lse), rows=[0, 1, 3, 4])
    last = x.prefix // 16 - 1
    for at, page in ((2, len(x.k)), (last, -1), (2, -2 ** 31), (last, 2 ** 31 - 1)):      # of the prefix: nobody's outputs are written
        kept = int(x.table[0, at])
        x.table[0, at] = page
        o, lse = run(x)
        assert attn.cache_device_status() == (1, 26) and (o == 7).all() and (lse == 7).all()
        x.table[0, at] = kept
    x.check(run(x), rows=[0, 1, 2, 3, 4])
    assert attn.cache_device_status() == (0, 0)


def test_stays_in_bounds_with_the_caller_s_workspace(attn):
    x = Batch([30, 4, 700] * 40, 10, 2, 128, 24, 1111, seed=2)
    assert not alone(x)
    want = x.call(attn)
    a = attn.DecodeArgs()
    a.B, a.H, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d = 120, 10, 2, len(x.k), 24, x.table.shape[1], 128
    need = int(attn.load().attn_paged_prefix_decode_workspace_size(ctypes.byref(a), 1111))
    assert need > 0
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    room, lses = torch.full((64 + x.q.numel() + 64,), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((1200 + 64,), 3.0, device="cuda")
    got = x.call(attn, o=room[64:-64].view_as(x.q), lse=lses[32:-32].view(120, 10), workspace=ws[:need])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[:64] == 3).all() and (room[-64:] == 3).all() and (lses[:32] == 3).all() and (lses[-32:] == 3).all()
    assert (ws[need:] == 0xFF).all()
    with pytest.raises(attn.AttnError):
        x.call(attn, workspace=ws[:need - 256])
    with pytest.raises(ValueError):
        attn.attn_paged_prefix_decode(x.q, x.k, x.v, x.lens, x.table, x.table.shape[1] * 24 + 1)


@pytest.mark.parametrize("times", [1, 20])
def test_rows_past_2_to_the_32_bytes(attn, times):
    """A cache of 5 GB, its pages at the far end."""
    x = Batch([30, 4, 200] * times, 8, 8, 128, 128, 700, seed=3)
    assert alone(x) == (times == 1)
    far = 2_400_000 // 128
    k, v = (torch.zeros((far + len(x.k), 128, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[far:], v[far:] = x.k, x.v
    table = torch.where(x.table >= 0, x.table + far, x.table)
    got = attn.attn_paged_prefix_decode(x.q, k, v, x.lens, table, 700, return_lse=True)
    want = x.call(attn)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("times,prefix", [(1, 200), (40, 1500)])
def test_captured_while_lengths_grow(attn, times, prefix):
    B, cut = 3 * times, prefix // 16
    x = Batch([1, 30, 4] * times, 8, 2, 128, 16, prefix, seed=7, spare=3)
    assert alone(x) == (times == 1)
    t = torch.arange(len(x.k), dtype=torch.int32)
    x.table[:, cut:] = t[cut:cut + B * (x.table.shape[1] - cut)].view(B, -1).cuda()
    x.table[0, :cut] = t[:cut].cuda()
    x.call(attn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = x.call(attn)
    for _ in range(4):
        x.lens.add_(1)
        x.q.copy_(draw(B, 8, 128, seed=int(x.lens[0])))
        graph.replay()
        x.check(got, rows=[0, 1, 2, B - 1])
        assert all(torch.equal(a, b) for a, b in zip(got, x.call(attn)))


def test_two_streams_with_workspaces_of_their_own(attn):
    batches = [Batch([30, 4, 700] * 40, 8, 2, 128, 16, 1500, seed=s) for s in (1, 2)]
    want = [x.call(attn) for x in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = [x.call(attn, stream=s) for x, s in zip(batches, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
