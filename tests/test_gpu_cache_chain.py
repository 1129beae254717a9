"""The operators around the paged cache together, as a decoding loop runs them (needs a GB300): rotate
and append, attend to the cache, accumulate weights, cut the caches to their budget, eagerly and as
one captured graph; and the prefill that fills the cache through attn_fwd_paged."""
import numpy as np
import pytest
import torch

import oracle
from tests import parity

pytestmark = pytest.mark.gpu

H, HKV, D, P, MOST = 8, 2, 128, 128, 3
BUDGET, SINKS, RECENT = 200, 4, 32


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


class Loop:
    """A decoding batch: one projection's rows in, attention outputs out."""

    def __init__(self, attn, B, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.attn, self.B, self.g = attn, B, g
        self.freqs, self.axes = attn.rope_freqs((32, 48, 48), spectrum="shared")
        self.kc = torch.zeros((B * MOST, P, HKV, D), dtype=torch.bfloat16, device="cuda")
        self.vc = torch.zeros_like(self.kc)
        self.table = torch.randperm(B * MOST, generator=g, device="cuda").to(torch.int32).view(B, MOST)
        self.weights = torch.zeros((B, HKV, MOST * P), device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.x = torch.empty((B, H + 2 * HKV, D), dtype=torch.bfloat16, device="cuda")
        self.pos = torch.zeros((3, B), dtype=torch.int32, device="cuda")
        self.cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def prefill(self, lens):
        total = sum(lens)
        x = torch.randn((total, H + 2 * HKV, D), generator=self.g, device="cuda").to(torch.bfloat16)
        cu = torch.as_tensor(np.cumsum([0] + list(lens)).astype(np.int32)).cuda()
        pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda().expand(3, total).contiguous()
        self.lens.copy_(torch.as_tensor(np.asarray(lens, dtype=np.int32)))
        self.pos.copy_(self.lens.expand(3, -1))
        q = self.attn.attn_paged_append(x[:, H:H + HKV], x[:, H + HKV:], self.kc, self.vc, cu, self.lens, self.table,
                                        q=x[:, :H], positions=pos, freqs=self.freqs, axes=self.axes, pairing="halves")
        return q, cu, self.attn.attn_fwd_paged(q, self.kc, self.vc, cu, self.lens, self.table, causal=True)

    def step(self):
        self.lens += 1
        q = self.attn.attn_paged_append(self.x[:, H:H + HKV], self.x[:, H + HKV:], self.kc, self.vc, self.cu, self.lens,
                                        self.table, q=self.x[:, :H], positions=self.pos, freqs=self.freqs,
                                        axes=self.axes, pairing="halves")
        o = self.attn.attn_paged_decode(q, self.kc, self.vc, self.lens, self.table, weights=self.weights)
        self.attn.attn_paged_evict(self.kc, self.vc, self.weights, self.lens, self.table, BUDGET, sinks=SINKS,
                                   recent=RECENT)
        self.pos += 1
        return q, o

    def state(self):
        return [t.clone() for t in (self.kc, self.vc, self.weights, self.lens)]


def test_prefill_and_decoding_match_the_oracle(attn):
    lp = Loop(attn, 3, 1)
    lens = [190, 60, 200]
    q, cu, o = lp.prefill(lens)
    ref = oracle.attention_paged(q.cpu(), lp.kc.cpu(), lp.vc.cpu(), cu.cpu().numpy(), lens, lp.table.cpu().numpy(),
                                 causal=True, want_a=True)
    res = parity.compare(o.cpu().view(torch.int16).numpy().view(np.uint16).reshape(-1, D),
                         ref["o_bits"].reshape(-1, D), ref["a"].reshape(-1, D))
    assert res["ok"], res
    for i in range(24):
        lp.x.normal_(generator=lp.g)
        before = [t.clone() for t in (lp.lens, lp.weights)]
        kept = lp.attn.attn_paged_evict
        # the cache as the attention sees it: after the append, before the eviction
        seen = {}

        def spy(*a, **kw):
            seen["k"], seen["v"], seen["n"], seen["w"] = lp.kc.clone(), lp.vc.clone(), lp.lens.clone(), lp.weights.clone()
            return kept(*a, **kw)

        lp.attn.attn_paged_evict = spy
        try:
            q, o = lp.step()
        finally:
            lp.attn.attn_paged_evict = kept
        n = seen["n"].tolist()
        assert n == [x + 1 for x in before[0].tolist()] and lp.lens.tolist() == [min(x, BUDGET) for x in n]
        ref = oracle.attention_paged(q.cpu(), seen["k"].cpu(), seen["v"].cpu(), np.arange(4), n,
                                     lp.table.cpu().numpy(), want_a=True)
        res = parity.compare(o.cpu().view(torch.int16).numpy().view(np.uint16).reshape(-1, D),
                             ref["o_bits"].reshape(-1, D), ref["a"].reshape(-1, D))
        assert res["ok"], (i, res)
        # each of the query heads spends a weight of one
        added = (seen["w"].double() - before[1].double()).sum((1, 2))
        assert ((added - H).abs() < 1e-3).all()
        assert not lp.weights[0, :, BUDGET:].any()
    assert attn.cache_device_status() == (0, 0) and attn.device_status()[0] == 0


def test_the_loop_as_a_graph(attn):
    eager, graphed = Loop(attn, 4, 2), Loop(attn, 4, 2)
    for lp in (eager, graphed):
        lp.prefill([180, 199, 1, 230])
    start = graphed.state() + [graphed.pos.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step()                                   # warm-up, then the state as it was
        for t, s in zip((graphed.kc, graphed.vc, graphed.weights, graphed.lens, graphed.pos), start):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, o = graphed.step()
    g = torch.Generator("cuda").manual_seed(5)
    for i in range(40):
        eager.x.normal_(generator=g)
        graphed.x.copy_(eager.x)
        _, want = eager.step()
        graph.replay()
        assert torch.equal(o.view(torch.int16), want.view(torch.int16)), i
    for a, b in zip(eager.state(), graphed.state()):
        assert torch.equal(a, b)
    assert attn.cache_device_status() == (0, 0)


def test_caches_past_four_gigabytes(attn):
    """Pages whose byte offsets pass 2^32: append, attend and evict there as in a small cache of the same pages."""
    B, H, Hkv, d, ps, n = 2, 8, 8, 128, 128, 300
    pages = 2 ** 32 // (ps * Hkv * d * 2) + 8                       # 4 GiB of keys and eight pages
    g = torch.Generator("cuda").manual_seed(3)
    far = torch.tensor([[pages - 1, 1, pages - 4], [pages - 2, pages - 3, 0]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device="cuda")
    x = torch.randn((B * n, H + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    w = torch.rand((B, Hkv, 3 * ps), generator=g, device="cuda")
    out = []
    for table, count in ((near, 6), (far, pages)):
        kc, vc = (torch.empty((count, ps, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lens, weights = torch.full((B,), n, dtype=torch.int32, device="cuda"), w.clone()
        attn.attn_paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, cu, lens, table)
        q = x[:B, :H].contiguous()
        o = attn.attn_paged_decode(q, kc, vc, lens, table, weights=weights)
        attn.attn_paged_evict(kc, vc, weights, lens, table, 200, sinks=3, recent=50)
        o2 = attn.attn_paged_decode(q, kc, vc, lens, table)
        out.append((o, o2, weights, lens, kc[table.long()].flatten(1, 2)[:, :200], vc[table.long()].flatten(1, 2)[:, :200]))
        del kc, vc
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert attn.cache_device_status() == (0, 0)


def test_rotary_positions_of_a_tensor_past_two_to_the_31_elements(attn):
    S, H, d = 131080, 128, 128
    freqs, axes = attn.rope_freqs((128,))
    q = torch.empty((1, S, H, d), dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 2 ** 31
    q[:, -4:].normal_()
    positions = torch.arange(S, dtype=torch.int32, device="cuda")[None]
    tail = q[:, -4:].clone()
    attn.attn_rope(q, None, positions, freqs, axes, q_out=q)
    want = attn.attn_rope(tail, None, positions[:, -4:], freqs, axes)
    assert torch.equal(q[:, -4:], want)
    assert attn.cache_device_status() == (0, 0)
