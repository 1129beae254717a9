"""The calls of a serving step together, as a program makes them (needs a GB300): attn_paged_reserve gives the new tokens their
pages and slots, attn_norm_rope_append writes them, attn_paged_prefix_decode attends behind the shared prefix; sequences end and
others take their pages; eagerly, on streams, and as one graph.  Against plain fp64 arithmetic over all tokens so far."""
import numpy as np
import pytest
import torch

from tests import norm_rope_ref as ref

pytestmark = pytest.mark.gpu

EPS, PAGE, H, HKV, D = 1e-6, 16, 8, 2, 64


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


class Server:
    """A batch of B sequences behind one prefix; `history` holds every sequence's tokens (k, v as projected)."""

    def __init__(self, attn, B, prefix, most, seed=0):
        self.attn, self.B, self.prefix = attn, B, prefix
        g = self.g = torch.Generator("cuda").manual_seed(seed)
        self.freqs, self.axes = attn.rope_freqs((D,))
        self.w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")) for _ in range(2)]
        shared, room = prefix // PAGE, -(-(prefix + most) // PAGE)
        pages = shared + B * (room - shared) // 2                    # not enough for all at their longest
        self.kc, self.vc = (torch.full((pages, PAGE, HKV, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((B, room), -1, dtype=torch.int32, device="cuda")
        self.table[:, :shared] = order[:shared]
        self.free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        self.free[:pages - shared] = order[shared:]
        self.count = torch.tensor([pages - shared], dtype=torch.int32, device="cuda")
        self.held = torch.full((B,), shared, dtype=torch.int32, device="cuda")
        self.shared = self.held.clone()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.history = [None] * B
        # the prefix, written once through sequence 0's row
        assert prefix % PAGE == 0
        x = self.draw(prefix)
        slots = (order[:shared].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
        self.write(x, slots, torch.arange(prefix, dtype=torch.int32, device="cuda"))
        self.first = x

    def draw(self, n):
        return torch.randn((n, H + 2 * HKV, D), generator=self.g, device="cuda").to(torch.bfloat16)

    def write(self, x, slots, positions):
        return self.attn.attn_norm_rope_append(x[:, H:H + HKV], x[:, H + HKV:], self.kc, self.vc, slots, q=x[:, :H], q_weight=self.w[0],
                                               k_weight=self.w[1], positions=positions[None], freqs=self.freqs, axes=self.axes, eps=EPS,
                                               pairing="halves")

    def step(self, x, cu, positions=None, slots=None):
        """New tokens x (lens already with them): their queries as written."""
        n = x.shape[0]
        slots = torch.empty(n, dtype=torch.int64, device="cuda") if slots is None else slots
        positions = torch.empty(n, dtype=torch.int32, device="cuda") if positions is None else positions
        self.attn.attn_paged_reserve(self.lens, cu, self.table, self.held, self.free, self.count, PAGE, shared_pages=self.shared,
                                     slots=slots, positions=positions)
        return self.write(x, slots, positions)

    def decode(self, q):
        return self.attn.attn_paged_prefix_decode(q, self.kc, self.vc, self.lens, self.table, self.prefix, return_lse=True)

    def begin(self, which, news):
        """Sequences `which` (that have ended, or are new) begin with prompts of `news` tokens behind the prefix."""
        counts = torch.zeros(self.B, dtype=torch.int32)
        counts[which] = torch.tensor(news, dtype=torch.int32)
        cu = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).to(torch.int32)]).cuda()
        x = self.draw(int(cu[-1]) + 3)                               # and three rows of padding
        self.lens[which] = torch.tensor(news, dtype=torch.int32, device="cuda") + self.prefix
        self.step(x, cu)
        for b in which:
            self.history[b] = x[int(cu[b]):int(cu[b + 1])]

    def end(self, which):
        self.lens[which] = 0
        for b in which:
            self.history[b] = None

    def turned(self, x, w, first):
        pos = np.arange(first, first + x.shape[0])[None]
        return ref.forward(x.cpu().double().numpy(), w.cpu().double().numpy(), EPS, pos, self.freqs.cpu().numpy(),
                           self.axes.cpu().numpy(), "halves")[0]

    def check(self, out, rows):
        """out against attention of the last token over the whole history.  Beside the bound of attn_paged_prefix_decode: keys and queries
        are bf16 roundings of normed ones, 2^-8 relative each, so logits are off by 2^-7 |q| |k| / sqrt(d) <= 2^-7 * 1.4^2 * 8 at
        the norms' lengths here, relative weights by that, the output by it times A (twice: the sum in the divisor)."""
        o, lse = (t.cpu().double().numpy() for t in out)
        for b in rows:
            if self.history[b] is None:
                assert np.isnan(o[b]).all() and (lse[b] == -np.inf).all()
                continue
            x = torch.cat([self.first, self.history[b]])
            k, v = self.turned(x[:, H:H + HKV], self.w[1], 0), x[:, H + HKV:].cpu().double().numpy()
            q = self.turned(x[-1:, :H], self.w[0], len(x) - 1)[0]
            for h in range(H):
                kh, vh = k[:, h // (H // HKV)], v[:, h // (H // HKV)]
                s = kh @ q[h] / np.sqrt(D)
                off = 2.0 ** -7 * (np.abs(kh) @ np.abs(q[h])).max() / np.sqrt(D)
                p = np.exp(s - s.max())
                want, A = p @ vh / p.sum(), p @ np.abs(vh) / p.sum()
                assert np.all(np.abs(o[b, h] - want) <= 2.0 ** -8 * np.abs(want) + (2 * off + 2.0 ** -7) * A), (b, h)
                assert abs(lse[b, h] - (s.max() + np.log(p.sum()))) <= off + 1e-3


@pytest.mark.parametrize("B,prefix", [(6, 48), (64, 4096)])      # the decoding kernel alone; the prefix's own kernels
@pytest.mark.parametrize("where", ["current", "stream", "graph"])
def test_serving(attn, B, prefix, where):
    s = Server(attn, B, prefix, most=96, seed=B)
    some = [0, 1, 2, B - 1]
    s.begin(list(range(B)), [5 + 7 * b % 23 for b in range(B)])
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    x, slots, positions = s.draw(B), torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")

    def turn():
        s.lens.add_((s.lens > 0).int())
        # (ended sequences have no token: their places are empty)
        cu = torch.cat([one[:1], (s.lens > 0).int().cumsum(0).to(torch.int32)])
        order = torch.where(s.lens > 0, cu[1:] - 1, B - 1).long()
        live = torch.zeros_like(x)
        live[order] = x                                            # the step's rows, packed
        q = s.step(live, cu, positions, slots)
        return s.decode(q[order])

    stream = torch.cuda.Stream() if where == "stream" else None
    graph, out = None, None
    if where == "graph":
        keep = [t.clone() for t in (s.lens, s.table, s.held, s.free, s.count, s.kc, s.vc)]
        turn()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = turn()
        for t, k in zip((s.lens, s.table, s.held, s.free, s.count, s.kc, s.vc), keep):
            t.copy_(k)
    for i in range(24):
        x.copy_(s.draw(B))
        if graph is not None:
            graph.replay()
        elif stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                out = turn()
            torch.cuda.current_stream().wait_stream(stream)
        else:
            out = turn()
        for b in range(B):
            if s.history[b] is not None:
                s.history[b] = torch.cat([s.history[b], x[b:b + 1]])
        if i % 6 == 5:
            s.check(out, some)
        if i == 8:
            s.end([1, B - 1])
        if i == 14:
            s.begin([1], [30])
    assert attn.cache_device_status() == (0, 0)
    # every page is somebody's or free
    held, table, n = s.held.tolist(), s.table.tolist(), int(s.count)
    owned = [p for b in range(B) for p in table[b][prefix // PAGE:held[b]]] + table[0][:prefix // PAGE] + s.free[:n].tolist()
    assert sorted(owned) == list(range(len(s.kc)))


def test_running_out_of_pages_changes_nothing(attn):
    """The step that finds too few pages writes no token: append passes over slots of -1."""
    s = Server(attn, 4, 32, most=64, seed=1)
    s.begin([0, 1], [40, 30])
    before = [t.clone() for t in (s.table, s.held, s.free, s.count, s.kc, s.vc)]
    s.lens[2:] = 32 + 64
    cu = torch.tensor([0, 0, 0, 64, 128], dtype=torch.int32, device="cuda")
    s.step(s.draw(128), cu)
    assert attn.cache_device_status() == (1, 25)
    assert all(torch.equal(a, b) for a, b in zip(before, (s.table, s.held, s.free, s.count, s.kc, s.vc)))
