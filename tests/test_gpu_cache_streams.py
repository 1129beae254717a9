"""The calls around the paged cache on a stream of the caller's, by object and by handle (needs a GB300): they run in that
stream's order, so each sees what the stream did before, and nothing of the current stream's."""
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


def step(attn, state, stream):
    """Append, attend, evict; state is rewritten."""
    x, kc, vc, w, lens, cu, table, pos, freqs, axes = state
    q = attn.attn_paged_append(x[:, 4:6], x[:, 6:], kc, vc, cu, lens, table, q=x[:, :4], positions=pos, freqs=freqs,
                               axes=axes, stream=stream)
    o, lse = attn.attn_paged_decode(q, kc, vc, lens, table, weights=w, return_lse=True, stream=stream)
    n = attn.attn_paged_evict(kc, vc, w, lens, table, 100, sinks=4, recent=16, stream=stream)
    return [q, o, lse, n, kc, vc, w]


def make(attn, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    freqs, axes = attn.rope_freqs((64,))
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    table = torch.as_tensor(np.random.default_rng(seed).permutation(24).reshape(3, 8).astype(np.int32)).cuda()
    return [normal(3, 8, 64), normal(24, 16, 2, 64), normal(24, 16, 2, 64), torch.zeros((3, 2, 128), device="cuda"),
            torch.tensor([101, 128, 60], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda"), table,
            torch.tensor([[100, 127, 59]], dtype=torch.int32, device="cuda"), freqs, axes]


@pytest.mark.parametrize("by", ["object", "handle"])
def test_in_the_stream_s_order(attn, by):
    want = [step(attn, make(attn, s), None) for s in range(4)]
    streams, states = [torch.cuda.Stream() for _ in range(2)], [make(attn, s) for s in range(4)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, state in enumerate(states):
        s = streams[i % 2]
        kept = state[0].clone()
        state[0].zero_()                             # on the current stream ...
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(200000)
            state[0].copy_(kept)                     # ... and the token behind a delay on the call's own
            kept.record_stream(s)
        got.append(step(attn, state, s if by == "object" else s.cuda_stream))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert attn.cache_device_status(streams[0] if by == "object" else streams[0].cuda_stream) == (0, 0)


def test_evict_keeps_a_workspace_of_the_caller_s(attn):
    import ctypes
    want = step(attn, make(attn, 7), None)
    x, kc, vc, w, lens, cu, table, pos, freqs, axes = make(attn, 7)
    a = attn.EvictArgs()
    a.B, a.Hkv, a.num_pages, a.page_size, a.max_pages, a.d, a.budget, a.sinks, a.recent = 3, 2, 24, 16, 8, 64, 100, 4, 16
    ws = torch.full((int(attn.load().attn_paged_evict_workspace_size(ctypes.byref(a))),), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = attn.attn_paged_append(x[:, 4:6], x[:, 6:], kc, vc, cu, lens, table, q=x[:, :4], positions=pos, freqs=freqs,
                               axes=axes, stream=s)
    attn.attn_paged_decode(q, kc, vc, lens, table, weights=w, stream=s)
    attn.attn_paged_evict(kc, vc, w, lens, table, 100, sinks=4, recent=16, stream=s, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want[3:], (lens, kc, vc, w)))
    assert attn.cache_device_status() == (0, 0)
