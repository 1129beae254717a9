"""attn_rope in place on slices of one buffer that lie side by side in other extents than the heads of a token
(needs a GB300): the same bits as on contiguous copies, and nothing else in the buffer changes."""
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["heads_of_bhsd", "longer_buffer", "token_ranges", "every_other_head"])
def test_in_place(attn, form, d):
    B, S, H, Hkv = 3, 21, 4, 2
    g = torch.Generator().manual_seed(d)
    layout = "bhsd" if form == "heads_of_bhsd" else "bshd"
    shape = {"heads_of_bhsd": (B, H + 2 * Hkv, S, d), "longer_buffer": (B, 40, H + 2 * Hkv, d),
             "token_ranges": (B, 2 * S + 1, H, d), "every_other_head": (B, S, 2 * H, d)}[form]
    x = torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
    q, k = {"heads_of_bhsd": (x[:, :H], x[:, H:H + Hkv]),
            "longer_buffer": (x[:, :S, :H], x[:, :S, H:H + Hkv]),
            "token_ranges": (x[:, :S], x[:, S:2 * S]),
            "every_other_head": (x[:, :, ::2], x[:, :, 1::2])}[form]
    freqs, axes = attn.rope_freqs((d // 2,))
    positions = torch.arange(5, 5 + S, dtype=torch.int32, device="cuda")[None]
    want = x.clone()
    rotated = attn.attn_rope(q.contiguous(), k.contiguous(), positions, freqs, axes, layout=layout)
    wq, wk = {"heads_of_bhsd": (want[:, :H], want[:, H:H + Hkv]),
              "longer_buffer": (want[:, :S, :H], want[:, :S, H:H + Hkv]),
              "token_ranges": (want[:, :S], want[:, S:2 * S]),
              "every_other_head": (want[:, :, ::2], want[:, :, 1::2])}[form]
    wq.copy_(rotated[0])
    wk.copy_(rotated[1])
    qo, ko = attn.attn_rope(q, k, positions, freqs, axes, layout=layout, q_out=q, k_out=k)
    assert qo is q and ko is k and torch.equal(x.view(torch.int16), want.view(torch.int16))
    assert attn.cache_device_status() == (0, 0)
