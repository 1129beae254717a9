"""Behind a shared prefix with groups of 9 and more query heads a K/V head, which the decoding kernel takes in blocks of 16 and 32: small
and large batches, whichever kernels they go to, against plain fp64 attention (needs a GB300; tolerances of test_gpu_prefix_decode.py)."""
import pytest

from tests.test_gpu_prefix_decode import Batch, attn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,G,Hkv,page,prefix,own", [
    (4, 16, 8, 16, 700, 30), (4, 16, 8, 16, 4800, 30), (4, 16, 8, 16, 5400, 30), (3, 9, 2, 7, 300, 9),
    (2, 32, 8, 16, 3300, 40), (2, 32, 8, 16, 4200, 40), (16, 32, 8, 16, 600, 40), (16, 32, 8, 24, 1500, 40),
    (2, 71, 1, 64, 8000, 70), (2, 71, 1, 64, 13000, 70), (40, 24, 1, 16, 130, 5), (200, 33, 1, 16, 130, 5),
])
def test_against_plain_attention(attn, d, B, G, Hkv, page, prefix, own):  # noqa: F811
    x = Batch([(own * (b % 3)) // 2 for b in range(B)], G * Hkv, Hkv, d, page, prefix, seed=B + G, scale=2.0)
    got = x.call(attn)
    assert attn.cache_device_status() == (0, 0)
    x.check(got, rows=sorted({0, 1, B // 2, B - 1}))
    again = x.call(attn)
    assert all((a == b).all() for a, b in zip(got, again))
