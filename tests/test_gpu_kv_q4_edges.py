"""The 4-bit KV cache entries at the ends of f32. Tolerances as in test_gpu_kv_q4.py,
and as derived beside each test."""
import numpy as np
import pytest

from oracle import qw3_oracle as orc
from test_gpu_kv_q4 import EPS, cu, new_cache, planes, rope_table, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("big,fits", [(524159.96875, True), (524160.0, None), (524160.03125, False)])
def test_append_keys_at_the_largest_scale(torch, big, fits):  # noqa: F811
    """Heads of one value c have norm 1 exactly whatever c: a key value just under
    524160 is held, one above is not, and no scale is ever infinite."""
    hd, M = 128, 512
    rng = np.random.default_rng(1)
    x = np.repeat(rng.uniform(0.5, 2, (M, 3, 1)).astype(np.float32), hd, 2)
    w = np.ones(hd, np.float32)
    w[7] = big
    rope = np.zeros((M, hd // 2, 2), np.float32)
    rope[..., 0] = 1
    cache = new_cache(torch, 1, M, 1, hd)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = cu(torch, np.ones(hd, np.float32))
    cache.append(cu(torch, x.reshape(M, -1)), one, cu(torch, w), 0.0, cu(torch, rope), status=status)
    k = cache.read(n=M)[0].cpu().numpy()[:, 0]
    assert np.isfinite(k).all()
    want = orc.kv_q4_decode(*orc.kv_q4_encode(np.broadcast_to(np.where(np.arange(hd) == 7, 0.0 if fits is False else big, 1.0), (M, hd))))
    if fits is False:
        want[:, :32] = 0                                      # the whole block goes
    assert np.array_equal(k[:, 32:], want[:, 32:])
    if fits is not None:
        assert np.array_equal(k, want) and int(status) == (0 if fits else 5)


def test_append_subnormal_scales(torch):  # noqa: F811
    """Scales among f16's subnormals, and at the border to zero, to nearest even."""
    hd, M = 64, 256
    rng = np.random.default_rng(2)
    x = np.zeros((M, 3, hd), np.float32)
    step = 8 * 2.0 ** -24
    x[:, 2] = rng.uniform(-1, 1, (M, hd)) * step
    x[:, 2, 3] = -(np.arange(M) / 8) * step                  # scales in eighths of the smallest subnormal, halves among them
    x[:, 2, 40] = np.exp(rng.uniform(np.log(1e-8), np.log(1e-4), M)) * 8
    one = cu(torch, np.ones(hd, np.float32))
    cache = new_cache(torch, 1, M, 1, hd)
    cache.append(cu(torch, x.reshape(M, -1)), one, one, EPS, cu(torch, rope_table(M, hd)))
    assert np.array_equal(cache.read(n=M)[1].cpu().numpy()[:, 0], orc.kv_q4_decode(*orc.kv_q4_encode(x[:, 2])))
    assert np.array_equal(planes(cache)[1][0, 1, 0].view(np.uint16) & 0x7fff, orc.kv_q4_encode(x[:, 2])[1].view(np.uint16) & 0x7fff)
