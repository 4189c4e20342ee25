"""Blocks whose scale rounds to 0, at every size of the head's scale: their
codes are 0 too."""
import numpy as np
import pytest
import torch

from tests import fp4_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -61, 2.0 ** -60, 3.7e-5, 2.0 ** 60, 2.0 ** 61, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [16, 20000])
def test_codes_are_zero_where_the_scale_is(pkv, cuda_device, scale, dtype, tokens):
    """amax / (6 k) from 0 to 2^-9, around the border of 2^-10 where the scale
    becomes 0; zeros, negative zeros and negative values among the others."""
    rng = np.random.default_rng(17)
    x = rng.standard_normal((tokens, 1, 8, 16)).astype(np.float32)
    x /= np.abs(x).max(-1, keepdims=True)
    ratio = rng.choice([0.0, 1e-12, 1e-5, 0.999 * 2.0 ** -10, 2.0 ** -10, 1.01 * 2.0 ** -10, 2.0 ** -9],
                       (tokens, 1, 8, 1))
    x = (x.astype(np.float64) * ratio * 6 * scale).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, :, :, ::2] = 0.0
    x = x.reshape(tokens, 1, 128)
    if dtype == "bf16":
        x = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(x))
    k = np.array([scale], np.float32)
    slots = np.arange(tokens, dtype=np.int64)
    pools = [torch.full((tokens // 16, 1, 16, 72), 0xAB, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    xt, st, kt = (torch.from_numpy(a).to(cuda_device) for a in (x, slots, k))
    xt = xt.to(torch.bfloat16) if dtype == "bf16" else xt
    pkv.kv_append_fp4(xt, -xt, st, kt, kt, *pools)
    for pool, y in zip(pools, (x, -x)):
        codes, scales = fp4_ref.quantise(y, k)
        assert (scales == 0).any() and (scales != 0).any()
        exp = np.full((tokens // 16, 1, 16, 72), 0xAB, np.uint8)
        fp4_ref.write(exp, codes, scales, slots)
        assert np.array_equal(pool.cpu().numpy(), exp)
