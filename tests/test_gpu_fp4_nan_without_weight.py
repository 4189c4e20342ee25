"""A NaN in a visible block of V is NaN in its 16 dims of the output however
small its token's weight is, and wherever the work is cut."""
import numpy as np
import pytest
import torch

from tests import fp4_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_ctas", [0, 1, 9])
@pytest.mark.parametrize("L", [70, 700, 4000, 9000])
def test_decode(pkv, cuda_device, L, max_ctas, out_dtype):
    """The last token has all the weight, by 2^2000; tokens with NaN blocks lie
    at the beginning, in the middle and beside it."""
    dev, H = cuda_device, 2
    pages = (L + 15) // 16
    s = torch.full((H,), 2.0 ** -6, device=dev)
    k = torch.zeros(L, H, 128, device=dev)
    v = torch.randn(L, H, 128, device=dev, generator=torch.Generator(device=dev).manual_seed(1))
    k[-1, :, 0] = 6
    spots = [(0, 0, 0), (L // 2, 1, 3), (L // 3, 0, 7), (L - 2, 1, 5)]
    for t, h, block in spots:
        v[t, h, 16 * block + 4] = float("nan")
    kc, vc = (pkv.fp4_cache(pages, H, 16, dev) for _ in range(2))
    pkv.kv_append_fp4(k, v, torch.arange(L, device=dev), s, s, kc, vc)
    q = torch.zeros(1, 8, 128, device=dev, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    args = (kc, vc, s, s, torch.arange(pages, device=dev, dtype=torch.int32)[None],
            torch.tensor([L], device=dev, dtype=torch.int32))
    sm = 2000 * np.log(2) / 6
    for window, sinks in ((0, 0), (L // 2 + 1, 1), (2, 0), (1, 0)):
        got = pkv.paged_gqa_decode_fp4(q, *args, sm_scale=sm, max_ctas=max_ctas, max_seq_len=L, out_dtype=out_dtype,
                                       window=window, sinks=sinks)
        exp = torch.zeros(1, 8, 128, dtype=torch.bool, device=dev)
        seen = set(fp4_ref.visible(L - 1, window, sinks).tolist())
        for t, h, block in spots:
            if t in seen:
                exp[:, 4 * h:4 * h + 4, 16 * block:16 * block + 16] = True
        assert torch.equal(got.isnan(), exp), (window, sinks)
