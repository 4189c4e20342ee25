"""Products of a softmax scale and a head's scale below the smallest fp32
number: all visible tokens weigh the same."""
import numpy as np
import pytest
import torch

from tests import fp4_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("call", ["prefill", "decode", "fp8_prefill"])
def test_scores_that_are_all_zero(pkv, cuda_device, call, out_dtype):
    dev, L, n, H = cuda_device, 300, 140, 2
    g = torch.Generator(device=dev).manual_seed(3)
    k, v = (torch.randn(L, H, 128, device=dev, generator=g) for _ in range(2))
    q = torch.randn(n, 4, 128, device=dev, generator=g).bfloat16()
    ks, vs = torch.full((H,), 2.0 ** -100, device=dev), torch.full((H,), 0.01, device=dev)
    slots = torch.arange(L, device=dev)
    bt, lens = torch.arange(19, device=dev, dtype=torch.int32)[None], torch.tensor([L], device=dev, dtype=torch.int32)
    cu = torch.tensor([0, n], device=dev, dtype=torch.int32)
    sm = 2.0 ** -60
    k = k * 2.0 ** -100
    if call == "fp8_prefill":
        kc, vc = (torch.zeros(19, H, 16, 128, dtype=torch.uint8, device=dev) for _ in range(2))
        pkv.kv_append_fp8(k, v, slots, ks, vs, kc, vc)
        val = vc.view(torch.float8_e4m3fn).float().permute(0, 2, 1, 3).reshape(-1, H, 128)[:L]
        val = val.double() * vs.double()[:, None]
    else:
        kc, vc = (pkv.fp4_cache(19, H, 16, dev) for _ in range(2))
        pkv.kv_append_fp4(k, v, slots, ks, vs, kc, vc)
        val = pkv.kv_read_fp4(slots, ks, vs, kc, vc, out_dtype=torch.float32)[1].double()
    val = val.cpu().numpy()
    for window, sinks in ((0, 0), (50, 3)) if call != "fp8_prefill" else ((0, 0),):
        if call == "decode":
            got = pkv.paged_gqa_decode_fp4(q[:1], kc, vc, ks, vs, bt, lens, out_dtype=out_dtype, sm_scale=sm,
                                           window=window, sinks=sinks)
            positions = [L - 1]
        elif call == "prefill":
            got = pkv.paged_prefill_fp4(q, cu, kc, vc, ks, vs, bt, lens, n, out_dtype=out_dtype, sm_scale=sm,
                                        window=window, sinks=sinks)
            positions = range(L - n, L)
        else:
            got = pkv.paged_prefill(q, cu, kc, vc, ks, vs, bt, lens, n, out_dtype=out_dtype, sm_scale=sm)
            positions = range(L - n, L)
        for i, p in enumerate(positions):
            seen = val[fp4_ref.visible(p, window, sinks)]
            ref, size = np.repeat(seen.mean(0), 2, 0), np.repeat(np.abs(seen).mean(0), 2, 0)
            # equal weights: the chains' 2^-15 of sum w |v| and the output's rounding
            tol = 2.0 ** -15 * size + (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(ref)
            off = np.abs(got[i].double().cpu().numpy() - ref)
            assert (off <= tol).all(), (call, window, p, off.max())
