"""Failure detection of the 4-bit calls without a fault: a worker or a CTA is
told (test facility) never to make its first load, its bounded wait runs out,
the call reports PKV_DEVERR_TIMEOUT, and the next call is exact."""
import time

import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.test_gpu_fp4_attention import Cache, _check, _decode

pytestmark = pytest.mark.gpu


def _withheld(pkv, call):
    pkv.pkv_test_withhold_load(0)
    try:
        t0 = time.time()
        err = call()
        torch.cuda.synchronize()
        dt = time.time() - t0
    finally:
        pkv.pkv_test_withhold_load(-1)
    assert int(err.item()) & pkv.DEVERR_TIMEOUT
    assert 1.5 < dt < 20.0


@pytest.mark.parametrize("max_ctas", [0, 4])                     # clusters, the list
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode_times_out_and_recovers(pkv, cuda_device, max_ctas, out_dtype):
    c = Cache(41, [300, 77, 0], 2, 16, cuda_device)
    q, qd = c.queries(3, 8)

    def call():
        e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out_dtype=out_dtype, max_seq_len=300,
                                 device_error=e, max_ctas=max_ctas)
        return e

    _withheld(pkv, call)
    _decode(pkv, c, q, qd, out_dtype=out_dtype, max_ctas=max_ctas)


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_times_out_and_recovers(pkv, cuda_device, window, out_dtype):
    c = Cache(42, [400], 1, 16, cuda_device)
    q, qd = c.queries(40, 8)
    cu = torch.tensor([0, 40], dtype=torch.int32, device=cuda_device)

    def call(e):
        return pkv.paged_prefill_fp4(qd, cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 40, out_dtype=out_dtype,
                                     max_kv_len=400, device_error=e, window=window, sinks=2)

    def withheld():
        e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        call(e)
        return e

    _withheld(pkv, withheld)
    e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = call(e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    for r in (0, 17, 39):
        ref = fp4_ref.attend(q[r].astype(np.float64), c.k[0], c.v[0], 360 + r, window, 2, fp4_ref.SM)
        _check(out[r], ref, fp4_ref.attention_tolerance(q[r], c.k[0], c.v[0], ref, fp4_ref.SM,
                                                        out_dtype == torch.bfloat16), r)
