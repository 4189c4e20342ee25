"""Failure detection of the block-scaled calls without a fault: a worker or a CTA
is told (test facility) never to make its first load, its bounded wait runs out,
the call reports PKV_DEVERR_TIMEOUT, and the next call is exact."""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.test_gpu_fp4_timeout import _withheld
from tests.test_gpu_fp8b_attention import SM, Cache, _check, _decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_ctas", [0, 4])                     # clusters, the list
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode_times_out_and_recovers(pkv, cuda_device, max_ctas, out_dtype):
    c = Cache(41, [300, 77, 0], 2, 16, cuda_device)
    q, qd = c.queries(3, 8)

    def call():
        e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled, c.lensd, out_dtype=out_dtype, max_seq_len=300, device_error=e,
                                  max_ctas=max_ctas)
        return e

    _withheld(pkv, call)
    _decode(pkv, c, q, qd, out_dtype=out_dtype, max_ctas=max_ctas)


@pytest.mark.parametrize("window,out_dtype,n,bound", [
    (0, torch.float32, 40, 400), (90, torch.bfloat16, 40, 400),
    (0, torch.float32, 40, 1100), (0, torch.bfloat16, 40, 1100),  # CTAs share the keys
    (0, torch.bfloat16, 30, 200000)])                             # and read them from the cache
def test_prefill_times_out_and_recovers(pkv, cuda_device, window, out_dtype, n, bound):
    c = Cache(42, [400], 1, 16, cuda_device)
    q, qd = c.queries(n, 8)
    cu = torch.tensor([0, n], dtype=torch.int32, device=cuda_device)
    e = torch.zeros(1, dtype=torch.int32, device=cuda_device)

    def call(e):
        return pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, n, out_dtype=out_dtype, max_kv_len=bound,
                                      device_error=e, window=window, sinks=2)

    def withheld():
        bad = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        call(bad)
        return bad

    _withheld(pkv, withheld)
    out = call(e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    for r in (0, 17, n - 1):
        ref = fp4_ref.attend(q[r].astype(np.float64), c.k[0], c.v[0], 400 - n + r, window, 2, SM)
        _check(out[r], ref, fp4_ref.attention_tolerance(q[r], c.k[0], c.v[0], ref, SM, out_dtype == torch.bfloat16), r)
