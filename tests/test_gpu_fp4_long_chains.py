"""Outputs over hundreds of thousands of tokens: neither the accumulation nor
the smallest weights may lose more as contexts grow."""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.fp4_long import LongCache
from tests.test_gpu_fp4_attention import Cache, _prefill, test_prefill_nan_rows as _nan_rows
from tests.test_gpu_fp4_timeout import _withheld

pytestmark = pytest.mark.gpu

L = 1 << 19


def _positive(pkv, dev, heavy):
    """V of one sign, every row and dim its own; all scores equal, or those of
    128 tokens 13 (log2 units) above the others': the first ones, or some after
    two thirds of the context."""
    g = torch.Generator(device=dev).manual_seed(5)
    at = {"none": -1, "first": 0, "late": 5 * 65536 + 1000}[heavy]

    def make(t0, t1):
        k = torch.zeros(t1 - t0, 8, 128, device=dev)
        if t0 <= at < t1:
            k[at - t0:at - t0 + 128, :, 0] = 6
        return k, torch.rand(t1 - t0, 8, 128, device=dev, generator=g) + 0.5

    c = LongCache(pkv, L, 8, dev, make, v_scale=torch.linspace(2.0 ** -6, 2.0 ** -5, 8, device=dev))
    q = torch.zeros(2, 16, 128, device=dev, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    return c, q, 13 * np.log(2) / 6 if at >= 0 else fp4_ref.SM       # (6 is held as it is)


@pytest.mark.parametrize("heavy", ["none", "first", "late"])
@pytest.mark.parametrize("call", ["prefill", "decode", "decode_one_cta"])
def test_bf16_output_of_one_sign_is_not_biased(pkv, cuda_device, call, heavy):
    """Truncating additions pull a sum of one sign towards zero.

    The weights are 2^2 (or more, by powers of two) and 2^-13 of that here, so
    powers of two that f16 holds; what is left are chains of at most 1024
    additions, each off by less than 2^-23 of the sum (2^-13 in all), and the
    output's rounding.  That is without a bias over 1024 different values (8
    heads x 128 dims): uniform within half a step of 2^-8 to 2^-7 of the
    value, so with a standard deviation below 2^-8 / sqrt(3) = 2.3e-3 each
    and 7.1e-5 for the mean of 1024; four of these.  One value alone may be off
    by its rounding and the chain's 2^-13.
    """
    c, q, sm = _positive(pkv, cuda_device, heavy)
    if call == "prefill":
        got, ref = c.prefill(q, sm), c.attend(q, sm, torch.tensor([L - 2, L - 1], device=cuda_device))[0]
    else:
        q = q[:1]
        got, ref = c.decode(q, sm, max_ctas=1 if call == "decode_one_cta" else 0), c.attend(q, sm)[0]
    rel = (got.double() - ref) / ref
    bias = float(rel.mean())
    assert abs(bias) <= 2.0 ** -13 + 4 * 7.1e-5, bias
    assert float(rel.abs().max()) <= 2.0 ** -8 + 2.0 ** -12


@pytest.mark.parametrize("G", [3, 8])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20000, 300), (16000, 1)])
def test_prefill_over_several_chains(pkv, cuda_device, G, window, sinks):
    """Contexts around one, two and more accumulation chains (16384 keys),
    chunks that end inside a query tile, rows behind the last one."""
    lens, ns = [40000, 16384, 16500, 33000, 60], [45, 20, 130, 1, 60]
    c = Cache(51 + G, lens, 1, 16, cuda_device)
    _prefill(pkv, c, ns, G, window, sinks, out_dtype=torch.bfloat16, sample=6)
    _prefill(pkv, c, ns, G, window, sinks, out_dtype=torch.bfloat16, q_spread=20.0, sample=3)


def test_prefill_over_several_chains_in_place(pkv, cuda_device):
    """The output over the queries, captured twice: the bits of a plain call."""
    c = Cache(57, [40000], 2, 64, cuda_device)
    _, qd = c.queries(33, 8)
    cu = torch.tensor([0, 33], dtype=torch.int32, device=cuda_device)
    args = (cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 33)
    ref = pkv.paged_prefill_fp4(qd, *args, max_kv_len=40000)
    assert torch.equal(pkv.paged_prefill_fp4(qd, *args, max_kv_len=40000), ref)
    out = qd.clone()
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(pkv.pkv_prefill_fp4_workspace_size(1, 2, 33, 40000), dtype=torch.uint8, device=cuda_device)
    with torch.cuda.graph(g):
        pkv.paged_prefill_fp4(out, *args, out=out, max_kv_len=40000, workspace=ws)
    for _ in range(2):
        out.copy_(qd)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.parametrize("lens,ns", [([20000], [300]), ([33000, 500], [200, 3])])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_prefill_nan_rows_over_several_chains(pkv, cuda_device, lens, ns, out_dtype):
    _nan_rows(pkv, cuda_device, out_dtype, lens, ns)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_prefill_bound_of_a_long_context(pkv, cuda_device, out_dtype):
    """The kernel of long contexts on short ones: the bits of the other one."""
    lens, ns = [400, 1, 300], [40, 1, 170]
    c = Cache(58, lens, 1, 16, cuda_device)
    _, qd = c.queries(sum(ns), 7)
    cu = torch.tensor([0, 40, 41, 211], dtype=torch.int32, device=cuda_device)

    def call(bound, window):
        e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        out = pkv.paged_prefill_fp4(qd, cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 170, max_kv_len=bound,
                                    out_dtype=out_dtype, device_error=e, window=window, sinks=2)
        return out, e

    for window in (0, 39000):
        ref, e = call(400, 0)
        assert int(e.item()) == 0
        got, e = call(40000, window)
        assert int(e.item()) == 0
        assert torch.equal(got, ref)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [0, 39000])
def test_prefill_of_a_long_context_times_out_and_recovers(pkv, cuda_device, window, out_dtype):
    c = Cache(59, [20000], 1, 64, cuda_device)
    _, qd = c.queries(40, 8)
    cu = torch.tensor([0, 40], dtype=torch.int32, device=cuda_device)

    def call(e):
        return pkv.paged_prefill_fp4(qd, cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 40, max_kv_len=40000,
                                     out_dtype=out_dtype, device_error=e, window=window, sinks=2)

    def withheld():
        e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        call(e)
        return e

    ref = call(None)
    _withheld(pkv, withheld)
    e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    assert torch.equal(call(e), ref)
    assert int(e.item()) == 0


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("call", ["prefill", "decode", "decode_one_cta"])
@pytest.mark.parametrize("units", [8.5, 2.5])
def test_many_small_weights_of_a_long_context(pkv, cuda_device, call, out_dtype, units):
    """One token takes most of the weight, a million others 2^-e of it each:
    in f16 with the largest weight at 4 they would be 8.5 (2.5) steps of 2^-24,
    half a step from the next one."""
    n, dev = 1 << 20, cuda_device

    def make(t0, t1):
        k, v = torch.zeros(t1 - t0, 1, 128, device=dev), torch.ones(t1 - t0, 1, 128, device=dev)
        if t0 == 0:
            k[0, :, 0] = 6
            v[0] = 0
        return k, v

    c = LongCache(pkv, n, 1, dev, make)
    _, k, _ = next(c.pieces())
    q = torch.zeros(2, 4, 128, device=dev, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    e = 26 - np.log2(units)
    sm = float(np.float32(e * np.log(2) / float(k[0, 0, 0])))
    if call == "prefill":
        ref, _ = c.attend(q, sm, torch.tensor([n - 2, n - 1], device=dev))
        got = c.prefill(q, sm, out_dtype=out_dtype)
    else:
        q = q[:1]
        ref, _ = c.attend(q, sm)
        got = c.decode(q, sm, out_dtype=out_dtype, max_ctas=1 if call == "decode_one_cta" else 0)
    # the tolerance of the other tests, with |v| <= 1 and the largest score of e ln 2
    tol = fp4_ref.attention_tolerance(q[0].double().cpu().numpy(), k[:1].cpu().numpy(), np.ones((1, 1, 128)),
                                      ref[0].cpu().numpy(), sm, out_dtype == torch.bfloat16)
    off = (got.double() - ref).abs().cpu().numpy()
    assert (off <= tol).all(), (off.max(), tol.min())
