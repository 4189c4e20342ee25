"""fp32 outputs of the 4-bit attention at the accuracy their two f16 parts and
short chains give, and sums beside one large contribution."""
import numpy as np
import pytest
import torch

from tests import fp4_ref, fp4_tight
from tests.fp4_long import LongCache
from tests.test_gpu_fp4_attention import Cache, _check, _dev

pytestmark = pytest.mark.gpu


class PositiveCache(Cache):
    """V of one sign: what truncating additions lose does not average out."""

    def __init__(self, seed, lens, hkv, P, dev):
        super().__init__(seed, lens, hkv, P, dev)
        self.v = [np.abs(v) for v in self.v]
        tiles = self.vc.view(self.pages, hkv, P // 16, 1152)
        tiles[..., :1024] &= 0x77                                # the codes' signs


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
@pytest.mark.parametrize("max_ctas", [0, 1])
def test_decode_fp32(pkv, cuda_device, positive, window, sinks, max_ctas):
    lens = [1, 2, 3, 5, 9, 20, 100, 700, 3000]
    c = (PositiveCache if positive else Cache)(41, lens, 2, 16, cuda_device)
    q, qd = c.queries(len(lens), 8, 0.05)
    got = pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out_dtype=torch.float32,
                                   max_seq_len=3000, window=window, sinks=sinks, max_ctas=max_ctas)
    for b, L in enumerate(lens):
        case = (q[b].astype(np.float64), c.k[b], c.v[b], L - 1, window, sinks, fp4_ref.SM)
        _check(got[b], fp4_ref.attend(*case), fp4_tight.tolerance(*case), (b, L))


@pytest.mark.parametrize("max_ctas", [0, 1, 5])
def test_decode_fp32_long_chain(pkv, cuda_device, max_ctas):
    """20000 tokens, with one CTA in four chains of 5000: folded."""
    c = PositiveCache(42, [20000], 1, 64, cuda_device)
    q, qd = c.queries(1, 8, 0.05)
    got = pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out_dtype=torch.float32,
                                   max_seq_len=20000, max_ctas=max_ctas)
    case = (q[0].astype(np.float64), c.k[0], c.v[0], 19999, 0, 0, fp4_ref.SM)
    _check(got[0], fp4_ref.attend(*case), fp4_tight.tolerance(*case), max_ctas)


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5), (6000, 200)])
def test_prefill_fp32(pkv, cuda_device, positive, window, sinks):
    lens, ns = [5, 100, 9000], [5, 60, 150]
    c = (PositiveCache if positive else Cache)(43, lens, 2, 16, cuda_device)
    q, qd = c.queries(sum(ns), 8, 0.05)
    cu = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    got = pkv.paged_prefill_fp4(qd, _dev(cu, c.dev), c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 150, max_kv_len=9000,
                                out_dtype=torch.float32, window=window, sinks=sinks)
    for b, (L, n) in enumerate(zip(lens, ns)):
        for r in sorted({0, 1, 2, 4, n // 2, n - 1}):
            case = (q[cu[b] + r].astype(np.float64), c.k[b], c.v[b], L - n + r, window, sinks, fp4_ref.SM)
            _check(got[cu[b] + r], fp4_ref.attend(*case), fp4_tight.tolerance(*case), (b, r))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("call", ["prefill", "decode", "decode_one_cta"])
@pytest.mark.parametrize("first", [1.0, -1.0])
@pytest.mark.parametrize("e", [12.0, 14.3, 20.0])
def test_small_contributions_beside_a_large_one(pkv, cuda_device, call, first, e, out_dtype):
    """The first token has almost all the weight and a V of `first`; 128K
    others with V = 1 and 2^-e of its weight are added to it one after the
    other."""
    n, dev = 131072, cuda_device

    def make(t0, t1):
        k, v = torch.zeros(t1 - t0, 1, 128, device=dev), torch.ones(t1 - t0, 1, 128, device=dev)
        if t0 == 0:
            k[0, :, 0] = 6
            v[0] = first
        return k, v

    c = LongCache(pkv, n, 1, dev, make)
    _, k, _ = next(c.pieces())
    q = torch.zeros(1 if call != "prefill" else 2, 4, 128, device=dev, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    S = e * np.log(2)
    sm = float(np.float32(S / float(k[0, 0, 0])))
    p = torch.tensor([n - 2, n - 1], device=dev) if call == "prefill" else None
    ref, size = c.attend(q, sm, p)
    if call == "prefill":
        got = c.prefill(q, sm, out_dtype=out_dtype)
    else:
        got = c.decode(q, sm, out_dtype=out_dtype, max_ctas=1 if call == "decode_one_cta" else 0)
    # scores of one product each: no chain; 4 roundings of factors (2^-24 S), the exponent of the small
    # weights (below 64: 2^-19 of log2 units, so 2^-19 of the weight) and the exponential (2^-22), in
    # numerator and normaliser
    delta = 4 * 2.0 ** -24 * S + 2.0 ** -19 + 2.0 ** -22
    if out_dtype == torch.float32:
        # chains of 64, two parts (2^-21, or 2^-37 of the largest weight a token), folds and joins (2^-20)
        tol = (2.0 ** -17 + 2.0 ** -21 + 2.0 ** -20 + 2 * delta) * size + n * 2.0 ** -37 + 2.0 ** -24 * ref.abs()
    else:
        # chains of 1024, weights rounded to f16 (2^-11, or 2^-27 of the largest one a token), the output's 2^-8
        tol = (2.0 ** -13 + 2.0 ** -11 + 2.0 ** -20 + 2 * delta) * size + n * 2.0 ** -27 + 2.0 ** -8 * ref.abs()
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
