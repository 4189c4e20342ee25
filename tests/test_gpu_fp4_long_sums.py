"""fp32 outputs over many tokens of like weights: a sum of like terms is rounded
the same way at every step, so it must not drift with the context's length."""
import numpy as np
import pytest
import torch

from tests import fp4_ref, fp4_tight
from tests.fp4_long import LongCache
from tests.test_gpu_fp4_attention import Cache, _check, _dev

pytestmark = pytest.mark.gpu

_caches = {}


def _cache(pkv, dev, n, constant):
    """One token with a score, the others with none; V of one sign, its rows
    different or all alike."""
    if (n, constant) not in _caches:
        _caches.clear()
        g = torch.Generator(device=dev).manual_seed(1)

        def make(t0, t1):
            k = torch.zeros(t1 - t0, 1, 128, device=dev)
            if t0 == 0:
                k[0, :, 0] = 6
            v = torch.rand(t1 - t0, 1, 128, device=dev, generator=g) + 0.5
            return k, v * 0 + v[:, :, :1].mean() if constant else v

        _caches[n, constant] = LongCache(pkv, n, 1, dev, make, v_scale=torch.full((1,), 0.013, device=dev))
    return _caches[n, constant]


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("n", [131072, 1 << 20])
@pytest.mark.parametrize("call", ["prefill", "decode", "decode_one_cta"])
def test_fp32_output(pkv, cuda_device, n, constant, call):
    """e: how far (log2 units) the first token's score lies above the others'.

    Against sum w |v| = |out|: chains of 64 truncating additions 2^-17, two f16
    parts 2^-21 and (below the largest weight by 2^16 and more) 2^-37 of the
    largest weight a token, fp32 sums and joins 2^-20, the score's 4 roundings
    of factors (2^-24 S), the exponents' (2^-19 for those under 64) and the
    exponential's (2^-22), in numerator and normaliser.
    """
    c = _cache(pkv, cuda_device, n, constant)
    q = torch.zeros(2 if call == "prefill" else 1, 4, 128, device=cuda_device, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    p = torch.tensor([n - 2, n - 1], device=cuda_device) if call == "prefill" else None
    for e in (0.0, 7.1, 12.3, 14.37, 16.61, 18.77, 20.3):
        S = e * np.log(2)
        sm = float(np.float32(S / 6)) if e else 1e-6
        ref, size = c.attend(q, sm, p)
        if call == "prefill":
            got = c.prefill(q, sm, out_dtype=torch.float32)
        else:
            got = c.decode(q, sm, out_dtype=torch.float32, max_ctas=1 if call == "decode_one_cta" else 0)
        delta = 4 * 2.0 ** -24 * S + 2.0 ** -19 + 2.0 ** -22
        most = 1 / (1 + (n - 1) * 2.0 ** -e) * 0.013 * 448 / 2      # the largest weight times the largest |v|
        tol = (2.0 ** -17 + 2.0 ** -21 + 2.0 ** -20 + 2 * delta) * size + n * 2.0 ** -37 * most
        off = (got.double() - ref).abs()
        assert bool((off <= tol).all()), (e, float((off / size).max()), float((tol / size).min()))


@pytest.mark.parametrize("hkv,G,window,sinks", [(8, 8, 0, 0), (3, 1, 0, 0), (2, 6, 17000, 500)])
def test_prefill_of_many_queries(pkv, cuda_device, hkv, G, window, sinks):
    """Chunks of hundreds of queries at 17 to 40 thousand tokens, so that many CTAs
    run at once, against the bound of the paths' roundings."""
    lens, ns = [40000, 16400, 33000], [600, 300, 450]
    c = Cache(61, lens, hkv, 64, cuda_device)
    q, qd = c.queries(sum(ns), hkv * G, 0.05)
    cu = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    args = (_dev(cu, c.dev), c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, max(ns))
    kw = dict(max_kv_len=max(lens), out_dtype=torch.float32, window=window, sinks=sinks)
    got = pkv.paged_prefill_fp4(qd, *args, **kw)
    for _ in range(3):
        assert torch.equal(pkv.paged_prefill_fp4(qd, *args, **kw), got)
    for b, (L, n) in enumerate(zip(lens, ns)):
        for r in (0, n // 3, n - 1):
            heads = [0, hkv - 1]
            pick = [h * G + g for h in heads for g in range(G)]
            case = (q[cu[b] + r][pick].astype(np.float64), c.k[b][:, heads], c.v[b][:, heads], L - n + r, window, sinks,
                    fp4_ref.SM)
            _check(got[cu[b] + r][pick], fp4_ref.attend(*case), fp4_tight.tolerance(*case), (b, r))
