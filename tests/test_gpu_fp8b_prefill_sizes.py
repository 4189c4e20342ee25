"""Prefill over blocks of very different sizes against the 64-bit form, as near as the
outputs' own terms (sum w |v|) and the documented absolute losses allow: an error of the
size of the largest value would hide what becomes of the small ones."""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.test_gpu_fp8b_attention import SIZES, SM, Cache, _check, _dev, _tight

pytestmark = pytest.mark.gpu


def _unit(c, b, n, g, window, sinks):
    """What V's widening may be off by, [Hq, 1]: in units of 2^(E - 6), E the exponent of the
    largest block that some query of the chunk sees, a value is rounded to f16, by at
    most 2^-25 where it is below 2^-14, and not at all above.  The weights' sum is 1."""
    L = c.lens[b]
    t = np.arange(L)
    seen = (t > L - n - window) | (t < sinks) if window else t >= 0
    # (a block that has one seen token counts; the exponents of its tokens are the same)
    blocks = np.zeros((L + 15) // 16, bool)
    np.logical_or.at(blocks, t // 16, seen)
    return np.repeat(2.0 ** -31 * c.scale[b][blocks[t // 16]].max(0), g)[:, None]


def _bf16(q, k, v, p, window, sinks, sm):
    """A bf16 output's tolerance, without V's widening.

    With A = sum w |v|: the weights' one rounding to f16, 2^-11 A; f16's lower end, where 2^-25 is
    lost of weights whose largest one is at least 2^2, so 2^-27 of it for each key; the tensor cores'
    truncating additions, eight a key tile, in one chain of at most 128 tiles, 2^-23 each; the
    normaliser's sums (40 in a tile and one a tile, 2^-24 each); what fp4_tight counts for scores,
    exponentials and factors; parts of the keys as the fp32 form's; and half a step of the output, 2^-8.
    """
    g = q.shape[0] // k.shape[1]
    t = fp4_ref.visible(p, window, sinks)
    s = np.einsum("hd,thd->ht", q, np.repeat(k[t], g, 1)) * sm
    w = np.exp(s - s.max(1, keepdims=True))
    total = w.sum(1)[:, None]
    A = np.einsum("ht,thd->hd", w, np.abs(np.repeat(v[t], g, 1))) / total
    tiles = min(128, p // 128 + 1)
    rel = 2.0 ** -11 + 8 * tiles * 2.0 ** -23 + (40 + tiles) * 2.0 ** -24
    lost = 2.0 ** -27 / total * np.repeat(np.abs(v[t]).sum(0), g, 0)
    ref = np.abs(fp4_ref.attend(q, k, v, p, window, sinks, sm))
    return rel * A + lost + _tight(q, k, v, p, window, sinks, sm) + 2.0 ** -8 * ref


def _run(pkv, c, ns, hq, out_dtype, window=0, sinks=0, bound=0, sm=SM, sample=12):
    cu = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    q, qd = c.queries(int(cu[-1]), hq, 2.0)
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    out = pkv.paged_prefill_fp8b(qd, _dev(cu, c.dev), *c.args, c.tabled, c.lensd, max(ns), out_dtype=out_dtype,
                                 max_kv_len=max(*c.lens, bound), sm_scale=sm, device_error=e, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    bf16 = out_dtype == torch.bfloat16
    for b, (L, n) in enumerate(zip(c.lens, ns)):
        unit = _unit(c, b, n, hq // c.hkv, window, sinks)
        for r in sorted({0, 1, n - 2, n - 1, *c.rng.integers(0, n, sample).tolist()} & set(range(n))):
            x, p = q[cu[b] + r].astype(np.float64), L - n + int(r)
            ref = fp4_ref.attend(x, c.k[b], c.v[b], p, window, sinks, sm)
            tol = (_bf16 if bf16 else _tight)(x, c.k[b], c.v[b], p, window, sinks, sm) + unit
            _check(out[cu[b] + r], ref, tol, (L, n, r, window, sinks))


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("sizes", list(SIZES))
def test_a_cta_a_query_tile(pkv, cuda_device, sizes, out_dtype):
    c = Cache(41, [40, 333, 900], 2, 16, cuda_device, sizes=SIZES[sizes])
    _run(pkv, c, [40, 33, 20], 8, out_dtype)
    _run(pkv, c, [40, 33, 20], 8, out_dtype, 90, 5)              # (not in sight: the one large token)


@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("bound", [0, 200000])                  # bf16: over copies, from the cache itself
def test_keys_shared_among_ctas(pkv, cuda_device, sizes, bound, out_dtype):
    c = Cache(42, [1300, 2100], 2, 16, cuda_device, sizes=SIZES[sizes])
    _run(pkv, c, [33, 20], 8, out_dtype, bound=bound, sample=6)
    _run(pkv, c, [33, 20], 8, out_dtype, 1100, 5, bound=bound, sample=6)


@pytest.mark.parametrize("up", [-20, 3, 13, 15, 100])
@pytest.mark.parametrize("out_dtype", DTYPES)
@pytest.mark.parametrize("bound", [0, 200000])
def test_keys_of_any_size(pkv, cuda_device, up, bound, out_dtype):
    """K's exponents 2^up higher, the softmax's scale as much lower; V of mixed sizes."""
    c = Cache(43, [1300, 700], 2, 16, cuda_device, sizes=SIZES["mixed"])
    c.exps[0] = np.where(c.exps[0] == 255, 255, c.exps[0].astype(np.int64) + up).astype(np.uint8)
    c.args[2].copy_(torch.from_numpy(c.exps[0]))
    c.k = [k * 2.0 ** up for k in c.k]
    _run(pkv, c, [33, 20], 8, out_dtype, bound=bound, sm=SM * 2.0 ** -up, sample=6)
