"""A NaN code of K takes the whole row of every query that sees it, wherever the
tokens beside it went: also where all that a warp, a piece or a part of the keys
sees is NaN, so that its largest score is still -inf."""
import numpy as np
import pytest
import torch

from tests import fp4_ref
from tests.test_gpu_fp8b_attention import SM, Cache, _check

pytestmark = pytest.mark.gpu


def _poison(c, b, tokens, head):
    slot = fp4_ref.slots_of(c.table[b], c.lens[b], c.P)
    for t in tokens:
        page, row = divmod(int(slot[t]), c.P)
        c.args[0][page, head, row, (7 * t) % 128] = 0x7F if t % 2 else 0xFF


def _decode_check(pkv, c, b, tokens, G, max_ctas, out_dtype, window=0, sinks=0):
    """Sequence b's rows of kv head 0 are NaN, all others the bits they were."""
    _, qd = c.queries(len(c.lens), G * c.hkv)
    kw = dict(max_seq_len=max(c.lens), max_ctas=max_ctas, out_dtype=out_dtype, window=window, sinks=sinks)
    base = pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled, c.lensd, **kw)
    _poison(c, b, tokens, 0)
    got = pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled, c.lensd, **kw)
    assert not torch.isnan(base).any()
    assert torch.isnan(got[b, :G]).all(), (b, tokens)
    rest = torch.ones(got.shape[:2], dtype=torch.bool)
    rest[b, :G] = False
    assert torch.equal(got[rest], base[rest])


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_ctas", [0, 2])
@pytest.mark.parametrize("L", [1, 2, 16, 17, 33, 65, 129, 1000, 2049, 8193])
def test_decode_newest_token(pkv, cuda_device, L, max_ctas, out_dtype):
    c = Cache(L, [L, 40], 2, 16, cuda_device)
    _decode_check(pkv, c, 0, [L - 1], 4, max_ctas, out_dtype)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_ctas", [0, 2, 40])
@pytest.mark.parametrize("L,first,last", [(96, 0, 32), (96, 32, 64), (700, 64, 96), (700, 352, 544), (5000, 2048, 2560),
                                          (5000, 0, 4992)])
def test_decode_whole_units(pkv, cuda_device, L, first, last, max_ctas, out_dtype):
    """Tokens first .. last - 1: all of a warp's, or of a CTA's."""
    c = Cache(L + first, [33, L], 1, 16, cuda_device)
    _decode_check(pkv, c, 1, range(first, last), 8, max_ctas, out_dtype)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_ctas", [0, 2])
@pytest.mark.parametrize("L,window,sinks,token", [(97, 34, 0, 96), (97, 1, 0, 96), (97, 1, 1, 0), (400, 129, 3, 399),
                                                  (400, 17, 0, 383), (2000, 1003, 1, 0), (2000, 1003, 1, 997)])
def test_decode_one_token_of_a_unit_in_the_window(pkv, cuda_device, L, window, sinks, token, max_ctas, out_dtype):
    c = Cache(L + window, [L, 5], 1, 16, cuda_device)
    _decode_check(pkv, c, 0, [token], 4, max_ctas, out_dtype, window, sinks)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,n,window,sinks,bound", [(1, 1, 0, 0, 0), (129, 1, 0, 0, 0), (129, 40, 0, 0, 0), (300, 9, 20, 1, 0),
                                                    (1025, 3, 0, 0, 0), (1025, 3, 0, 0, 200000), (3000, 20, 1200, 1, 0)])
def test_prefill_newest_token(pkv, cuda_device, L, n, window, sinks, bound, out_dtype):
    """Of a chunk the last row alone sees the newest token."""
    c = Cache(L + n, [L], 2, 16, cuda_device)
    q, qd = c.queries(n, 8)
    cu = torch.tensor([0, n], dtype=torch.int32, device=cuda_device)

    _poison(c, 0, [L - 1], 0)
    got = pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, n, max_kv_len=max(L, bound), out_dtype=out_dtype,
                                 window=window, sinks=sinks)
    assert torch.isnan(got[n - 1, :4]).all()
    for r in range(n):
        x, p = q[r].astype(np.float64), L - n + r
        ref = fp4_ref.attend(x, c.k[0], c.v[0], p, window, sinks, SM)
        tol = fp4_ref.attention_tolerance(x, c.k[0][:p + 1], c.v[0][:p + 1], ref, SM, out_dtype == torch.bfloat16)
        h = 4 if r == n - 1 else 0
        _check(got[r, h:], ref[h:], tol[h:], ("beside the NaN", r))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,first,last,bound", [(300, 128, 256, 0), (1500, 0, 256, 0), (1500, 1024, 1280, 0), (1500, 1024, 1280, 200000)])
def test_prefill_whole_key_tiles(pkv, cuda_device, L, first, last, bound, out_dtype):
    """All keys of a tile, or of a part that CTAs share."""
    c = Cache(L + first, [L], 1, 16, cuda_device)
    _, qd = c.queries(4, 4)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=cuda_device)
    _poison(c, 0, range(first, last), 0)
    got = pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, 4, max_kv_len=max(L, bound), out_dtype=out_dtype)
    assert torch.isnan(got).all()
