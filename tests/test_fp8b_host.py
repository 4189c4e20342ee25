"""The block-scaled FP8 cache and the page plan without a GPU: the refusals of
their calls (none of them reaches a CUDA call) and the plain forms that the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import paged_fp8_kv_03_gb300 as pkv
from tests import fp4_ref, fp8b_ref

A = ctypes.c_void_p(0x10000)         # never dereferenced
B = ctypes.c_void_p(0x20000)
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5, 7


def _off(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.fixture(scope="module")
def lib():
    return pkv.load()


def _append(lib, **kw):
    a = dict(k=A, v=A, dt=1, T=4, H=8, D=128, slots=A, kc=A, vc=B, ke=A, ve=B, np_=10, P=16, err=None)
    a.update(kw)
    return lib.pkv_kv_append_fp8b(a["k"], a["v"], a["dt"], a["T"], a["H"], a["D"], a["slots"], a["kc"], a["vc"],
                                  a["ke"], a["ve"], a["np_"], a["P"], a["err"], None)


def _read(lib, **kw):
    a = dict(slots=A, T=4, H=8, D=128, kc=A, vc=B, ke=A, ve=B, np_=10, P=16, k=A, v=A, dt=0, err=None)
    a.update(kw)
    return lib.pkv_kv_read_fp8b(a["slots"], a["T"], a["H"], a["D"], a["kc"], a["vc"], a["ke"], a["ve"], a["np_"],
                                a["P"], a["k"], a["v"], a["dt"], a["err"], None)


def _decode(lib, **kw):
    a = dict(q=A, kc=A, vc=B, ke=A, ve=B, bt=A, maxp=4, lens=A, maxl=0, psz=None, B=2, Hq=16, Hkv=2, D=128, P=16,
             np_=8, sm=0.088, W=0, S=0, out=A, odt=1, ws=A, wsb=1 << 30, err=None, ctas=0)
    a.update(kw)
    return lib.pkv_paged_gqa_decode_fp8b(a["q"], a["kc"], a["vc"], a["ke"], a["ve"], a["bt"], a["maxp"], a["lens"],
                                         a["maxl"], a["psz"], a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], a["np_"],
                                         a["sm"], a["W"], a["S"], a["out"], a["odt"], a["ws"], a["wsb"], a["err"],
                                         a["ctas"], None)


def _prefill(lib, **kw):
    a = dict(q=A, cu=A, T=4, maxq=4, kc=A, vc=B, ke=A, ve=B, bt=A, maxp=4, lens=A, psz=None, B=2, maxkv=64, tot=0,
             Hq=16, Hkv=2, D=128, P=16, np_=8, sm=0.088, W=0, S=0, out=A, odt=1, ws=A, wsb=1 << 30, err=None)
    a.update(kw)
    return lib.pkv_paged_prefill_fp8b(a["q"], a["cu"], a["T"], a["maxq"], a["kc"], a["vc"], a["ke"], a["ve"], a["bt"],
                                      a["maxp"], a["lens"], a["psz"], a["B"], a["maxkv"], a["tot"], a["Hq"], a["Hkv"],
                                      a["D"], a["P"], a["np_"], a["sm"], a["W"], a["S"], a["out"], a["odt"], a["ws"],
                                      a["wsb"], a["err"], None)


def _plan(lib, **kw):
    a = dict(past=A, new=A, B=2, bt=A, maxp=4, P=16, pool=A, np_=8, lens=A, cu=A, slots=A, pos=None, T=4, err=None)
    a.update(kw)
    return lib.pkv_plan_pages(a["past"], a["new"], a["B"], a["bt"], a["maxp"], a["P"], a["pool"], a["np_"], a["lens"],
                              a["cu"], a["slots"], a["pos"], a["T"], a["err"], None)


def _release(lib, **kw):
    a = dict(lens=A, keep=None, B=2, bt=A, maxp=4, P=16, pool=A, np_=8, err=None)
    a.update(kw)
    return lib.pkv_release_pages(a["lens"], a["keep"], a["B"], a["bt"], a["maxp"], a["P"], a["pool"], a["np_"],
                                 a["err"], None)


@pytest.mark.parametrize("call", [_append, _read])
def test_row_calls_refuse(lib, call):
    for bad, status in ((dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(np_=0), SHAPE), (dict(dt=7), DTYPE),
                        (dict(D=64), UNSUPPORTED), (dict(P=8), UNSUPPORTED), (dict(P=48), UNSUPPORTED),
                        (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(ke=None), NULL),
                        (dict(ve=None), NULL), (dict(vc=None), NULL), (dict(k=_off(8)), ALIGN),
                        (dict(kc=_off(8)), ALIGN), (dict(slots=_off(4)), ALIGN), (dict(err=_off(2)), ALIGN)):
        assert call(lib, **bad) == status, bad
    assert call(lib, T=0, k=None, v=None, slots=None) == OK


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_attention_calls_refuse(lib, call):
    for bad, status in ((dict(Hq=12, Hkv=8), SHAPE), (dict(B=-1), SHAPE), (dict(maxp=0), SHAPE), (dict(np_=0), SHAPE),
                        (dict(W=-1), SHAPE), (dict(S=-1), SHAPE), (dict(sm=float("nan")), SHAPE),
                        (dict(sm=float("inf")), SHAPE), (dict(odt=5), DTYPE), (dict(Hq=18, Hkv=2), UNSUPPORTED),
                        (dict(D=64), UNSUPPORTED), (dict(P=512), UNSUPPORTED), (dict(B=8193), UNSUPPORTED),
                        (dict(np_=1 << 28, P=256), UNSUPPORTED), (dict(psz=A, maxp=1 << 24), UNSUPPORTED),
                        (dict(q=None), NULL), (dict(ke=None), NULL), (dict(ve=None), NULL), (dict(bt=None), NULL),
                        (dict(lens=None), NULL), (dict(out=None), NULL), (dict(q=_off(8)), ALIGN),
                        (dict(out=_off(8)), ALIGN), (dict(bt=_off(2)), ALIGN), (dict(psz=_off(2)), ALIGN),
                        (dict(ws=None), WORKSPACE), (dict(ws=_off(16)), WORKSPACE)):
        assert call(lib, **bad) == status, bad
    assert call(lib, B=0, q=None, bt=None, lens=None, out=None) == OK


def test_more_refusals(lib):
    assert _decode(lib, maxl=-1) == SHAPE
    assert _decode(lib, ctas=-1) == SHAPE
    for bad in (dict(T=-1), dict(maxq=-1), dict(maxkv=-1), dict(tot=-1), dict(sm=0.0), dict(sm=-1.0)):
        assert _prefill(lib, **bad) == SHAPE, bad
    assert _prefill(lib, T=0, q=None) == OK
    assert _prefill(lib, wsb=16) == WORKSPACE
    assert _prefill(lib, cu=_off(2)) == ALIGN
    assert _prefill(lib, Hq=8193, Hkv=8193) == UNSUPPORTED
    assert pkv.pkv_decode_fp8b_workspace_size(2, 12, 8) == 0
    assert pkv.pkv_decode_fp8b_workspace_size(2, 16, 8, page_size=8) == 0
    assert pkv.pkv_decode_fp8b_workspace_size(2, 16, 8, max_seq_len=-1) == 0
    for bad in ((-1, 8, 1, 64), (1, 0, 1, 64), (1, 8, -1, 64), (1, 8, 1, -1), (1, 8, 1, 64, -1), (1, 8, 1, 64, 0, -1),
                (1, 8, 1, 64, 0, 0, -1)):
        assert pkv.pkv_prefill_fp8b_workspace_size(*bad) == 0, bad


def test_prefill_workspace_of_few_rows():
    """Room for the states of the CTAs that share a query tile's keys, where there may be such."""
    size = pkv.pkv_prefill_fp8b_workspace_size
    copies = lambda b, h, tiles: 256 * h * ((tiles * 128 * (512 + 16) + tiles * 8) // 256) + 4096 * b  # noqa: E731 (about)
    assert size(1, 8, 64, 1024) - size(1, 8, 64, 896) > 152 * 256 * 528      # 8 key tiles: shared
    assert size(10, 8, 64, 1024) < copies(10, 8, 80) + 100000                # more CTAs than half the SMs
    assert size(1, 8, 64, 32768, 0, 500, 0) < copies(1, 8, 8) + 100000       # a window that hides the past
    assert size(1, 8, 64, 1 << 20, 890) < copies(1, 8, 9) + 100000           # no sequence that long
    # a long context has as many parts as keep each at 128 key tiles
    assert size(9, 8, 64, 1 << 20, 1 << 20) - copies(9, 8, 8192 + 9) > 76 * 64 * 256 * 528 - 100000


def test_plan_calls_refuse(lib):
    for call in (_plan, _release):
        for bad, status in ((dict(B=-1), SHAPE), (dict(maxp=0), SHAPE), (dict(np_=0), SHAPE), (dict(P=8), UNSUPPORTED),
                            (dict(P=24), UNSUPPORTED), (dict(B=8193), UNSUPPORTED), (dict(np_=1 << 31), UNSUPPORTED),
                            (dict(np_=(1 << 30) + 1), UNSUPPORTED),
                            (dict(maxp=1 << 27), UNSUPPORTED), (dict(bt=None), NULL), (dict(pool=None), NULL),
                            (dict(lens=None), NULL), (dict(bt=_off(2)), ALIGN), (dict(pool=_off(2)), ALIGN),
                            (dict(lens=_off(1)), ALIGN), (dict(err=_off(2)), ALIGN)):
            assert call(lib, **bad) == status, bad
    for bad, status in ((dict(T=-1), SHAPE), (dict(past=None), NULL), (dict(new=None), NULL), (dict(cu=None), NULL),
                        (dict(slots=None), NULL), (dict(slots=_off(4)), ALIGN), (dict(pos=_off(2)), ALIGN)):
        assert _plan(lib, **bad) == status, bad
    assert _plan(lib, T=(1 << 30) + 1) == UNSUPPORTED
    assert _release(lib, keep=_off(2)) == ALIGN
    assert _release(lib, B=0, lens=None, bt=None, pool=None) == OK


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0: the checks never read it."""
    is_cuda = True

    def get_device(self):
        return 0


def _fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


def _refused(call, good, cases):
    for name, bad, error in cases:
        with pytest.raises(error):
            call(**{**good, name: bad})


def test_binding_refuses():
    u8, i64, i32, bf = torch.uint8, torch.int64, torch.int32, torch.bfloat16
    z, slots, pool, exps = _fake(3, 2, 128), _fake(3, dtype=i64), _fake(4, 2, 32, 128, dtype=u8), _fake(4, 2, 2, dtype=u8)
    caches = dict(k_cache=pool, v_cache=pool, k_exp=exps, v_exp=exps)
    bad_caches = [("k_cache", _fake(4, 2, 32, 72, dtype=u8), ValueError), ("v_cache", _fake(5, 2, 32, 128, dtype=u8), ValueError),
                  ("k_exp", _fake(4, 2, 1, dtype=u8), ValueError), ("v_exp", _fake(4, 2, 2), TypeError),
                  ("k_exp", torch.zeros(4, 2, 2, dtype=u8), ValueError), ("k_cache", _fake(4, 2, 32, dtype=u8), ValueError)]
    _refused(pkv.kv_append_fp8b, dict(k_new=z, v_new=z, slot_mapping=slots, **caches), bad_caches + [
        ("k_new", torch.zeros(3, 2, 128), ValueError), ("k_new", 3, TypeError), ("v_new", z.to(bf), TypeError),
        ("v_new", _fake(2, 2, 128), ValueError), ("slot_mapping", _fake(3), TypeError),
        ("slot_mapping", _fake(2, dtype=i64), ValueError), ("k_new", _fake(3, 128, 2).transpose(1, 2), ValueError)])
    _refused(pkv.kv_read_fp8b, dict(slot_mapping=slots, k_out=z, v_out=z, **caches), bad_caches + [
        ("k_out", None, ValueError), ("v_out", _fake(3, 3, 128), ValueError), ("k_out", _fake(3, 2, 128, dtype=i32), TypeError)])
    q, bt, lens, ws = _fake(2, 8, 128, dtype=bf), _fake(2, 3, dtype=i32), _fake(2, dtype=i32), _fake(64, dtype=u8)
    attn = dict(q=q, block_table=bt, seq_lens=lens, out=_fake(2, 8, 128), workspace=ws, **caches)
    bad_attn = bad_caches + [("q", _fake(2, 8, 128), TypeError), ("out", _fake(2, 8, 64), ValueError),
                             ("block_table", _fake(3, 3, dtype=i32), ValueError), ("seq_lens", _fake(2), TypeError),
                             ("workspace", _fake(64), TypeError), ("window", -1, ValueError), ("sinks", -1, ValueError),
                             ("seq_page_sizes", _fake(3, dtype=i32), ValueError)]
    _refused(pkv.paged_gqa_decode_fp8b, dict(max_seq_len=64, **attn), bad_attn + [("max_seq_len", 1 << 31, ValueError),
                                                                                  ("max_ctas", 1 << 32, ValueError)])
    _refused(pkv.paged_prefill_fp8b, dict(cu_q=_fake(3, dtype=i32), max_q_len=1, max_kv_len=64, **attn), bad_attn + [
        ("cu_q", _fake(2, dtype=i32), ValueError), ("max_q_len", 1 << 31, ValueError), ("max_kv_len", 1 << 40, ValueError)])
    pages = _fake(12, dtype=i32)
    plan = dict(past_lens=lens, new_lens=lens, block_table=bt, pool=pages, page_size=16, seq_lens=lens,
                cu_q=_fake(3, dtype=i32), slot_mapping=slots, positions=_fake(3, dtype=i32))
    _refused(pkv.plan_pages, plan, [
        ("past_lens", _fake(2), TypeError), ("new_lens", _fake(3, dtype=i32), ValueError),
        ("block_table", _fake(3, 3, dtype=i32), ValueError), ("pool", _fake(4, dtype=i32), ValueError),
        ("pool", _fake(12), TypeError), ("seq_lens", _fake(1, dtype=i32), ValueError),
        ("cu_q", _fake(2, dtype=i32), ValueError), ("slot_mapping", _fake(3, dtype=i32), TypeError),
        ("positions", _fake(2, dtype=i32), ValueError), ("max_tokens", 7, ValueError)])
    with pytest.raises(ValueError):
        pkv.plan_pages(lens, lens, bt, pages, 16)
    _refused(pkv.release_pages, dict(seq_lens=lens, block_table=bt, pool=pages, page_size=16), [
        ("keep_lens", _fake(3, dtype=i32), ValueError), ("pool", _fake(3, dtype=i32), ValueError),
        ("seq_lens", torch.zeros(2, dtype=i32), ValueError)])


def test_page_pool_on_the_host():
    pool = pkv.page_pool(5, "cpu")
    assert pool.tolist() == [5, 0, 0, 0, 0, 1, 2, 3, 4]
    assert pkv.page_pool(5, "cpu", [3, 1]).tolist() == [2, 0, 0, 0, 3, 1, 0, 0, 0]
    with pytest.raises(ValueError):
        pkv.page_pool(1, "cpu", [0, 0])


def test_plain_form_of_the_codes():
    """E4M3 of the plain form: every code's value comes back as that code, the
    middle of two goes to the even one; exponents at both sides of a border."""
    v = fp4_ref.e4m3_values()[:127]
    assert (fp8b_ref.e4m3(v) == np.arange(127)).all()
    mid = (v[:-1] + v[1:]) / 2
    assert (fp8b_ref.e4m3(mid) % 2 == 0).all()
    assert (fp8b_ref.e4m3(-mid) >= 128).all()
    for e in (-117, -3, 0, 5, 118):
        assert fp8b_ref.exponent(448.0 * 2.0 ** e) == e
        assert fp8b_ref.exponent(np.nextafter(448.0 * 2.0 ** e, np.inf)) == e + 1
    assert fp8b_ref.exponent(0.0) == -117 and fp8b_ref.exponent(1e300) == 119


def test_plain_form_of_the_plan():
    """Pages come from the list's end; releasing what a plan took restores it."""
    table = np.full((3, 4), -1, np.int32)
    free = [9, 8, 7, 6, 5, 4]
    lens, cu, slots, pos, err = fp8b_ref.plan([0, 0, 0], [17, 0, 16], table, free, 16, 40, 10)
    assert err == 0 and free == [9, 8, 7] and table[0, :2].tolist() == [4, 5] and table[2, 0] == 6
    assert cu.tolist() == [0, 17, 17, 33] and lens.tolist() == [17, 0, 16]
    assert slots[:18].tolist() == list(range(64, 80)) + [80, 96] and (slots[33:] == -1).all()
    assert fp8b_ref.release(lens, None, table, free, 16, 10) == 0 and free == [9, 8, 7, 6, 5, 4]
    assert fp8b_ref.plan([0, 0, 0], [64, 48, 0], table, free, 16, 112, 10)[4] == 64
    assert fp8b_ref.plan([0, 60, 0], [1, 5, 0], table, free, 16, 112, 10)[4] == 4
