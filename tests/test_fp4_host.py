"""The 4-bit cache without a GPU: the refusals of its calls (none of them
reaches a CUDA call) and the plain form the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_fp8_kv_03_gb300 as pkv
from tests import fp4_ref

A = ctypes.c_void_p(0x10000)         # never dereferenced
B = ctypes.c_void_p(0x20000)
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5, 7


def _off(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.fixture(scope="module")
def lib():
    return pkv.load()


def _append(lib, **kw):
    a = dict(k=A, v=A, dt=1, T=4, H=8, D=128, slots=A, ks=A, vs=A, kc=A, vc=B, np_=10, P=16, err=None)
    a.update(kw)
    return lib.pkv_kv_append_fp4(a["k"], a["v"], a["dt"], a["T"], a["H"], a["D"], a["slots"], a["ks"], a["vs"],
                                 a["kc"], a["vc"], a["np_"], a["P"], a["err"], None)


def _read(lib, **kw):
    a = dict(slots=A, T=4, H=8, D=128, ks=A, vs=A, kc=A, vc=B, np_=10, P=16, k=A, v=A, dt=0, err=None)
    a.update(kw)
    return lib.pkv_kv_read_fp4(a["slots"], a["T"], a["H"], a["D"], a["ks"], a["vs"], a["kc"], a["vc"], a["np_"],
                               a["P"], a["k"], a["v"], a["dt"], a["err"], None)


def _decode(lib, **kw):
    a = dict(q=A, kc=A, vc=B, ks=A, vs=A, bt=A, maxp=4, lens=A, maxl=0, psz=None, B=2, Hq=16, Hkv=2, D=128, P=16,
             np_=8, sm=0.088, W=0, S=0, out=A, odt=1, ws=A, wsb=1 << 30, err=None, ctas=0)
    a.update(kw)
    return lib.pkv_paged_gqa_decode_fp4(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["maxp"], a["lens"],
                                        a["maxl"], a["psz"], a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], a["np_"],
                                        a["sm"], a["W"], a["S"], a["out"], a["odt"], a["ws"], a["wsb"], a["err"],
                                        a["ctas"], None)


def _prefill(lib, **kw):
    a = dict(q=A, cu=A, T=4, maxq=4, kc=A, vc=B, ks=A, vs=A, bt=A, maxp=4, lens=A, psz=None, B=2, maxkv=64, tot=0,
             Hq=16, Hkv=2, D=128, P=16, np_=8, sm=0.088, W=0, S=0, out=A, odt=1, ws=A, wsb=1 << 30, err=None)
    a.update(kw)
    return lib.pkv_paged_prefill_fp4(a["q"], a["cu"], a["T"], a["maxq"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"],
                                     a["maxp"], a["lens"], a["psz"], a["B"], a["maxkv"], a["tot"], a["Hq"], a["Hkv"],
                                     a["D"], a["P"], a["np_"], a["sm"], a["W"], a["S"], a["out"], a["odt"], a["ws"],
                                     a["wsb"], a["err"], None)


@pytest.mark.parametrize("call", [_append, _read])
def test_row_calls_refuse(lib, call):
    for bad, status in ((dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(np_=0), SHAPE), (dict(dt=7), DTYPE),
                        (dict(D=64), UNSUPPORTED), (dict(P=8), UNSUPPORTED), (dict(P=48), UNSUPPORTED),
                        (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(ks=None), NULL),
                        (dict(vc=None), NULL), (dict(k=_off(8)), ALIGN), (dict(kc=_off(8)), ALIGN),
                        (dict(slots=_off(4)), ALIGN), (dict(err=_off(2)), ALIGN)):
        assert call(lib, **bad) == status, bad
    assert call(lib, T=0, k=None, v=None, slots=None) == OK


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_attention_calls_refuse(lib, call):
    for bad, status in ((dict(Hq=12, Hkv=8), SHAPE), (dict(B=-1), SHAPE), (dict(maxp=0), SHAPE), (dict(np_=0), SHAPE),
                        (dict(W=-1), SHAPE), (dict(S=-1), SHAPE), (dict(sm=float("nan")), SHAPE),
                        (dict(sm=float("inf")), SHAPE), (dict(odt=5), DTYPE), (dict(Hq=18, Hkv=2), UNSUPPORTED),
                        (dict(D=64), UNSUPPORTED), (dict(P=512), UNSUPPORTED), (dict(B=8193), UNSUPPORTED),
                        (dict(np_=1 << 28, P=256), UNSUPPORTED), (dict(psz=A, maxp=1 << 24), UNSUPPORTED),
                        (dict(q=None), NULL), (dict(bt=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
                        (dict(q=_off(8)), ALIGN), (dict(out=_off(8)), ALIGN), (dict(bt=_off(2)), ALIGN),
                        (dict(psz=_off(2)), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=_off(16)), WORKSPACE)):
        assert call(lib, **bad) == status, bad
    assert call(lib, B=0, q=None, bt=None, lens=None, out=None) == OK


def test_more_refusals(lib):
    assert _decode(lib, maxl=-1) == SHAPE
    for bad in (dict(T=-1), dict(maxq=-1), dict(maxkv=-1), dict(tot=-1), dict(sm=0.0), dict(sm=-1.0)):
        assert _prefill(lib, **bad) == SHAPE, bad
    assert _prefill(lib, T=0, q=None) == OK
    assert _prefill(lib, wsb=16) == WORKSPACE
    assert _prefill(lib, cu=_off(2)) == ALIGN
    assert pkv.pkv_decode_fp4_workspace_size(2, 12, 8) == 0
    assert pkv.pkv_decode_fp4_workspace_size(2, 16, 8, page_size=8) == 0
    assert pkv.pkv_decode_fp4_workspace_size(2, 16, 8, max_seq_len=-1) == 0
    for bad in ((-1, 8, 1, 64), (1, 0, 1, 64), (1, 8, -1, 64), (1, 8, 1, -1), (1, 8, 1, 64, -1), (1, 8, 1, 64, 0, -1),
                (1, 8, 1, 64, 0, 0, -1)):
        assert pkv.pkv_prefill_fp4_workspace_size(*bad) == 0, bad


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0: the checks never read it."""
    is_cuda = True

    def get_device(self):
        return 0


def _fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


def test_binding_refuses():
    f32, u8, i64 = torch.float32, torch.uint8, torch.int64
    z, s, slots = _fake(3, 2, 128), _fake(2), _fake(3, dtype=i64)
    pool = _fake(4, 2, 16, 72, dtype=u8)
    good = dict(k_new=z, v_new=z, slot_mapping=slots, k_scale=s, v_scale=s, k_cache=pool, v_cache=pool)
    for name, bad, error in (("k_new", torch.zeros(3, 2, 128), ValueError), ("k_new", 3, TypeError),
                             ("v_new", z.to(torch.bfloat16), TypeError), ("k_new", _fake(3, 128), ValueError),
                             ("v_new", _fake(2, 2, 128), ValueError), ("slot_mapping", _fake(3), TypeError),
                             ("slot_mapping", _fake(4, dtype=i64), ValueError), ("k_scale", _fake(3), ValueError),
                             ("v_scale", _fake(2, dtype=torch.float64), TypeError),
                             ("k_cache", _fake(4, 2, 16, 128, dtype=u8), ValueError),
                             ("v_cache", _fake(4, 2, 32, 72, dtype=u8), ValueError),
                             ("k_new", _fake(3, 128, 2).transpose(1, 2), ValueError),
                             ("k_cache", torch.zeros(4, 2, 16, 72, dtype=u8), ValueError)):
        with pytest.raises(error):
            pkv.kv_append_fp4(**{**good, name: bad})
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        pkv.kv_append_fp4(**{**good, "k_new": z.half(), "v_new": z.half()})
    with pytest.raises(ValueError, match="both outputs"):
        pkv.kv_read_fp4(slots, s, s, pool, pool, k_out=z)
    with pytest.raises(ValueError, match="negative"):
        pkv._check_window(-1, 0)

    q = _fake(3, 4, 128).to(torch.bfloat16)
    bt, lens = _fake(3, 5, dtype=torch.int32), _fake(3, dtype=torch.int32)
    ws = _fake(1024, dtype=u8)
    good = dict(q=q, k_cache=pool, v_cache=pool, k_scale=s, v_scale=s, block_table=bt, seq_lens=lens, out=q,
                workspace=ws)
    for name, bad, error in (("q", z, ValueError), ("q", _fake(3, 4, 128), TypeError), ("out", _fake(3, 4, 64), ValueError),
                             ("out", q.half(), TypeError), ("block_table", _fake(2, 5, dtype=torch.int32), ValueError),
                             ("seq_lens", _fake(2, dtype=torch.int32), ValueError), ("k_scale", _fake(3), ValueError),
                             ("seq_lens", _fake(3), TypeError), ("workspace", s, TypeError), ("window", -1, ValueError),
                             ("seq_page_sizes", _fake(2, dtype=torch.int32), ValueError), ("sinks", -2, ValueError)):
        with pytest.raises(error):
            pkv.pkv_paged_gqa_decode_fp4(**{**good, name: bad})
    pre = dict(good, cu_q=_fake(4, dtype=torch.int32), max_q_len=2, max_kv_len=80)
    for name, bad, error in (("cu_q", lens, ValueError), ("cu_q", _fake(4), TypeError), ("out", z, ValueError),
                             ("window", -1, ValueError), ("k_cache", _fake(4, 1, 16, 72, dtype=u8), ValueError)):
        with pytest.raises(error):
            pkv.pkv_paged_prefill_fp4(**{**pre, name: bad})


# ---------------------------------------------------------------- the plain form
def test_plain_scales_match_the_fp8_oracle():
    """Block scales are E4M3 of amax / (6 k): the FP8 oracle's own cast."""
    rng = np.random.default_rng(0)
    x = fp4_ref.rows(rng, 200, 2) * np.exp(rng.standard_normal((200, 2, 1)) * 4).astype(np.float32)
    k = np.array([0.02, 1.7], np.float32)
    _, s = fp4_ref.quantise(x, k)
    amax = np.abs(x.reshape(200, 2, 8, 16)).max(-1)
    ratio = (amax / (np.float32(6) * k.reshape(1, 2, 1))).astype(np.float32)
    assert np.array_equal(s, oracle.e4m3_encode(ratio))


def test_plain_codes_are_the_nearest_ones():
    """No code is further from x than any other of its block's values, and a
    tie goes to the even code."""
    rng = np.random.default_rng(1)
    k = np.array([1.0], np.float32)
    x = (rng.integers(-48, 49, (64, 1, 128)) / 8.0).astype(np.float32)      # many exact ties
    x[:, :, ::16] = 6.0                                                     # every block's scale is 1
    c, s = fp4_ref.quantise(x, k)
    assert np.all(fp4_ref.e4m3_values()[s] == 1.0)
    v = fp4_ref.E2M1[c & 7] * np.where(c >= 8, -1, 1)
    every = np.concatenate((fp4_ref.E2M1, -fp4_ref.E2M1))
    best = np.abs(x[..., None] - every).min(-1)
    assert np.array_equal(np.abs(x - v), best)
    tie = (np.abs(np.abs(x)[..., None] - fp4_ref.E2M1) == best[..., None]).sum(-1) == 2
    assert tie.any() and np.all(c[tie] % 2 == 0)


def test_plain_special_values():
    k = np.array([1.0], np.float32)
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, 0:16] = np.nan
    x[0, 0, 16] = np.inf
    x[0, 0, 17] = -np.inf
    x[0, 0, 18] = 1.0
    x[0, 0, 32] = 1e6
    x[0, 0, 48] = 6 * 2.0 ** -10                                            # ratio 2^-10: a tie, to zero
    x[0, 0, 64] = 6 * 2.0 ** -9
    x[0, 0, 65] = -0.0
    c, s = fp4_ref.quantise(x, k)
    assert list(s[0, 0]) == [0x7F, 0x7E, 0x7E, 0, 1, 0, 0, 0]
    assert not c[0, 0, :16].any() and not c[0, 0, 48:64].any()
    assert list(c[0, 0, 16:19]) == [7, 15, 0] and c[0, 0, 32] == 7
    assert list(c[0, 0, 64:66]) == [7, 8]


def test_plain_round_trip_keeps_values():
    """Values that the format holds come back as they are, twice."""
    rng = np.random.default_rng(2)
    x = fp4_ref.rows(rng, 40, 3)
    k = fp4_ref.scale_of(x)
    pool = np.zeros((4, 3, 16, 72), np.uint8)
    slots = rng.permutation(64)[:40]
    fp4_ref.write(pool, *fp4_ref.quantise(x, k), slots)
    y = (fp4_ref.block_values(pool, slots) * k.reshape(1, 3, 1)).astype(np.float32)
    again = pool.copy()
    fp4_ref.write(again, *fp4_ref.quantise(y, k), slots)
    z = (fp4_ref.block_values(again, slots) * k.reshape(1, 3, 1)).astype(np.float32)
    assert np.array_equal(y, z)
    # the largest step around a value is a third of it (4 to 6) and half of that is its error; the
    # block's largest value is clipped by at most 1/16, what lies below half the smallest code is lost
    amax = np.abs(x.reshape(40, 3, 8, 16)).max(-1, keepdims=True)
    err = np.abs(x - y).reshape(40, 3, 8, 16)
    assert np.all(err <= amax * (1.0 / 6 + 1.0 / 16))


def test_plain_window_counts():
    assert list(fp4_ref.visible(9, 3, 2)) == [0, 1, 7, 8, 9]
    assert list(fp4_ref.visible(9, 3, 0)) == [7, 8, 9]
    assert list(fp4_ref.visible(9, 3, 100)) == list(range(10))
    assert list(fp4_ref.visible(9, 0, 5)) == list(range(10))
    assert list(fp4_ref.visible(0, 1, 0)) == [0]
    assert fp4_ref.visible(-1, 4, 4).size == 0


def test_binding_refuses_what_is_no_tensor():
    u8, i32 = torch.uint8, torch.int32
    pool, s = _fake(4, 2, 16, 72, dtype=u8), _fake(2)
    q = _fake(3, 4, 128).to(torch.bfloat16)
    good = dict(q=q, k_cache=pool, v_cache=pool, k_scale=s, v_scale=s, block_table=_fake(3, 5, dtype=i32),
                seq_lens=_fake(3, dtype=i32), out=q, workspace=_fake(64, dtype=u8))
    for name in good:
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            pkv.pkv_paged_gqa_decode_fp4(**{**good, name: [1, 2, 3]})
    with pytest.raises(TypeError, match="cu_q must be a torch.Tensor"):
        pkv.pkv_paged_prefill_fp4(**good, cu_q=[0, 1, 2, 3], max_q_len=2, max_kv_len=80)
    rows = dict(slot_mapping=_fake(3, dtype=torch.int64), k_scale=s, v_scale=s, k_cache=pool, v_cache=pool,
                k_out=_fake(3, 2, 128), v_out=_fake(3, 2, 128))
    for name in rows:
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            pkv.pkv_kv_read_fp4(**{**rows, name: 5})
