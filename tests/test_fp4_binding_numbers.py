"""Numbers beyond 32 bits in the 4-bit calls of the binding: windows and sinks
mean what they say, bounds are refused."""
import ctypes

import pytest
import torch

import paged_fp8_kv_03_gb300 as pkv
from tests.test_fp4_host import _fake

FAR = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 70]
MOST = 2 ** 31 - 1


@pytest.fixture
def sent(monkeypatch):
    """What the calls hand to the library, as ctypes would pass it on."""
    got = []

    def call(name, dev, stream, fn, *args):
        got.append([a if t is ctypes.c_void_p else t(a).value for t, a in zip(fn.argtypes, args)])

    monkeypatch.setattr(pkv, "_call", call)
    return got


def _good():
    pool, s, i32 = _fake(4, 2, 16, 72, dtype=torch.uint8), _fake(2), torch.int32
    q = _fake(3, 4, 128).to(torch.bfloat16)
    return dict(q=q, k_cache=pool, v_cache=pool, k_scale=s, v_scale=s, block_table=_fake(3, 5, dtype=i32),
                seq_lens=_fake(3, dtype=i32), out=q, workspace=_fake(1024, dtype=torch.uint8))


def _decode(**kw):
    pkv.pkv_paged_gqa_decode_fp4(**_good(), **kw)


def _prefill(**kw):
    pkv.pkv_paged_prefill_fp4(**_good(), cu_q=_fake(4, dtype=torch.int32), **{"max_q_len": 2, "max_kv_len": 80, **kw})


@pytest.mark.parametrize("call,window,sinks", [(_decode, 17, 18), (_prefill, 21, 22)])
def test_far_windows_and_sinks(sent, call, window, sinks):
    call(window=40, sinks=3)
    assert (sent[-1][window], sent[-1][sinks]) == (40, 3)
    for n in FAR:
        call(window=n, sinks=n)
        assert (sent[-1][window], sent[-1][sinks]) == (MOST, MOST)
    for n in (-1, -2 ** 32, -2 ** 31 - 5):
        with pytest.raises(ValueError, match="negative"):
            call(window=n)
        with pytest.raises(ValueError, match="negative"):
            call(sinks=n)


@pytest.mark.parametrize("n", FAR + [-2 ** 32 + 7])
def test_far_bounds_are_refused(sent, n):
    for call, names in ((_decode, ("max_seq_len", "max_ctas")), (_prefill, ("max_q_len", "max_kv_len"))):
        for name in names:
            with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
                call(**{name: n})
    assert not sent
    for kw in (dict(max_seq_len=n), dict(max_ctas=n)):
        with pytest.raises(ValueError, match="must fit 32 bits"):
            pkv.pkv_decode_fp4_workspace_size(2, 16, 2, **kw)
    for a in ((2, 2, n, 100), (2, 2, 100, n)):
        with pytest.raises(ValueError, match="must fit 32 bits"):
            pkv.pkv_prefill_fp4_workspace_size(*a)


def test_prefill_workspace_of_far_windows():
    whole = pkv.pkv_prefill_fp4_workspace_size(2, 2, 100, 5000)
    for n in FAR:
        assert pkv.pkv_prefill_fp4_workspace_size(2, 2, 100, 5000, 0, n) == whole
        assert pkv.pkv_prefill_fp4_workspace_size(2, 2, 100, 5000, 0, 64, n) == whole
    assert pkv.pkv_prefill_fp4_workspace_size(2, 2, 100, 5000, 0, -2 ** 32) == 0
