"""Plain CUDA tensors that do not fit, through the compiled fast path of the binding: it hands
them back, the checks in Python say what is wrong, and nothing is written.  And what both
paths do with arguments that fit is the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu

u8, i32, i64, bf, f32 = torch.uint8, torch.int32, torch.int64, torch.bfloat16, torch.float32


def _t(*shape, dtype=f32, device="cuda"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def _calls(pkv):
    """name: (call, arguments that fit, arguments that do not with their errors)."""
    z, slots, pool, exps = _t(3, 2, 128), _t(3, dtype=i64), _t(4, 2, 32, 128, dtype=u8), _t(4, 2, 2, dtype=u8)
    slots += torch.arange(3, device="cuda")
    caches = dict(k_cache=pool, v_cache=pool.clone(), k_exp=exps, v_exp=exps.clone())
    err = _t(1, dtype=i32)
    bad_caches = [("k_cache", _t(4, 2, 32, 72, dtype=u8), ValueError), ("v_cache", _t(5, 2, 32, 128, dtype=u8), ValueError),
                  ("k_cache", _t(4, 2, 32, 128), TypeError), ("k_exp", _t(4, 2, 1, dtype=u8), ValueError),
                  ("v_exp", _t(4, 2, 2), TypeError), ("k_exp", _t(4, 2, 2, dtype=u8, device="cpu"), ValueError),
                  ("k_cache", _t(4, 2, 32, dtype=u8), ValueError), ("v_cache", _t(4, 32, 2, 128, dtype=u8).transpose(1, 2), ValueError),
                  ("device_error", _t(1, dtype=i64), TypeError), ("device_error", _t(1, dtype=i32, device="cpu"), ValueError)]
    rows = dict(k_new=z + 1, v_new=z + 2, slot_mapping=slots, device_error=err, **caches)
    bad_rows = [("k_new", _t(3, 2, 128, device="cpu"), ValueError), ("k_new", None, TypeError), ("v_new", _t(3, 2, 128, dtype=bf), TypeError),
                ("v_new", _t(2, 2, 128), ValueError), ("k_new", _t(3, 2, 128, dtype=torch.float16), TypeError),
                ("k_new", _t(3, 128, 2).transpose(1, 2), ValueError), ("slot_mapping", _t(3, dtype=i32), TypeError),
                ("slot_mapping", _t(2, dtype=i64), ValueError), ("slot_mapping", _t(6, dtype=i64)[::2], ValueError)]
    read = dict(slot_mapping=slots, k_out=_t(3, 2, 128), v_out=_t(3, 2, 128), device_error=err, **caches)
    bad_read = [("k_out", _t(3, 3, 128), ValueError), ("v_out", _t(3, 2, 128, device="cpu"), ValueError),
                ("k_out", _t(3, 2, 128, dtype=i32), TypeError), ("v_out", _t(3, 2, 256)[..., ::2], ValueError)]
    q = torch.randn(2, 8, 128, device="cuda").to(bf)
    attn = dict(q=q, block_table=_t(2, 3, dtype=i32), seq_lens=_t(2, dtype=i32) + 40, out=_t(2, 8, 128), device_error=err, **caches)
    bad_attn = [("q", _t(2, 8, 128), TypeError), ("q", _t(2, 8, 128, dtype=bf, device="cpu"), ValueError),
                ("q", _t(8, 2, 128, dtype=bf).transpose(0, 1), ValueError), ("out", _t(2, 8, 64), ValueError),
                ("out", _t(2, 8, 128, dtype=torch.float16), TypeError), ("block_table", _t(3, 3, dtype=i32), ValueError),
                ("block_table", _t(2, 6, dtype=i32)[:, ::2], ValueError), ("block_table", _t(2, 3, dtype=i64), TypeError),
                ("seq_lens", _t(2), TypeError), ("seq_lens", _t(2, dtype=i32, device="cpu"), ValueError),
                ("workspace", _t(64), TypeError), ("workspace", _t(64, dtype=u8), pkv.PkvError), ("window", -1, ValueError),
                ("sinks", -1, ValueError), ("seq_page_sizes", _t(3, dtype=i32), ValueError), ("seq_page_sizes", _t(2), TypeError),
                ("sm_scale", float("nan"), pkv.PkvError)]
    past, new = _t(2, dtype=i32), _t(2, dtype=i32) + 1
    plan = dict(past_lens=past, new_lens=new, block_table=_t(2, 3, dtype=i32), pool=pkv.page_pool(8, "cuda"), page_size=16,
                seq_lens=_t(2, dtype=i32), cu_q=_t(3, dtype=i32), slot_mapping=_t(3, dtype=i64), positions=_t(3, dtype=i32),
                device_error=err)
    bad_plan = [("past_lens", _t(2), TypeError), ("past_lens", _t(2, dtype=i32, device="cpu"), ValueError),
                ("new_lens", _t(3, dtype=i32), ValueError), ("new_lens", _t(4, dtype=i32)[::2], ValueError),
                ("block_table", _t(3, 3, dtype=i32), ValueError), ("pool", _t(4, dtype=i32), ValueError), ("pool", _t(12), TypeError),
                ("seq_lens", _t(1, dtype=i32), ValueError), ("cu_q", _t(2, dtype=i32), ValueError),
                ("slot_mapping", _t(3, dtype=i32), TypeError), ("positions", _t(2, dtype=i32), ValueError),
                ("positions", _t(3, dtype=i64), TypeError), ("page_size", 24, pkv.PkvError), ("page_size", -16, pkv.PkvError)]
    table = torch.tensor([[4, 5, 0], [6, 7, 0]], dtype=i32, device="cuda")
    release = dict(seq_lens=_t(2, dtype=i32) + 20, block_table=table, pool=pkv.page_pool(8, "cuda", range(4)), page_size=16,
                   keep_lens=_t(2, dtype=i32), device_error=err)
    bad_release = [("keep_lens", _t(3, dtype=i32), ValueError), ("pool", _t(3, dtype=i32), ValueError),
                   ("seq_lens", _t(2, dtype=i32, device="cpu"), ValueError), ("block_table", _t(2, 3, dtype=i64), TypeError),
                   ("page_size", 48, pkv.PkvError)]
    return {
        "append": (pkv.kv_append_fp8b, rows, bad_caches + bad_rows),
        "read": (pkv.kv_read_fp8b, read, bad_caches + bad_read),
        "decode": (pkv.paged_gqa_decode_fp8b, dict(max_seq_len=64, **attn),
                   bad_caches + bad_attn + [("max_seq_len", 1 << 31, ValueError), ("max_seq_len", -1, pkv.PkvError),
                                            ("max_ctas", 1 << 32, ValueError), ("max_ctas", -1, pkv.PkvError)]),
        "prefill": (pkv.paged_prefill_fp8b, dict(cu_q=_t(3, dtype=i32) + torch.arange(3, dtype=i32, device="cuda"), max_q_len=1,
                                                 max_kv_len=64, **attn),
                    bad_caches + bad_attn + [("cu_q", _t(2, dtype=i32), ValueError), ("cu_q", _t(3, dtype=i64), TypeError),
                                             ("max_q_len", 1 << 31, ValueError), ("max_kv_len", 1 << 40, ValueError),
                                             ("sm_scale", 0.0, pkv.PkvError)]),
        "plan": (pkv.plan_pages, plan, bad_plan),
        "release": (pkv.release_pages, release, bad_release),
    }


NAMES = ["append", "read", "decode", "prefill", "plan", "release"]


def _tensors(args):
    return {n: x for n, x in args.items() if isinstance(x, torch.Tensor)}


@pytest.mark.parametrize("name", NAMES)
def test_refusals(pkv, cuda_device, name):
    call, good, bad = _calls(pkv)[name]
    assert pkv._fast is not pkv._NoFast
    before = {n: x.clone() for n, x in _tensors(good).items()}
    for arg, value, error in bad:
        args = {**good, arg: value}
        kept = value.clone() if isinstance(value, torch.Tensor) else None
        with pytest.raises(error):
            call(**args)
        torch.cuda.synchronize()
        for n, x in _tensors(good).items():
            assert torch.equal(x, before[n]), (arg, value, n)
        assert kept is None or torch.equal(value, kept)


@pytest.mark.parametrize("name", NAMES)
def test_the_same_without_the_fast_path(pkv, cuda_device, monkeypatch, name):
    """(random fields of the caches: the same ones for both)"""
    results = []
    for fast in (True, False):
        call, good, _ = _calls(pkv)[name]
        gen = torch.Generator("cuda").manual_seed(5)
        for n in ("k_cache", "v_cache", "k_exp", "v_exp"):
            if n in good:
                good[n].random_(100, 126, generator=gen)
        if "q" in good:
            good["q"].normal_(generator=gen)
        if not fast:
            monkeypatch.setattr(pkv, "_fast", pkv._NoFast)
        call(**good)
        torch.cuda.synchronize()
        results.append(_tensors(good))
    changed = 0
    for n, x in results[0].items():
        assert torch.equal(x, results[1][n]), n
        changed += not torch.equal(x, _tensors(_calls(pkv)[name][1])[n])
    assert changed > 0
