"""The 4-bit cache's writer and reader on the GPU: page bytes equal to the
plain form's, values equal to its products."""
import numpy as np
import pytest
import torch

from tests import fp4_ref

pytestmark = pytest.mark.gpu


def _dev(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _pools(pages, H, P, dev, byte=0xAB):
    return [torch.full((pages, H, P, 72), byte, dtype=torch.uint8, device=dev) for _ in range(2)]


def _expect(k, v, ks, vs, slots, pages, H, P, byte=0xAB):
    out = []
    for x, s in ((k, ks), (v, vs)):
        pool = np.full((pages, H, P, 72), byte, np.uint8)
        fp4_ref.write(pool, *fp4_ref.quantise(x, s), slots)
        out.append(pool)
    return out


@pytest.mark.parametrize("T,H,P", [(1, 1, 16), (1, 8, 16), (5, 3, 32), (64, 8, 16), (33, 7, 64), (257, 2, 128),
                                   (130, 5, 256), (1021, 1, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_are_the_plain_forms(pkv, cuda_device, T, H, P, dtype):
    rng = np.random.default_rng(T * 31 + H * 7 + P)
    k, v = fp4_ref.rows(rng, T, H), fp4_ref.rows(rng, T, H)
    ks, vs = fp4_ref.scale_of(k), fp4_ref.scale_of(v) * np.float32(0.7)      # some blocks of V saturate
    if dtype == "bf16":
        kb, vb = fp4_ref.to_bf16_bits(k), fp4_ref.to_bf16_bits(v)
        k, v = fp4_ref.from_bf16_bits(kb), fp4_ref.from_bf16_bits(vb)
        kt, vt = (_dev(b.view(np.int16), cuda_device).view(torch.bfloat16) for b in (kb, vb))
    else:
        kt, vt = _dev(k, cuda_device), _dev(v, cuda_device)
    pages = T // P + 3
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    slots[::9] = -1
    kc, vc = _pools(pages, H, P, cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    st = _dev(slots, cuda_device)
    pkv.kv_append_fp4(kt, vt, st, _dev(ks, cuda_device), _dev(vs, cuda_device), kc, vc, err)
    ek, ev = _expect(k, v, ks, vs, slots, pages, H, P)
    assert np.array_equal(kc.cpu().numpy(), ek)
    assert np.array_equal(vc.cpu().numpy(), ev)

    for out_dtype in (torch.float32, torch.bfloat16):
        ko = torch.full((T, H, 128), 7.0, dtype=out_dtype, device=cuda_device)
        vo = torch.full_like(ko, 7.0)
        pkv.kv_read_fp4(st, _dev(ks, cuda_device), _dev(vs, cuda_device), kc, vc, ko, vo, device_error=err)
        for got, pool, s in ((ko, ek, ks), (vo, ev, vs)):
            exp = torch.from_numpy((fp4_ref.block_values(pool, slots) * s.reshape(1, H, 1)).astype(np.float32))
            exp = exp.to(out_dtype)
            exp[torch.from_numpy(slots < 0)] = 7.0
            assert torch.equal(got.cpu(), exp)
    assert int(err.item()) == 0


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-12, 3.7e-5, 1.0, 2.0 ** 100])
def test_every_ratio_rounds_like_the_plain_form(pkv, cuda_device, scale):
    """Values around every border of both conversions, at extreme scales."""
    rng = np.random.default_rng(5)
    T = 512
    x = (rng.integers(-52, 53, (T, 1, 128)) / 8.0).astype(np.float32)
    x *= (1.0 + rng.integers(-2, 3, x.shape) * 2.0 ** -23).astype(np.float32)
    x[:, :, ::16] *= rng.choice([1e-3, 0.02, 1.0, 30.0, 447.0, 1e4], (T, 1, 8)).astype(np.float32)
    with np.errstate(over="ignore"):
        x = (x * np.float32(scale)).astype(np.float32)
    k = np.array([scale], np.float32)
    kc, vc = _pools(T // 16, 1, 16, cuda_device)
    slots = np.arange(T, dtype=np.int64)
    pkv.kv_append_fp4(_dev(x, cuda_device), _dev(-x, cuda_device), _dev(slots, cuda_device), _dev(k, cuda_device),
                      _dev(k, cuda_device), kc, vc)
    ek, ev = _expect(x, -x, k, k, slots, T // 16, 1, 16)
    assert np.array_equal(kc.cpu().numpy(), ek)
    assert np.array_equal(vc.cpu().numpy(), ev)


def test_special_values(pkv, cuda_device):
    x = np.zeros((16, 1, 128), np.float32)
    x[0, 0, :16] = np.nan
    x[1, 0, 3] = np.nan
    x[2, 0, 16], x[2, 0, 17], x[2, 0, 18] = np.inf, -np.inf, 1.0
    x[3, 0, 0], x[3, 0, 1] = 3e38, -3e38
    x[4, 0, 0], x[4, 0, 1] = 6 * 2.0 ** -10, 6 * 2.0 ** -9
    x[5] = -0.0
    x[6, 0, 0], x[6, 0, 1] = 1.0, -1e-30
    x[7] = 1e-38
    k = np.ones(1, np.float32)
    slots = np.arange(16, dtype=np.int64)
    kc, vc = _pools(1, 1, 16, cuda_device)
    st, kt = _dev(slots, cuda_device), _dev(k, cuda_device)
    pkv.kv_append_fp4(_dev(x, cuda_device), _dev(x, cuda_device), st, kt, kt, kc, vc)
    ek, _ = _expect(x, x, k, k, slots, 1, 1, 16)
    assert np.array_equal(kc.cpu().numpy(), ek) and torch.equal(kc, vc)
    got, _ = pkv.kv_read_fp4(st, kt, kt, kc, vc, out_dtype=torch.float32)
    assert torch.isnan(got[0, 0, :16]).all() and torch.isnan(got[1, 0, :16]).all()
    assert not torch.isnan(got[0, 0, 16:]).any() and not torch.isnan(got[2:]).any()
    assert got[2, 0, 16] == 2688 and got[2, 0, 17] == -2688 and got[2, 0, 18] == 0


def test_slots_outside_the_pool(pkv, cuda_device):
    x = torch.ones(4, 2, 128, device=cuda_device)
    slots = torch.tensor([-1, 3, 64, 1 << 40], dtype=torch.int64, device=cuda_device)
    s = torch.ones(2, device=cuda_device)
    kc, vc = _pools(4, 2, 16, cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    pkv.kv_append_fp4(x, x, slots, s, s, kc, vc, err)
    assert int(err.item()) == pkv.DEVERR_SLOT
    one = np.ones((4, 2, 128), np.float32)
    ek, _ = _expect(one, one, np.ones(2, np.float32), np.ones(2, np.float32), [-1, 3, -1, -1], 4, 2, 16)
    assert np.array_equal(kc.cpu().numpy(), ek) and np.array_equal(vc.cpu().numpy(), ek)
    err.zero_()
    ko = torch.full((4, 2, 128), 7.0, device=cuda_device)
    vo = torch.full((4, 2, 128), 8.0, device=cuda_device)
    pkv.kv_read_fp4(slots, s, s, kc, vc, ko, vo, device_error=err)
    assert int(err.item()) == pkv.DEVERR_SLOT
    # a block of ones: s = E4M3(1 / 6) = 1.375 / 8 (the nearer of 1.25 / 8 and 1.375 / 8), codes 6
    assert (ko[0] == 7).all() and (vo[0] == 8).all()
    assert (ko[1] == 6 * 1.375 / 8).all() and (vo[1] == 6 * 1.375 / 8).all()
    assert (ko[2:] == 0).all() and (vo[2:] == 0).all()


def test_empty_and_repeated(pkv, cuda_device):
    s = torch.ones(2, device=cuda_device)
    kc, vc = _pools(2, 2, 16, cuda_device, 0x11)
    none = torch.empty(0, 2, 128, device=cuda_device)
    pkv.kv_append_fp4(none, none, torch.empty(0, dtype=torch.int64, device=cuda_device), s, s, kc, vc)
    assert (kc == 0x11).all()
    k, v = pkv.kv_read_fp4(torch.tensor([5, 5, 5], device=cuda_device), s, s, kc, vc)
    assert k.shape == (3, 2, 128) and torch.equal(k[0], k[1]) and torch.equal(k[0], k[2]) and torch.equal(k, v)
    k, _ = pkv.kv_read_fp4(torch.tensor([-1], device=cuda_device), s, s, kc, vc)
    assert (k == 0).all()


def test_offsets_past_32_bits(pkv, cuda_device):
    """A pool of more than 2^32 bytes: its last and first pages."""
    pages, H, P = 240_000, 16, 16                                # 4.4 GB a pool
    kc, vc = [torch.empty((pages, H, P, 72), dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    rng = np.random.default_rng(8)
    x = fp4_ref.rows(rng, 6, H)
    s = fp4_ref.scale_of(x)
    slots = np.array([pages * P - 1, 0, pages * P - 17, 1, 233_017 * P + 5, 7], np.int64)
    st, sd, xd = (_dev(a, cuda_device) for a in (slots, s, x))
    pkv.kv_append_fp4(xd, xd, st, sd, sd, kc, vc)
    got, _ = pkv.kv_read_fp4(st, sd, sd, kc, vc, out_dtype=torch.float32)
    codes, scales = fp4_ref.quantise(x, s)
    small = np.zeros((1, H, 16, 72), np.uint8)
    fp4_ref.write(small, codes, scales, range(6))
    exp = (fp4_ref.block_values(small, range(6)) * s.reshape(1, H, 1)).astype(np.float32)
    assert np.array_equal(got.cpu().numpy(), exp)


def test_on_another_stream_and_in_a_graph(pkv, cuda_device):
    rng = np.random.default_rng(9)
    x = fp4_ref.rows(rng, 40, 4)
    s = fp4_ref.scale_of(x)
    slots = rng.permutation(64)[:40].astype(np.int64)
    st, sd, xd = (_dev(a, cuda_device) for a in (slots, s, x))
    kc, vc = _pools(4, 4, 16, cuda_device)
    ko, vo = torch.zeros((40, 4, 128), device=cuda_device), torch.zeros((40, 4, 128), device=cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.kv_append_fp4(xd, xd, st, sd, sd, kc, vc, stream=side)
    pkv.kv_read_fp4(st, sd, sd, kc, vc, ko, vo, stream=side)
    side.synchronize()
    ek, _ = _expect(x, x, s, s, slots, 4, 4, 16)
    assert np.array_equal(kc.cpu().numpy(), ek) and torch.equal(ko, vo)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_append_fp4(xd, xd, st, sd, sd, kc, vc)
        pkv.kv_read_fp4(st, sd, sd, kc, vc, ko, vo)
    y = fp4_ref.rows(rng, 40, 4)
    xd.copy_(_dev(y, cuda_device))
    graph.replay()
    torch.cuda.synchronize()
    ek, _ = _expect(y, y, s, s, slots, 4, 4, 16)
    exp = (fp4_ref.block_values(ek, slots) * s.reshape(1, 4, 1)).astype(np.float32)
    assert np.array_equal(ko.cpu().numpy(), exp)


@pytest.mark.parametrize("T,H,dtype", [(9001, 8, torch.bfloat16), (70003, 5, torch.bfloat16),
                                       (40013, 8, torch.float32)])
def test_large_calls_are_small_ones(pkv, cuda_device, T, H, dtype):
    """In large calls a thread takes several tokens: pages and rows are those
    of the same tokens in small calls, with slots that are not written and
    slots outside the pool between them."""
    P, pages = 16, T // 16 + 2
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(T, H, 128, generator=g, device=cuda_device).to(dtype) for _ in range(2))
    ks, vs = (0.01 + 0.01 * torch.rand(H, generator=g, device=cuda_device) for _ in range(2))
    slots = torch.randperm(pages * P, generator=g, device=cuda_device)[:T]
    slots[5::7] = -1
    slots[T // 2] = pages * P
    slots[-1] = 1 << 40
    step = 500
    pools, outs = [], []
    for cuts in ([(0, T)], [(i, min(i + step, T)) for i in range(0, T, step)]):
        err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        kc, vc = (torch.full((pages, H, P, 72), 0x55, dtype=torch.uint8, device=cuda_device) for _ in range(2))
        for lo, hi in cuts:
            pkv.kv_append_fp4(k[lo:hi], v[lo:hi], slots[lo:hi], ks, vs, kc, vc, err)
        assert int(err.item()) == pkv.DEVERR_SLOT
        pools.append((kc, vc))
        err.zero_()
        ko, vo = (torch.full((T, H, 128), 9.0, dtype=dtype, device=cuda_device) for _ in range(2))
        for lo, hi in cuts:
            pkv.pkv_kv_read_fp4(slots[lo:hi], ks, vs, *pools[0], ko[lo:hi], vo[lo:hi], err)
        assert int(err.item()) == pkv.DEVERR_SLOT
        outs.append((ko, vo))
    for x, y in zip(pools[0] + outs[0], pools[1] + outs[1]):
        assert torch.equal(x, y)
    assert (outs[0][0][slots == -1] == 9).all() and (outs[0][0][slots >= pages * P] == 0).all()
