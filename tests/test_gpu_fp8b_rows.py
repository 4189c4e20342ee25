"""Writing the block-scaled FP8 cache and reading it back: codes and exponent
bytes equal the plain form's, bit for bit, and so do the values read."""
import numpy as np
import pytest
import torch

from tests import fp4_ref, fp8b_ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


class Pools:
    """K and V pools on the device beside the plain form's, filled with the
    blocks of earlier requests."""

    def __init__(self, rng, pages, H, P, dev, pkv):
        self.pkv, self.dev = pkv, dev
        self.cache = [rng.integers(0, 256, (pages, H, P, 128), dtype=np.uint8) for _ in range(2)]
        self.exps = [rng.integers(110, 140, (pages, H, P // 16), dtype=np.uint8) for _ in range(2)]
        self.cache_d, self.exps_d = [_dev(c, dev) for c in self.cache], [_dev(e, dev) for e in self.exps]

    def args(self):
        return (*self.cache_d, *self.exps_d)

    def append(self, rows, slots, dtype, err=0):
        e = torch.zeros(1, dtype=torch.int32, device=self.dev)
        new = [_dev(r, self.dev).to(dtype) for r in rows]
        self.pkv.kv_append_fp8b(*new, _dev(slots, self.dev), *self.args(), device_error=e)
        for x, c, s in zip(new, self.cache, self.exps):
            fp8b_ref.append(c, s, x.float().cpu().numpy(), slots)
        assert int(e.item()) == err
        self.check()

    def check(self):
        for got, ref in zip(self.exps_d, self.exps):
            assert (got.cpu().numpy() == ref).all(), np.argwhere(got.cpu().numpy() != ref)[:4]
        for got, ref in zip(self.cache_d, self.cache):
            assert fp8b_ref.same(got.cpu().numpy(), ref)


def _two(rng, T, H, spread=1.0):
    return [fp4_ref.rows(rng, T, H, spread) * np.exp(rng.standard_normal((T, 1, 1))).astype(np.float32) for _ in range(2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,P,T", [(8, 16, 1), (1, 16, 16), (5, 32, 100), (3, 64, 513), (2, 128, 777), (1, 256, 4099),
                                   (9, 16, 64)])
def test_append_a_sequence(pkv, cuda_device, dtype, H, P, T):
    """A chunk from position 0, and one that starts inside a block."""
    rng = np.random.default_rng(T + H)
    pages = T // P + 4
    p = Pools(rng, 2 * pages, H, P, cuda_device, pkv)
    for past in (0, 5):
        table = rng.permutation(2 * pages)
        pos = np.arange(past, past + T)
        p.append(_two(rng, T, H), (table[pos // P] * P + pos % P).astype(np.int64), DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_token_by_token(pkv, cuda_device, dtype):
    """Decode steps of a batch: blocks begin, grow and keep their exponent; rows
    that were there are rounded where it grows."""
    rng = np.random.default_rng(3)
    B, H, P, steps = 9, 3, 32, 40
    p = Pools(rng, 2 * B + 1, H, P, cuda_device, pkv)
    table = rng.permutation(2 * B).reshape(B, 2)
    start = rng.integers(0, 20, B)
    for i in range(steps):
        pos = start + i
        slots = (table[np.arange(B), pos // P] * P + pos % P).astype(np.int64)
        p.append([x * 2.0 ** (i % 7) for x in _two(rng, B, H)], slots, DTYPES[dtype])


@pytest.mark.parametrize("T", [1, 31, 700, 5000])
def test_append_in_any_order_with_padding(pkv, cuda_device, T):
    """A block's tokens in any order within 32 of the call's, padding between
    them, runs that begin and end inside blocks, rows 0 left out."""
    rng = np.random.default_rng(T)
    H, P = 2, 64
    blocks = T // 8 + 2
    p = Pools(rng, blocks * 16 // P + 2, H, P, cuda_device, pkv)
    slots, ids = [], rng.permutation(blocks)
    for b in ids:
        rows = rng.permutation(16)[:rng.integers(1, 17)]
        run = np.concatenate((16 * b + rows, np.full(rng.integers(0, 32 - len(rows) + 1), -1)))
        slots.append(rng.permutation(run))
        if rng.random() < 0.2:
            slots.append(np.full(rng.integers(1, 90), -7))
    slots = np.concatenate(slots)[:T].astype(np.int64)
    p.append(_two(rng, len(slots), H), slots, torch.float32)


def test_append_special_values(pkv, cuda_device):
    """Zeros, the smallest and largest numbers, both sides of a border between
    exponents, infinities and NaN; a block of nothing but them."""
    rng = np.random.default_rng(5)
    p = Pools(rng, 9, 2, 16, cuda_device, pkv)
    rows = _two(rng, 9 * 16, 2)
    x = rows[0]
    x[0:16] = 0
    x[16:32] *= 1e-44
    x[32:48] = np.float32(3.4e38) * np.sign(x[32:48])
    x[48:64] = np.clip(x[48:64], -1, 1)
    x[48, 0, 3], x[48, 1, 3] = 448, np.nextafter(np.float32(448), np.float32(1e3))
    x[64:80, 0, 5], x[65, 1, 7], x[70, 0, 9] = np.nan, np.inf, -np.inf
    x[80:96] = np.nan
    x[96:112] = np.inf
    x[112:128] = -0.0
    with np.errstate(over="ignore"):
        rows[1][100:] *= np.float32(1e30)
    slots = np.arange(9 * 16, dtype=np.int64)
    p.append(rows, slots, torch.float32)
    # and rows added to such blocks, one at a time
    for r in (3, 9):
        new = _two(rng, 9, 2, 1e-3)
        p.append(new, (np.arange(9) * 16 + r).astype(np.int64), torch.bfloat16)
        p.append([y * 1e6 for y in new], (np.arange(9) * 16 + r + 1).astype(np.int64), torch.float32)


def test_append_slots_outside_the_pool(pkv, cuda_device):
    rng = np.random.default_rng(6)
    p = Pools(rng, 4, 2, 16, cuda_device, pkv)
    p.append(_two(rng, 5, 2), np.array([3, 64, -1, 2 ** 40, 20], np.int64), torch.float32, err=pkv.DEVERR_SLOT)
    p.append(_two(rng, 0, 2), np.zeros(0, np.int64), torch.float32)


def test_append_beyond_32_bits(pkv, cuda_device):
    """The last pages of a pool of more than 2^31 bytes."""
    H, P, pages = 8, 256, 9000                                   # 2.36e9 bytes of codes
    cache = torch.zeros((pages, H, P, 128), dtype=torch.uint8, device=cuda_device)
    exps = torch.zeros((pages, H, P // 16), dtype=torch.uint8, device=cuda_device)
    rng = np.random.default_rng(7)
    x = fp4_ref.rows(rng, 40, H)
    slots = np.arange(pages * P - 40, pages * P, dtype=np.int64)
    xd, sd = _dev(x, cuda_device), _dev(slots, cuda_device)
    v = torch.zeros_like(cache)
    ve = torch.zeros_like(exps)
    pkv.kv_append_fp8b(xd, xd, sd, cache, v, exps, ve)
    k_out, v_out = pkv.kv_read_fp8b(sd, cache, v, exps, ve, out_dtype=torch.float32)
    c, e = np.zeros((1, H, P, 128), np.uint8), np.zeros((1, H, P // 16), np.uint8)
    fp8b_ref.append(c, e, x, slots - (pages - 1) * P)
    ref = fp8b_ref.read(c, e, slots - (pages - 1) * P)
    assert (k_out.double().cpu().numpy() == ref).all() and torch.equal(k_out, v_out)
    assert int(cache[:-1].count_nonzero()) == 0 and int(exps[:-1].count_nonzero()) == 0


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("H,P,T", [(1, 16, 1), (8, 16, 100), (3, 64, 999), (5, 256, 4097)])
def test_read(pkv, cuda_device, out, H, P, T):
    rng = np.random.default_rng(T)
    pages = 40
    p = Pools(rng, pages, H, P, cuda_device, pkv)
    slots = rng.integers(0, pages * P, T).astype(np.int64)       # some more than once
    slots[rng.random(T) < 0.1] = -3
    if T > 50:
        slots[17] = pages * P
    e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    outs = [torch.full((T, H, 128), 7.0, dtype=DTYPES[out], device=cuda_device) for _ in range(2)]
    pkv.kv_read_fp8b(_dev(slots, cuda_device), *p.args(), k_out=outs[0], v_out=outs[1], device_error=e)
    assert int(e.item()) == (pkv.DEVERR_SLOT if T > 50 else 0)
    for got, c, x in zip(outs, p.cache, p.exps):
        ref = fp8b_ref.read(c, x, slots)
        got = got.double().cpu().numpy()
        assert (got[slots < 0] == 7).all()
        assert np.array_equal(got[slots >= 0], ref[slots >= 0], equal_nan=True)


def test_read_every_code_and_byte(pkv, cuda_device):
    """All 256 codes with the exponents that append can write, and with bytes it
    cannot, as far as fp32 holds them."""
    pages = 256
    cache = np.zeros((pages, 1, 16, 128), np.uint8)
    cache[:, 0, 0], cache[:, 0, 1] = np.arange(128), np.arange(128, 256)
    exps = np.arange(256, dtype=np.uint8).reshape(pages, 1, 1)
    cd, ed = _dev(cache, cuda_device), _dev(exps, cuda_device)
    slots = np.concatenate((np.arange(255) * 16, np.arange(255) * 16 + 1))
    ref = fp8b_ref.read(cache, exps, slots)
    k, _ = pkv.kv_read_fp8b(_dev(slots, cuda_device), cd, cd, ed, ed, out_dtype=torch.float32)
    with np.errstate(over="ignore"):
        assert np.array_equal(k.cpu().numpy(), ref.astype(np.float32), equal_nan=True)
    k, _ = pkv.kv_read_fp8b(_dev(slots, cuda_device), cd, cd, ed, ed)
    mine = (slots // 16 >= 10) & (slots // 16 <= 246)
    assert np.array_equal(k.double().cpu().numpy()[mine], ref[mine], equal_nan=True)


def test_rows_in_a_graph_and_on_another_stream(pkv, cuda_device):
    rng = np.random.default_rng(8)
    a, b = (Pools(np.random.default_rng(9), 8, 2, 16, cuda_device, pkv) for _ in range(2))
    x = [_dev(r, cuda_device) for r in _two(rng, 50, 2)]
    slots = _dev(np.arange(60, 110, dtype=np.int64), cuda_device)
    pkv.kv_append_fp8b(*x, slots, *a.args())
    ref = pkv.kv_read_fp8b(slots, *a.args())
    torch.cuda.synchronize()
    out = [torch.zeros_like(r) for r in ref]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_append_fp8b(*x, slots, *b.args())
        pkv.kv_read_fp8b(slots, *b.args(), k_out=out[0], v_out=out[1])
    g.replay()
    torch.cuda.synchronize()
    for i, j in zip((*ref, *a.args()), (*out, *b.args())):
        assert torch.equal(i, j)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.kv_read_fp8b(slots, *a.args(), stream=side)
    side.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(got, ref))
