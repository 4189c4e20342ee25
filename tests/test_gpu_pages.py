"""The page plan: pages, tables, slots, positions and the free list equal the
plain form's."""
import numpy as np
import pytest
import torch

from tests import fp8b_ref

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(np.asarray(x, np.int32), device=dev)


class Plan:
    """A pool, a table and their plain forms."""

    def __init__(self, pkv, dev, pages, B, max_pages, P, seed=0, free=None):
        rng = np.random.default_rng(seed)
        self.pkv, self.dev, self.pages, self.P = pkv, dev, pages, P
        self.free = rng.permutation(pages).tolist() if free is None else list(free)
        self.pool = pkv.page_pool(pages, dev, self.free)
        self.table = np.full((B, max_pages), -1, np.int32)
        self.table_d = _i32(self.table, dev)
        self.lens = np.zeros(B, np.int32)

    def step(self, new, rows, err=0, in_place=False, positions=True):
        e = torch.zeros(1, dtype=torch.int32, device=self.dev)
        past = _i32(self.lens, self.dev)
        B = len(self.lens)
        lens = past if in_place else torch.full((B,), -9, dtype=torch.int32, device=self.dev)
        cu = torch.full((B + 1,), -9, dtype=torch.int32, device=self.dev)
        slots = torch.full((rows,), -9, dtype=torch.int64, device=self.dev)
        pos = torch.full((rows,), -9, dtype=torch.int32, device=self.dev) if positions else None
        self.pkv.pkv_plan_pages(past, _i32(new, self.dev), self.table_d, self.pool, self.P, lens, cu, slots, pos, e)
        ref = fp8b_ref.plan(self.lens.tolist(), list(new), self.table, self.free, self.P, rows, self.pages)
        assert int(e.item()) == ref[4] == err
        for got, want in zip((lens, cu, slots, pos), ref):
            assert got is None or np.array_equal(got.cpu().numpy(), want)
        self.lens = ref[0]
        self.check()
        return slots, cu, lens

    def release(self, keep=None, err=0, lens=None):
        e = torch.zeros(1, dtype=torch.int32, device=self.dev)
        lens = self.lens if lens is None else np.asarray(lens, np.int32)
        self.pkv.release_pages(_i32(lens, self.dev), self.table_d, self.pool, self.P,
                               None if keep is None else _i32(keep, self.dev), e)
        got = fp8b_ref.release(lens.tolist(), None if keep is None else list(keep), self.table, self.free, self.P,
                               self.pages)
        assert int(e.item()) == got == err
        if got in (0, 2):
            self.lens = np.zeros_like(self.lens) if keep is None else np.array(keep, np.int32)
        self.check()

    def check(self):
        pool = self.pool.cpu().numpy()
        assert pool[0] == len(self.free) and (pool[1:4] == 0).all()
        assert pool[4:4 + pool[0]].tolist() == self.free
        assert np.array_equal(self.table_d.cpu().numpy(), self.table)


@pytest.mark.parametrize("B,P,top", [(1, 16, 40), (3, 16, 1), (64, 16, 300), (300, 32, 90), (1021, 64, 50), (7, 256, 3000),
                                     (8192, 16, 20)])
def test_plan_steps(pkv, cuda_device, B, P, top):
    """Prompts, then single tokens, chunks and idle sequences, a rollback, and
    everything given back."""
    rng = np.random.default_rng(B)
    max_pages = (3 * top + 20) // P + 2
    p = Plan(pkv, cuda_device, B * max_pages + 5, B, max_pages, P, seed=B)
    before = list(p.free)
    first = rng.integers(0, top + 1, B)
    p.step(first, int(first.sum()) + 9)
    for i in range(3):
        new = np.ones(B, int) if i == 0 else rng.integers(0, 3, B) * rng.integers(0, top // 3 + 2, B)
        new = np.minimum(new, max_pages * P - p.lens)
        p.step(new, int(new.sum()) + (0 if i else 3), in_place=i == 1, positions=i != 2)
    p.release(np.maximum(p.lens - rng.integers(0, 9, B), 0))
    p.release()
    assert sorted(p.free) == sorted(before)


def test_release_restores_the_list(pkv, cuda_device):
    p = Plan(pkv, cuda_device, 500, 20, 20, 16)
    before = list(p.free)
    p.step([17 * i % 200 for i in range(20)], 4000)
    p.release()
    assert p.free == before


def test_many_rows(pkv, cuda_device):
    """More rows than the grid has threads."""
    p = Plan(pkv, cuda_device, 9000, 5, 4096, 64)
    p.step([100000, 1, 0, 250000, 77777], 450000)
    p.release()


def test_all_or_nothing(pkv, cuda_device):
    """What cannot be planned or released changes nothing."""
    p = Plan(pkv, cuda_device, 10, 3, 8, 16)
    p.step([40, 30, 0], 80)
    p.step([60, 40, 60], 200, err=pkv.DEVERR_POOL)
    p.step([1, 1, 1], 2, err=pkv.DEVERR_SEQLEN)                  # more tokens than rows
    p.step([1, -1, 1], 20, err=pkv.DEVERR_SEQLEN)
    p.step([1, 99, 1], 300, err=pkv.DEVERR_SEQLEN)               # beyond the table's row
    p.step([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], 16, err=pkv.DEVERR_SEQLEN)
    p.lens[1] = -4
    p.step([1, 1, 1], 20, err=pkv.DEVERR_SEQLEN, in_place=True)
    p.lens[1] = 30
    p.release([41, 0, 0], err=pkv.DEVERR_SEQLEN)
    p.release([-1, 0, 0], err=pkv.DEVERR_SEQLEN)
    p.release(lens=[40, 129, 0], err=pkv.DEVERR_SEQLEN)
    p.release(lens=[128, 128, 0], err=pkv.DEVERR_POOL)           # more than were taken
    p.step([1, 0, 17], 40)
    p.release()


def test_a_free_count_that_cannot_be(pkv, cuda_device):
    for count in (-1, 11, 2 ** 31 - 1, -2 ** 31):
        p = Plan(pkv, cuda_device, 10, 2, 4, 16)
        p.pool[0] = count
        keep = p.pool.clone()
        e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        lens, cu, slots, _ = pkv.plan_pages(_i32([3, 0], cuda_device), _i32([1, 20], cuda_device), p.table_d, p.pool, 16, 30,
                                            device_error=e)
        assert int(e.item()) == pkv.DEVERR_POOL and lens.tolist() == [3, 0] and not cu.any() and (slots == -1).all()
        pkv.release_pages(_i32([3, 0], cuda_device), p.table_d, p.pool, 16, device_error=e)
        assert torch.equal(p.pool, keep) and (p.table_d == -1).all()


def test_pages_outside_the_pool(pkv, cuda_device):
    """A bad page of the list or the table is flagged; its tokens get no slot."""
    p = Plan(pkv, cuda_device, 10, 2, 4, 16, free=[3, 10, -2, 7])
    p.step([20, 0], 24, err=pkv.DEVERR_PAGE)
    p.step([0, 5], 8, err=pkv.DEVERR_PAGE)
    p.release([0, 0], err=pkv.DEVERR_PAGE)
    p = Plan(pkv, cuda_device, 10, 1, 4, 16)
    p.step([20], 20)
    p.table[0, 1] = 99
    p.table_d[0, 1] = 99
    p.step([3], 3, err=pkv.DEVERR_PAGE)


def test_empty_calls(pkv, cuda_device):
    p = Plan(pkv, cuda_device, 4, 2, 2, 16)
    p.step([0, 0], 0)
    p.step([0, 0], 5)
    e = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    none = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    lens, cu, slots, pos = pkv.plan_pages(none, none, torch.zeros((0, 3), dtype=torch.int32, device=cuda_device), p.pool, 16, 4,
                                          device_error=e)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 4 and pos.tolist() == [0] * 4 and int(e.item()) == 0
    pkv.release_pages(none, torch.zeros((0, 3), dtype=torch.int32, device=cuda_device), p.pool, 16)
    p.check()


@pytest.mark.parametrize("B,rows", [(5, 8), (700, 3000)])
def test_captured_steps(pkv, cuda_device, B, rows):
    """One captured decode step, replayed: lengths advance in place, pages and
    slots follow, on one CTA and on many."""
    P, steps = 16, 40
    p = Plan(pkv, cuda_device, 3 * B, B, 3, P)
    lens, new = _i32(np.zeros(B), cuda_device), _i32(np.ones(B), cuda_device)
    cu, slots = torch.empty(B + 1, dtype=torch.int32, device=cuda_device), torch.empty(rows, dtype=torch.int64, device=cuda_device)
    pos, e = torch.empty(rows, dtype=torch.int32, device=cuda_device), torch.zeros(1, dtype=torch.int32, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.plan_pages(lens, new, p.table_d, p.pool, P, seq_lens=lens, cu_q=cu, slot_mapping=slots, positions=pos, device_error=e)
    for _ in range(steps):
        g.replay()
        ref = fp8b_ref.plan(p.lens.tolist(), [1] * B, p.table, p.free, P, rows, p.pages)
        p.lens = ref[0]
        for got, want in zip((lens, cu, slots, pos), ref):
            assert np.array_equal(got.cpu().numpy(), want)
        p.check()
    assert int(e.item()) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.release_pages(lens, p.table_d, p.pool, P, stream=side)
    side.synchronize()
    fp8b_ref.release(p.lens.tolist(), None, p.table, p.free, P, p.pages)
    p.check()
