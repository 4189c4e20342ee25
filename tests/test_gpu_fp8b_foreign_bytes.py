"""Appending to blocks whose byte no append of this library has written: the formulas hold
for every byte that is a scale."""
import numpy as np
import pytest
import torch

from tests import fp8b_ref
from tests.test_gpu_fp8b_rows import DTYPES, Pools, _two

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-38, 1e-4, 1.0, 1e10, 3e36, 1e38])
@pytest.mark.parametrize("first,count", [(1, 1), (5, 3), (1, 15)])
def test_append_to_blocks_of_any_byte(pkv, cuda_device, dtype, size, first, count):
    """Rows first .. first + count - 1 of blocks with the bytes 0 .. 254, a block a page."""
    rng = np.random.default_rng(first + count)
    p = Pools(rng, 255, 2, 16, cuda_device, pkv)
    for i in range(2):
        p.exps[i][:] = np.arange(255, dtype=np.uint8)[:, None, None]
        p.exps_d[i].copy_(torch.from_numpy(p.exps[i]))
    slots = (np.arange(255)[:, None] * 16 + first + np.arange(count)).reshape(-1).astype(np.int64)
    with np.errstate(over="ignore"):
        rows = [np.clip(x * np.float32(size), -3.3e38, 3.3e38).astype(np.float32) for x in _two(rng, len(slots), 2)]
    p.append(rows, slots, DTYPES[dtype])


def test_new_rows_of_a_large_byte_read_back(pkv, cuda_device):
    """Beside a block's byte of 250 new rows are as large as they were, to half a step of it."""
    rng = np.random.default_rng(1)
    p = Pools(rng, 3, 2, 16, cuda_device, pkv)
    for x in p.exps_d:
        x.fill_(250)
    slots = np.array([3, 20, 36], np.int64)
    x = torch.from_numpy(rng.choice([-1.0, 1.0], (3, 2, 128)) * np.exp2(rng.uniform(118, 126, (3, 2, 128)))).float().to(cuda_device)
    sd = torch.from_numpy(slots).to(cuda_device)
    pkv.kv_append_fp8b(x, -x, sd, *p.args())
    k, v = pkv.kv_read_fp8b(sd, *p.args(), out_dtype=torch.float32)
    # half a step of 2^-3, or of the smallest one, 2^-9 2^(250 - 127)
    tol = 2.0 ** -4 * x.abs().double() + 2.0 ** -10 * 2.0 ** 123
    assert ((k.double() - x).abs() <= tol).all() and ((v.double() + x).abs() <= tol).all()
    assert all((e[pg] == 250).all() for e in p.exps_d for pg in range(3))
