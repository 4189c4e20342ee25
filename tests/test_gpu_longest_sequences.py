"""Sequences near the largest 32-bit length, of which a window shows the end:
decode takes all that a block table can name, prefill those whose length
rounded up to whole key tiles still fits 32 bits."""
import numpy as np
import pytest
import torch

from tests import fp4_ref

pytestmark = pytest.mark.gpu

TABLE = (1 << 27) - 1                                            # pages of 16 tokens: 2^31 - 16 tokens
LONGEST = 2 ** 31 - 128


@pytest.fixture(scope="module")
def table(cuda_device):
    t = torch.zeros(1, TABLE, dtype=torch.int32, device=cuda_device)
    t[0, -24:] = torch.arange(1, 25, dtype=torch.int32, device=cuda_device)
    yield t


class Far:
    """24 pages of 16 tokens, the last ones of the table; page 0, all its other
    entries, holds zeros.  Token i of the 384 sits at 2^31 - 16 - 384 + i."""

    def __init__(self, pkv, dev):
        g = torch.Generator(device=dev).manual_seed(9)
        self.pkv, self.dev = pkv, dev
        k, v = (torch.randn(384, 1, 128, device=dev, generator=g) for _ in range(2))
        self.q = torch.randn(3, 4, 128, device=dev, generator=g).bfloat16()
        self.s = torch.full((1,), 0.01, device=dev)
        self.kc, self.vc = (pkv.fp4_cache(25, 1, 16, dev) for _ in range(2))
        slots = torch.arange(16, 400, device=dev)
        pkv.kv_append_fp4(k, v, slots, self.s, self.s, self.kc, self.vc)
        self.back = [x.double().cpu().numpy() for x in pkv.kv_read_fp4(slots, self.s, self.s, self.kc, self.vc,
                                                                         out_dtype=torch.float32)]
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)

    def lens(self, L):
        return torch.tensor([L], dtype=torch.int32, device=self.dev)

    def flags(self):
        torch.cuda.synchronize()
        e = int(self.err.item())
        self.err.zero_()
        return e

    def check(self, got, q, position, bf16=False):
        q, at = q.double().cpu().numpy(), position - (2 ** 31 - 16 - 384)
        ref = fp4_ref.attend(q, *self.back, at, 64, 0, fp4_ref.SM)
        tol = fp4_ref.attention_tolerance(q, *self.back, ref, fp4_ref.SM, bf16)
        assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("max_ctas", [0, 1])
def test_decode(pkv, cuda_device, table, max_ctas):
    f = Far(pkv, cuda_device)

    def run(L):
        return pkv.paged_gqa_decode_fp4(f.q[:1], f.kc, f.vc, f.s, f.s, table, f.lens(L), out_dtype=torch.float32,
                                        max_seq_len=2 ** 31 - 1, window=64, device_error=f.err, max_ctas=max_ctas)

    for L in (2 ** 31 - 300, LONGEST, 2 ** 31 - 17, 2 ** 31 - 16):
        got = run(L)
        assert f.flags() == 0
        f.check(got[0], f.q[0], L - 1)
    for L in (2 ** 31 - 15, 2 ** 31 - 1):                        # beyond the table: clamped and flagged
        assert torch.equal(run(L), got)
        assert f.flags() == pkv.DEVERR_SEQLEN


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill(pkv, cuda_device, table, out_dtype):
    f = Far(pkv, cuda_device)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=cuda_device)

    def run(L):
        out = torch.full(f.q.shape, 9.0, dtype=out_dtype, device=cuda_device)
        return pkv.paged_prefill_fp4(f.q, cu, f.kc, f.vc, f.s, f.s, table, f.lens(L), 3, out=out,
                                     max_kv_len=2 ** 31 - 1, window=64, device_error=f.err)

    for L in (2 ** 31 - 300, LONGEST):
        got = run(L)
        assert f.flags() == 0
        for i in range(3):
            f.check(got[i], f.q[i], L - 3 + i, out_dtype == torch.bfloat16)
    for L in (LONGEST + 1, 2 ** 31 - 16, 2 ** 31 - 1):           # not written, flagged
        assert (run(L) == 9).all()
        assert f.flags() == pkv.DEVERR_SEQLEN


def test_fp8_prefill(pkv, cuda_device, table):
    """Copies of such sequences never fit a workspace: not written, flagged."""
    f = Far(pkv, cuda_device)
    kc, vc = (torch.zeros(25, 1, 16, 128, dtype=torch.uint8, device=cuda_device) for _ in range(2))
    cu = torch.tensor([0, 3], dtype=torch.int32, device=cuda_device)
    for L in (LONGEST, LONGEST + 1, 2 ** 31 - 16):
        out = torch.full(f.q.shape, 9.0, dtype=torch.float32, device=cuda_device)
        pkv.paged_prefill(f.q, cu, kc, vc, f.s, f.s, table, f.lens(L), 3, out=out, max_kv_len=2 ** 31 - 1,
                          max_total_kv=1000, device_error=f.err)
        assert f.flags() == pkv.DEVERR_SEQLEN
        assert (out == 9).all()
