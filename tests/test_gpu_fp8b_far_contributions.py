"""Decode where the largest weight and the largest contribution are far apart: tokens of a score
so much lower that their weight alone is below fp32's range meet values so much larger that
they make the output."""
import numpy as np
import pytest
import torch

from tests import fp4_ref, fp8b_ref
from tests.test_gpu_fp8b_attention import SM, _check, _dev, _tight_decode

pytestmark = pytest.mark.gpu


class _Two:
    """One sequence of one kv head whose tokens lie one behind another in the pool; every second run of
    `run` tokens has scores lower by about 2 a |g|^2 sm and values larger by 2^(up - down)."""

    def __init__(self, L, run, a, down, up, hq, dev):
        rng = np.random.default_rng(L + run)
        far = (np.arange(L) // run % 2 == 1)
        g = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(rng.choice([-1.0, 1.0], 128)))
        k = np.where(far[:, None, None], -a, a) * g * (1 + 0.01 * rng.standard_normal((L, 1, 1)))
        v = rng.standard_normal((L, 1, 128)) * np.exp2(np.where(far, up, down))[:, None, None]
        pages = (L + 15) // 16
        slots = np.arange(L, dtype=np.int64)
        cache = [np.zeros((pages, 1, 16, 128), np.uint8) for _ in range(2)]
        exps = [np.zeros((pages, 1, 1), np.uint8) for _ in range(2)]
        for i, x in enumerate((k, v)):
            fp8b_ref.append(cache[i], exps[i], x.astype(np.float32), slots)
        self.lens = [L]
        self.k, self.v = ([fp8b_ref.read(cache[i], exps[i], slots)] for i in range(2))
        self.scale = [np.exp2(exps[1][slots // 16, :, 0].astype(np.float64) - 127)]
        self.args = [_dev(x, dev) for x in (*cache, *exps)]
        self.table = torch.arange(pages, dtype=torch.int32, device=dev)[None]
        self.lensd = torch.tensor([L], dtype=torch.int32, device=dev)
        self.q = np.repeat(g[None], hq, 0) * np.exp2(-np.arange(hq) % 2)[:, None]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_ctas", [0, 1, 5])
@pytest.mark.parametrize("L,run", [(32, 16), (64, 32), (700, 32), (1500, 16), (3000, 1504)])
@pytest.mark.parametrize("a,down,up", [(6.0, -100, 100), (5.0, -90, 75), (2.0, -20, 40), (6.0, -110, 90), (6.0, 0, 20)])
def test_decode(pkv, cuda_device, L, run, a, down, up, max_ctas, out_dtype):
    c = _Two(L, run, a, down, up, 4, cuda_device)
    got = pkv.paged_gqa_decode_fp8b(_dev(c.q[None], cuda_device).to(torch.bfloat16), *c.args, c.table, c.lensd, max_seq_len=L,
                                    max_ctas=max_ctas, out_dtype=out_dtype)
    ref = fp4_ref.attend(c.q, c.k[0], c.v[0], L - 1, 0, 0, SM)
    tol = _tight_decode(c, 0, c.q, L - 1, 0, 0, SM)
    if out_dtype == torch.bfloat16:
        # the weights' one part (2^-11 of sum w |v|), chains of 1024 additions (2^-13), what is lost below
        # 2^-26 of the largest contribution instead of 2^-37, and half a step of the output
        s = np.einsum("hd,thd->ht", c.q, np.repeat(c.k[0], 4, 1)) * SM
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        A = np.einsum("ht,td->hd", w, np.abs(c.v[0][:, 0]))
        top = (w * c.scale[0][:, 0]).max(1)[:, None]
        tol = tol + (2.0 ** -11 + 2.0 ** -13) * A + 2.0 ** -26 * top * (np.abs(c.v[0][:, 0]) / c.scale[0]).sum(0) + 2.0 ** -8 * np.abs(ref)
    _check(got[0], ref, tol, (L, run, a, down, up))
