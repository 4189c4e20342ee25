"""Long 4-bit caches made and attended on the GPU in 64 bits, a piece at a
time, for the accuracy tests."""
import torch


class LongCache:
    """One sequence of L tokens in pages of 64 in order; make(t0, t1) gives K
    and V rows fp32 [t1 - t0, hkv, 128] of its tokens."""

    def __init__(self, pkv, L, hkv, dev, make, k_scale=2.0 ** -6, v_scale=None):
        self.pkv, self.L, self.hkv, self.dev = pkv, L, hkv, dev
        pages = (L + 63) // 64
        self.kc, self.vc = (pkv.fp4_cache(pages, hkv, 64, dev) for _ in range(2))
        self.ks = torch.full((hkv,), k_scale, device=dev)
        self.vs = torch.full((hkv,), 2.0 ** -6, device=dev) if v_scale is None else v_scale
        for t0 in range(0, L, 65536):
            t1 = min(L, t0 + 65536)
            pkv.kv_append_fp4(*make(t0, t1), torch.arange(t0, t1, device=dev), self.ks, self.vs, self.kc, self.vc)
        self.table = torch.arange(pages, device=dev, dtype=torch.int32)[None]
        self.lens = torch.tensor([L], device=dev, dtype=torch.int32)

    def pieces(self):
        """K and V as the cache holds them, fp64, 65536 tokens at a time."""
        unit = torch.ones(self.hkv, device=self.dev)              # e s is exact in fp32, and so are products in 64 bits
        for t0 in range(0, self.L, 65536):
            slots = torch.arange(t0, min(self.L, t0 + 65536), device=self.dev)
            k, v = self.pkv.kv_read_fp4(slots, unit, unit, self.kc, self.vc, out_dtype=torch.float32)
            yield t0, k.double() * self.ks.double()[:, None], v.double() * self.vs.double()[:, None]

    def attend(self, q, sm, positions=None):
        """Queries [N, hq, 128] at their positions (the last one, if none are
        given): (out, sum w |v|), both [N, hq, 128] in 64 bits."""
        N, hq, _ = q.shape
        g, q = hq // self.hkv, q.double()
        p = torch.full((N,), self.L - 1, device=self.dev) if positions is None else positions
        m = torch.full((N, hq), -float("inf"), dtype=torch.float64, device=self.dev)
        l, o, a = torch.zeros_like(m), torch.zeros_like(q), torch.zeros_like(q)
        for t0, k, v in self.pieces():
            k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
            s = torch.einsum("nhd,thd->nht", q, k) * sm
            s.masked_fill_((t0 + torch.arange(k.shape[0], device=self.dev) > p[:, None])[:, None], -float("inf"))
            top = torch.maximum(m, s.amax(2))
            w, f = (s - top[..., None]).exp(), (m - top).exp()
            l, m = l * f + w.sum(2), top
            o = o * f[..., None] + torch.einsum("nht,thd->nhd", w, v)
            a = a * f[..., None] + torch.einsum("nht,thd->nhd", w, v.abs())
        return o / l[..., None], a / l[..., None]

    def decode(self, q, sm, **kw):
        return self.pkv.paged_gqa_decode_fp4(q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, sm_scale=sm,
                                             max_seq_len=self.L, **kw)

    def prefill(self, q, sm, **kw):
        cu = torch.tensor([0, q.shape[0]], device=self.dev, dtype=torch.int32)
        return self.pkv.paged_prefill_fp4(q, cu, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, q.shape[0],
                                          max_kv_len=self.L, sm_scale=sm, **kw)
