"""Decode and prefill attention over the 4-bit cache against the 64-bit form."""
import numpy as np
import pytest
import torch

from tests import fp4_ref

pytestmark = pytest.mark.gpu


def _dev(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


class Cache:
    """K and V of a batch in shuffled pages; rows nobody wrote hold NaN scales
    and the table's spare entries point outside the pool."""

    def __init__(self, seed, lens, hkv, P, dev, page_sizes=None, spread=1.0, hidden=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.hkv, self.P, self.dev = rng, list(lens), hkv, P, dev
        sizes = page_sizes or [P] * len(lens)
        self.page_sizes = page_sizes
        runs = [[sizes[b] // P] * ((L + sizes[b] - 1) // sizes[b]) for b, L in enumerate(lens)]
        order = [(b, i) for b, r in enumerate(runs) for i in range(len(r))]
        rng.shuffle(order)
        self.max_pages = max(1, max((len(r) for r in runs), default=1)) + 1
        self.table = np.full((len(lens), self.max_pages), -5, np.int32)
        at = 1
        for b, i in order:
            self.table[b, i] = at
            at += runs[b][i]
        self.pages = at + 1
        self.k, self.v = [], []
        pools = [np.full((self.pages, hkv, P, 72), 0xFF, np.uint8) for _ in range(2)]
        self.ks, self.vs = (rng.uniform(0.02, 0.06, hkv).astype(np.float32) for _ in range(2))
        for b, L in enumerate(lens):
            slots = fp4_ref.slots_of(self.table[b], L, P, sizes[b])
            for pool, s, keep in ((pools[0], self.ks, self.k), (pools[1], self.vs, self.v)):
                fp4_ref.write(pool, *fp4_ref.quantise(fp4_ref.rows(rng, L, hkv, spread), s), slots)
                keep.append(fp4_ref.block_values(pool, slots) * s.astype(np.float64).reshape(1, hkv, 1))
        self.kc, self.vc = (_dev(p, dev) for p in pools)
        self.ksd, self.vsd, self.lensd = _dev(self.ks, dev), _dev(self.vs, dev), _dev(np.array(lens, np.int32), dev)
        self.psd = None if page_sizes is None else _dev(np.array(page_sizes, np.int32), dev)
        if hidden:                                               # (window, sinks, first query's position of b)
            window, sinks, pos = hidden
            for b in range(len(lens)):
                for i in range(self.max_pages):
                    t = np.arange(i * sizes[b], min((i + 1) * sizes[b], lens[b]))
                    if not ((t > pos[b] - window) | (t < sinks)).any():
                        self.table[b, i] = 1 << 30
        self.tabled = _dev(self.table, dev)

    def queries(self, rows, hq, spread=1.0):
        q = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(self.rng.standard_normal((rows, hq, 128)) * spread))
        return q, _dev(q, self.dev).to(torch.bfloat16)


def _check(got, ref, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, float(np.abs(got - ref).max()), int(bad.sum()), np.argwhere(bad)[:3].tolist())


def _decode(pkv, c, q, qd, window=0, sinks=0, out_dtype=torch.float32, err=0, sm=fp4_ref.SM, **kw):
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    out = torch.full(qd.shape, 9.0, dtype=out_dtype, device=c.dev)
    got = pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out=out, sm_scale=sm,
                                   device_error=e, window=window, sinks=sinks,
                                   max_seq_len=max(max(c.lens), 1), seq_page_sizes=c.psd, **kw)
    torch.cuda.synchronize()
    assert int(e.item()) == err
    for b, L in enumerate(c.lens):
        ref = fp4_ref.attend(q[b].astype(np.float64), c.k[b], c.v[b], L - 1, window, sinks, sm)
        _check(got[b], ref, fp4_ref.attention_tolerance(q[b], c.k[b], c.v[b], ref, sm, out_dtype == torch.bfloat16),
               ("decode", b, L, window, sinks))
    return got


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 64, 100, 257, 511, 700]


@pytest.mark.parametrize("hkv,G,P", [(1, 8, 16), (2, 4, 32), (3, 1, 64), (8, 2, 16), (2, 7, 128), (1, 3, 256),
                                     (5, 5, 16), (2, 6, 16)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode_all_lengths(pkv, cuda_device, hkv, G, P, out_dtype):
    c = Cache(hkv * 100 + G, LENS, hkv, P, cuda_device)
    q, qd = c.queries(len(LENS), hkv * G)
    _decode(pkv, c, q, qd, out_dtype=out_dtype)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (15, 3), (16, 0), (16, 16), (17, 20), (33, 4),
                                          (100, 40), (400, 1), (700, 5), (5000, 4), (40, 2000)])
def test_decode_window(pkv, cuda_device, window, sinks):
    """Windows and sinks against every length; pages nobody sees have table
    entries outside the pool."""
    c = Cache(window * 13 + sinks, LENS, 2, 16, cuda_device, hidden=(window, sinks, [L - 1 for L in LENS]))
    q, qd = c.queries(len(LENS), 8)
    _decode(pkv, c, q, qd, window, sinks)
    _decode(pkv, c, q, qd, window, sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("max_ctas", [1, 3, 7, 40])
def test_decode_any_split(pkv, cuda_device, max_ctas):
    lens = [3000, 1, 0, 519, 2048]
    c = Cache(5, lens, 2, 16, cuda_device)
    q, qd = c.queries(len(lens), 12)
    _decode(pkv, c, q, qd, max_ctas=max_ctas)
    _decode(pkv, c, q, qd, 700, 9, max_ctas=max_ctas)


def test_decode_long_chain(pkv, cuda_device):
    """One worker over a long sequence: its accumulator is folded."""
    c = Cache(6, [20000], 1, 64, cuda_device)
    q, qd = c.queries(1, 8)
    _decode(pkv, c, q, qd, max_ctas=1)
    _decode(pkv, c, q, qd)


@pytest.mark.parametrize("max_ctas", [0, 5, 23])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode_one_long_sequence(pkv, cuda_device, max_ctas, out_dtype):
    """A segment over many CTAs' ranges, beside short and empty ones."""
    c = Cache(29, [40, 6000, 0, 7], 2, 16, cuda_device)
    q, qd = c.queries(4, 14)
    a = _decode(pkv, c, q, qd, out_dtype=out_dtype, max_ctas=max_ctas)
    assert torch.equal(_decode(pkv, c, q, qd, out_dtype=out_dtype, max_ctas=max_ctas), a)
    _decode(pkv, c, q, qd, 5000, 100, out_dtype=out_dtype, max_ctas=max_ctas)


@pytest.mark.parametrize("max_ctas", [0, 3])
@pytest.mark.parametrize("B,G,window,sinks", [(300, 8, 0, 0), (700, 3, 0, 0), (300, 7, 50, 3)])
def test_decode_many_short_sequences(pkv, cuda_device, B, G, window, sinks, max_ctas):
    """Many more (sequence, head) rows than warps, most of them whole, some cut."""
    rng = np.random.default_rng(B)
    c = Cache(31, [int(x) for x in rng.choice([0, 1, 20, 64, 90, 250], B)], 2, 16, cuda_device)
    q, qd = c.queries(B, 2 * G)
    a = _decode(pkv, c, q, qd, window, sinks, max_ctas=max_ctas)
    assert torch.equal(_decode(pkv, c, q, qd, window, sinks, max_ctas=max_ctas), a)


@pytest.mark.parametrize("spread", [30.0, 1e-4, 1e4])
def test_decode_large_and_small_scores(pkv, cuda_device, spread):
    """Scores from almost equal to one that takes all the weight, rising and
    falling along the sequence."""
    c = Cache(7, [1, 40, 333, 1500], 2, 16, cuda_device)
    q, qd = c.queries(4, 8, spread)
    _decode(pkv, c, q, qd, sm=fp4_ref.SM / max(1.0, spread / 30))
    _decode(pkv, c, q, qd, 100, 4, sm=fp4_ref.SM / max(1.0, spread / 30))
    _decode(pkv, c, q, qd, sm=-fp4_ref.SM / max(1.0, spread / 30))


def test_decode_page_sizes_per_sequence(pkv, cuda_device):
    lens = [700, 33, 1, 256, 90]
    c = Cache(8, lens, 2, 16, cuda_device, page_sizes=[64, 16, 256, 128, 32])
    q, qd = c.queries(5, 8)
    _decode(pkv, c, q, qd)
    _decode(pkv, c, q, qd, 50, 3)
    c.psd[1] = 24
    got = _call_flagged(pkv, c, qd, pkv.DEVERR_PAGESIZE)
    assert (got[1] == 0).all()


def _call_flagged(pkv, c, qd, bit, **kw):
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    got = pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out_dtype=torch.float32,
                                   device_error=e, seq_page_sizes=c.psd, **{"max_seq_len": max(c.lens), **kw})
    torch.cuda.synchronize()
    assert int(e.item()) == bit
    return got


def test_decode_bad_pages_and_lengths(pkv, cuda_device):
    """A page outside the pool reads as zeros (score 0, value 0); lengths are
    clamped; both are flagged."""
    c = Cache(9, [100, 64], 2, 16, cuda_device)
    q, qd = c.queries(2, 8)
    c.tabled[0, 2] = c.pages
    c.k[0][32:48] = 0
    c.v[0][32:48] = 0
    _decode(pkv, c, q, qd, err=pkv.DEVERR_PAGE)
    _decode(pkv, c, q, qd, 20, 4)                                # not seen there: not looked at
    c.tabled[0, 2] = -1
    _decode(pkv, c, q, qd, err=pkv.DEVERR_PAGE)
    c.tabled[0, 2] = 3
    c.lensd[1] = -3
    got = _call_flagged(pkv, c, qd, pkv.DEVERR_SEQLEN)
    assert (got[1] == 0).all()
    c.lensd[1] = 64
    full = _call_flagged(pkv, c, qd, 0)
    c.lensd[1] = 2 ** 31 - 1
    # clamped to 100 tokens, of which the table has pages for 64: the others read as zeros
    got = _call_flagged(pkv, c, qd, pkv.DEVERR_SEQLEN | pkv.DEVERR_PAGE, max_seq_len=64 + 36)
    assert torch.equal(got[0], full[0])
    c.lensd[1] = 65
    got = _call_flagged(pkv, c, qd, pkv.DEVERR_SEQLEN, max_seq_len=64)
    assert torch.equal(got[1], full[1])


def test_decode_nan_rows(pkv, cuda_device):
    """A NaN block of V in sight is NaN in its 16 dims; out of sight it is not
    seen; a NaN in K takes the whole row."""
    c = Cache(10, [200], 1, 16, cuda_device)
    q, qd = c.queries(1, 4)
    base = _decode(pkv, c, q, qd, 50, 3)
    slot = fp4_ref.slots_of(c.table[0], 200, 16)
    pool = c.vc.view(c.pages, 1, 1, 1152)
    pg, r = divmod(int(slot[100]), 16)
    pool[pg, 0, 0, 1024 + 8 * r + 5] = 0x7F
    assert torch.equal(_call_flagged(pkv, c, qd, 0, window=50, sinks=3), base)
    got = _call_flagged(pkv, c, qd, 0)
    assert torch.isnan(got[..., 80:96]).all() and not torch.isnan(got[..., :80]).any()
    assert not torch.isnan(got[..., 96:]).any()
    c.kc.view(c.pages, 1, 1, 1152)[pg, 0, 0, 1024 + 8 * r] = 0xFF
    assert torch.isnan(_call_flagged(pkv, c, qd, 0)).all()


def test_decode_deterministic_in_graphs_and_streams(pkv, cuda_device):
    """Twice the same bits; captured calls with one workspace each; another
    stream; large batch of empty and short sequences."""
    lens = [0, 5, 900, 33, 0, 1] * 50
    c = Cache(11, lens, 1, 16, cuda_device)
    q, qd = c.queries(len(lens), 3)
    a = _decode(pkv, c, q, qd, 60, 2)
    assert torch.equal(_decode(pkv, c, q, qd, 60, 2), a)
    outs, graphs = [], []
    for w in (60, 0):
        out = torch.zeros_like(a)
        ws = torch.empty(pkv.pkv_decode_fp4_workspace_size(len(lens), 3, 1, max_seq_len=900), dtype=torch.uint8,
                         device=cuda_device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out=out, workspace=ws,
                                     max_seq_len=900, window=w, sinks=2)
        outs.append(out)
        graphs.append((g, ws))
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out_dtype=torch.float32,
                                   max_seq_len=900, stream=side)
    side.synchronize()
    assert torch.equal(got, outs[1])


def test_decode_workspace_needs_no_initialisation(pkv, cuda_device):
    lens = [4000, 17, 0]
    c = Cache(12, lens, 2, 16, cuda_device)
    q, qd = c.queries(3, 4)
    n = pkv.pkv_decode_fp4_workspace_size(3, 4, 2, max_seq_len=4000)
    a, b = (pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, out_dtype=torch.float32,
                                     max_seq_len=4000,
                                     workspace=torch.full((n,), v, dtype=torch.uint8, device=cuda_device))
            for v in (0, 0xFF))
    assert torch.equal(a, b) and not torch.isnan(a).any()
    with pytest.raises(pkv.PkvError):
        pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, max_seq_len=4000,
                                 workspace=torch.empty(max(n - 256, 0), dtype=torch.uint8, device=cuda_device))


# ---------------------------------------------------------------- prefill
def _prefill(pkv, c, ns, hq, window=0, sinks=0, out_dtype=torch.float32, q_spread=1.0, sm=fp4_ref.SM, sample=40,
             total=0, err=0, pad_rows=3, skip=()):
    cu = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    q, qd = c.queries(int(cu[-1]) + pad_rows, hq, q_spread)
    out = torch.full(qd.shape, 9.0, dtype=out_dtype, device=c.dev)
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    pkv.paged_prefill_fp4(qd, _dev(cu, c.dev), c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, max(max(ns), 1), out=out,
                          max_kv_len=max(max(c.lens), 1), sm_scale=sm, device_error=e, window=window, sinks=sinks,
                          max_total_kv=total, seq_page_sizes=c.psd)
    torch.cuda.synchronize()
    assert int(e.item()) == err
    assert (out[int(cu[-1]):] == 9).all()                        # rows behind the last chunk
    bf16 = out_dtype == torch.bfloat16
    for b, (L, n) in enumerate(zip(c.lens, ns)):
        if b in skip:
            assert (out[int(cu[b]):int(cu[b + 1])] == 9).all()
            continue
        rows = np.arange(n) if n <= sample else np.unique(
            np.concatenate(([0, 1, n - 2, n - 1], c.rng.integers(0, n, sample))))
        for r in rows:
            x = q[cu[b] + r].astype(np.float64)
            p = L - n + int(r)
            ref = fp4_ref.attend(x, c.k[b], c.v[b], p, window, sinks, sm)
            _check(out[cu[b] + r], ref, fp4_ref.attention_tolerance(x, c.k[b][:p + 1], c.v[b][:p + 1], ref, sm, bf16),
                   ("prefill", b, L, n, int(r), window, sinks))
    return qd, out


@pytest.mark.parametrize("hkv,G,P", [(1, 8, 16), (2, 4, 32), (3, 1, 64), (2, 7, 128), (1, 3, 256), (2, 5, 16),
                                     (1, 6, 16), (8, 2, 16)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_ragged(pkv, cuda_device, hkv, G, P, out_dtype):
    """Chunks of no, one and many queries; whole sequences; odd lengths."""
    lens, ns = [1, 50, 300, 128, 17, 129, 0, 385], [1, 0, 45, 128, 17, 1, 0, 130]
    c = Cache(hkv * 10 + G, lens, hkv, P, cuda_device)
    _prefill(pkv, c, ns, hkv * G, out_dtype=out_dtype, sample=12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (16, 4), (100, 0), (128, 128), (129, 130),
                                          (300, 7), (600, 1), (5000, 4), (64, 600)])
def test_prefill_window(pkv, cuda_device, window, sinks):
    lens, ns = [700, 333, 900, 20, 256], [200, 1, 129, 20, 256]
    c = Cache(window + sinks, lens, 2, 16, cuda_device,
              hidden=(window, sinks, [L - n for L, n in zip(lens, ns)]))
    _prefill(pkv, c, ns, 6, window, sinks, sample=16)
    _prefill(pkv, c, ns, 6, window, sinks, out_dtype=torch.bfloat16, sample=10)


def test_prefill_long_context(pkv, cuda_device):
    """More key tiles than one accumulation segment; a window that skips most
    of them; the sum bound of the workspace."""
    lens, ns = [9000, 150], [260, 150]
    c = Cache(21, lens, 1, 64, cuda_device)
    _prefill(pkv, c, ns, 8, sample=10, total=9150)
    _prefill(pkv, c, ns, 8, 2000, 5, sample=10, total=9150)
    _prefill(pkv, c, ns, 8, 6000, 200, out_dtype=torch.bfloat16, sample=10)


@pytest.mark.parametrize("spread", [30.0, 1e-3])
def test_prefill_large_and_small_scores(pkv, cuda_device, spread):
    c = Cache(22, [900, 64], 2, 16, cuda_device)
    _prefill(pkv, c, [150, 64], 8, q_spread=spread, sample=20)
    _prefill(pkv, c, [150, 64], 8, 90, 2, q_spread=spread, sample=20)


def test_prefill_page_sizes_and_errors(pkv, cuda_device):
    lens, ns = [300, 90, 64], [100, 90, 10]
    c = Cache(23, lens, 2, 16, cuda_device, page_sizes=[64, 16, 256])
    _prefill(pkv, c, ns, 4, sample=10)
    _prefill(pkv, c, ns, 4, 40, 3, sample=10)
    c.psd[1] = 20
    _prefill(pkv, c, ns, 4, sample=10, err=pkv.DEVERR_PAGESIZE, skip=(1,))
    c.psd[1] = 16
    c.lensd[0] = 50                                              # shorter than its chunk
    _prefill(pkv, c, ns, 4, sample=10, err=pkv.DEVERR_SEQLEN, skip=(0,))
    c.lensd[0] = 300
    c.tabled[1, 2] = c.pages + 7
    c.k[1][32:48] = 0
    c.v[1][32:48] = 0
    _prefill(pkv, c, ns, 4, sample=10, err=pkv.DEVERR_PAGE)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,ns", [([400, 3], [200, 3]), ([9000], [300])])
def test_prefill_nan_rows(pkv, cuda_device, out_dtype, lens, ns):
    """A NaN block of V is NaN in its 16 dims of the queries that see it, one
    of K in their whole rows; the others' rows are as without it."""
    c = Cache(26, lens, 2, 16, cuda_device)
    cu = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    _, qd = c.queries(int(cu[-1]), 8)
    n, L = ns[0], lens[0]

    def run(window):
        out = torch.full(qd.shape, 9.0, dtype=out_dtype, device=c.dev)
        ws = torch.full((pkv.pkv_prefill_fp4_workspace_size(len(lens), 2, n, L, 0, window, 5),), 0xFF,
                        dtype=torch.uint8, device=c.dev)
        pkv.paged_prefill_fp4(qd, _dev(cu, c.dev), c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, n, out=out,
                              max_kv_len=L, window=window, sinks=5, workspace=ws)
        return out.float().cpu().numpy()

    clean = {w: run(w) for w in (0, 70)}
    slots = fp4_ref.slots_of(c.table[0], L, 16)
    v_at, k_at = L - n + 60, L - n + 150
    for pool, h, t, block in ((c.vc, 1, v_at, 3), (c.vc, 1, 2, 6), (c.kc, 0, k_at, 0)):
        pg, r = divmod(int(slots[t]), 16)
        pool.view(c.pages, 2, 1, 1152)[pg, h, 0, 1024 + 8 * r + block] = 0x7F
    p = L - n + np.arange(n)
    for w in (0, 70):
        exp = clean[w].copy()

        def sees(t):
            return np.flatnonzero((p >= t) & ((w == 0) | (t > p - w) | (t < 5)))

        exp[sees(v_at), 4:, 48:64] = np.nan
        exp[sees(2), 4:, 96:112] = np.nan
        exp[sees(k_at), :4] = np.nan
        assert np.array_equal(run(w), exp, equal_nan=True), w


def test_prefill_one_query_is_a_decode_step(pkv, cuda_device):
    lens = [1, 130, 77, 600]
    c = Cache(24, lens, 2, 16, cuda_device)
    for w, s in ((0, 0), (64, 3)):
        qd, out = _prefill(pkv, c, [1] * 4, 8, w, s, pad_rows=0)
        q = qd.float().cpu().numpy()
        _decode(pkv, c, q, qd, w, s)


def test_prefill_deterministic_and_captured(pkv, cuda_device):
    lens, ns = [500, 200], [200, 100]
    c = Cache(25, lens, 2, 16, cuda_device)
    qd, a = _prefill(pkv, c, ns, 8, 100, 5, sample=4, pad_rows=0)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device=cuda_device)
    n = pkv.pkv_prefill_fp4_workspace_size(2, 2, 200, 500, 0, 100, 5)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda_device)
    out = torch.zeros_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_prefill_fp4(qd, cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 200, out=out, max_kv_len=500,
                              workspace=ws, window=100, sinks=5)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)


# ---------------------------------------------------------------- a run of them
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 4)])
def test_a_prompt_and_its_answer(pkv, cuda_device, window, sinks):
    """Calibrate, write a prompt in two chunks with their attention, decode
    some steps, read the cache back: every output against the 64-bit form."""
    rng = np.random.default_rng(31)
    hkv, hq, P, total = 2, 8, 16, 150
    k, v = fp4_ref.rows(rng, total, hkv), fp4_ref.rows(rng, total, hkv)
    pages = 14
    table = rng.permutation(pages)[:10].astype(np.int32)
    slots = fp4_ref.slots_of(table, total, P)
    kd, vd, sd, bt = (_dev(x, cuda_device) for x in (k, v, slots, table.reshape(1, -1)))
    kmax, vmax, ks, vs = (torch.zeros(hkv, device=cuda_device) for _ in range(4))
    pkv.pkv_kv_calibrate(kd[:140], vd[:140], kmax, vmax, ks, vs)
    kc, vc = pkv.fp4_cache(pages, hkv, P), pkv.fp4_cache(pages, hkv, P)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ksn, vsn = ks.cpu().numpy(), vs.cpu().numpy()
    pools = [np.zeros((pages, hkv, P, 72), np.uint8) for _ in range(2)]
    for pool, x, s in ((pools[0], k, ksn), (pools[1], v, vsn)):
        fp4_ref.write(pool, *fp4_ref.quantise(x, s), slots)
    kv = [fp4_ref.block_values(p, slots) * s.astype(np.float64).reshape(1, hkv, 1)
          for p, s in ((pools[0], ksn), (pools[1], vsn))]

    def check(q, out, p):
        ref = fp4_ref.attend(q.astype(np.float64), *kv, p, window, sinks, fp4_ref.SM)
        _check(out, ref, fp4_ref.attention_tolerance(q, kv[0][:p + 1], kv[1][:p + 1], ref, fp4_ref.SM, True), p)

    for lo, hi in ((0, 90), (90, 140)):
        pkv.kv_append_fp4(kd[lo:hi], vd[lo:hi], sd[lo:hi], ks, vs, kc, vc, err)
        q = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(rng.standard_normal((hi - lo, hq, 128))))
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device=cuda_device)
        lens = torch.tensor([hi], dtype=torch.int32, device=cuda_device)
        out = pkv.paged_prefill_fp4(_dev(q, cuda_device).to(torch.bfloat16), cu, kc, vc, ks, vs, bt, lens, hi - lo,
                                    device_error=err, window=window, sinks=sinks)
        for r in (0, 1, 40, hi - lo - 1):
            check(q[r], out[r], lo + r)
    for t in range(140, total):
        pkv.kv_append_fp4(kd[t:t + 1], vd[t:t + 1], sd[t:t + 1], ks, vs, kc, vc, err)
        q = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(rng.standard_normal((1, hq, 128))))
        lens = torch.tensor([t + 1], dtype=torch.int32, device=cuda_device)
        out = pkv.paged_gqa_decode_fp4(_dev(q, cuda_device).to(torch.bfloat16), kc, vc, ks, vs, bt, lens,
                                       device_error=err, window=window, sinks=sinks)
        check(q[0], out[0], t)
    assert int(err.item()) == 0
    assert np.array_equal(kc.cpu().numpy(), pools[0]) and np.array_equal(vc.cpu().numpy(), pools[1])
    got, _ = pkv.kv_read_fp4(sd, ks, vs, kc, vc, out_dtype=torch.float32)
    exp = (fp4_ref.block_values(pools[0], slots) * ksn.reshape(1, hkv, 1)).astype(np.float32)
    assert np.array_equal(got.cpu().numpy(), exp)


@pytest.mark.parametrize("batch,max_ctas", [(8192, 0), (8192, 200), (5000, 1000)])
def test_decode_large_batches(pkv, cuda_device, batch, max_ctas):
    """Thousands of sequences, one of them long: the rows are those of the
    same sequences in small batches."""
    lens = [3, 0, 40, 17, 1, 90]
    c = Cache(27, lens + [3000], 1, 16, cuda_device)
    pick = np.arange(batch) % len(lens)
    pick[batch // 2] = len(lens)
    q, qd = c.queries(batch, 2)
    at = _dev(pick, cuda_device)
    table, lensd = c.tabled[at].contiguous(), c.lensd[at].contiguous()
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, table, lensd, out_dtype=torch.float32,
                                   max_seq_len=3000, max_ctas=max_ctas, device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for b in (*range(12), batch // 2 - 1, batch // 2, batch // 2 + 1, batch - 2, batch - 1):
        k, v, L = c.k[pick[b]], c.v[pick[b]], len(c.k[pick[b]])
        ref = fp4_ref.attend(q[b].astype(np.float64), k, v, L - 1, 0, 0, fp4_ref.SM)
        _check(out[b], ref, fp4_ref.attention_tolerance(q[b], k, v, ref, fp4_ref.SM, False), b)


def test_calls_at_once_on_two_streams(pkv, cuda_device):
    """Decode and prefill on two streams at the same time, with workspaces of
    their own, give the bits of the calls one after the other."""
    lens = [5000, 300, 2000]
    c = Cache(28, lens, 2, 16, cuda_device)
    _, qd = c.queries(3, 8)
    _, qp = c.queries(600, 8)
    cu = torch.tensor([0, 300, 400, 600], dtype=torch.int32, device=cuda_device)

    def decode(stream=None):
        return pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, max_seq_len=5000,
                                        out_dtype=torch.float32, stream=stream)

    def prefill(stream=None):
        return pkv.paged_prefill_fp4(qp, cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 300, max_kv_len=5000,
                                     window=1000, sinks=4, stream=stream)

    ref = decode(), prefill()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((decode(), prefill()))
    torch.cuda.synchronize()
    for d, p in got:
        assert torch.equal(d, ref[0]) and torch.equal(p, ref[1])


@pytest.mark.parametrize("as_int", [False, True])
def test_allocating_calls_on_another_stream(pkv, cuda_device, as_int):
    """What a call allocates belongs to the stream it runs on: work still ahead
    on the current stream does not write to it."""
    lens = [900, 33]
    c = Cache(30, lens, 2, 16, cuda_device)
    _, qd = c.queries(2, 8)
    _, qp = c.queries(60, 8)
    cu = torch.tensor([0, 40, 60], dtype=torch.int32, device=cuda_device)
    slots = _dev(fp4_ref.slots_of(c.table[0], 900, 16), cuda_device)
    slots[7] = -1
    calls = [lambda s: pkv.paged_gqa_decode_fp4(qd, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, stream=s,
                                                max_seq_len=900, max_ctas=3),
             lambda s: pkv.paged_prefill_fp4(qp, cu, c.kc, c.vc, c.ksd, c.vsd, c.tabled, c.lensd, 40, max_kv_len=900,
                                             stream=s),
             lambda s: pkv.kv_read_fp4(slots, c.ksd, c.vsd, c.kc, c.vc, stream=s)[0]]
    side = torch.cuda.Stream()
    for call in calls:
        ref = call(None)
        n = ref.numel() * ref.element_size()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)                            # some 10 ms of the current stream
        for size in (n, n, 1 << 20, 4 << 20, 16 << 20):
            torch.empty(size, dtype=torch.uint8, device=cuda_device).fill_(0x7F)
        got = call(side.cuda_stream if as_int else side)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [12.0, 20.0, 26.0, 27.5])
def test_many_small_weights(pkv, cuda_device, e, out_dtype):
    """One token takes almost all the weight; 128K others, 2^-e of it each,
    still count."""
    L, dev = 131072, cuda_device
    k, v = torch.zeros(L, 1, 128, device=dev), torch.ones(L, 1, 128, device=dev)
    k[0, :, 0] = 6
    v[0] = 0
    s = torch.full((1,), 2.0 ** -6, device=dev)
    kc, vc = pkv.fp4_cache(L // 16, 1, 16), pkv.fp4_cache(L // 16, 1, 16)
    slots = torch.arange(L, device=dev)
    pkv.kv_append_fp4(k, v, slots, s, s, kc, vc)
    kr, vr = (x.double().cpu().numpy() for x in pkv.kv_read_fp4(slots, s, s, kc, vc, out_dtype=torch.float32))
    q = torch.zeros(2, 4, 128, device=dev, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    sm = float(np.float32(e * np.log(2) / kr[0, 0, 0]))
    bt = torch.arange(L // 16, device=dev, dtype=torch.int32)[None]
    ln = torch.tensor([L], device=dev, dtype=torch.int32)
    cu = torch.tensor([0, 2], device=dev, dtype=torch.int32)
    x = q[0].double().cpu().numpy()
    ref = fp4_ref.attend(x, kr, vr, L - 1, 0, 0, sm)
    tol = fp4_ref.attention_tolerance(x, kr, vr, ref, sm, out_dtype == torch.bfloat16)
    got = pkv.paged_gqa_decode_fp4(q[1:], kc, vc, s, s, bt, ln, out_dtype=out_dtype, sm_scale=sm, max_seq_len=L)
    _check(got[0], ref, tol, "decode")
    got = pkv.paged_prefill_fp4(q, cu, kc, vc, s, s, bt, ln, 2, out_dtype=out_dtype, sm_scale=sm, max_kv_len=L)
    _check(got[1], ref, tol, "prefill")
