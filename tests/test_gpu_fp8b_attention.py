"""Decode and prefill attention over the block-scaled FP8 cache against the
64-bit form."""
import numpy as np
import pytest
import torch

from tests import fp4_ref, fp4_tight, fp8b_ref

pytestmark = pytest.mark.gpu

SM = fp8b_ref.SM


def _dev(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


class Cache:
    """K and V of a batch in shuffled pages; rows nobody wrote hold NaN codes, blocks
    nobody wrote the byte 255, and the table's spare entries point outside the pool.
    sizes(rng, L): each token's size."""

    def __init__(self, seed, lens, hkv, P, dev, page_sizes=None, spread=1.0, hidden=None, sizes=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.hkv, self.P, self.dev = rng, list(lens), hkv, P, dev
        own = page_sizes or [P] * len(lens)
        runs = [[own[b] // P] * ((L + own[b] - 1) // own[b]) for b, L in enumerate(lens)]
        order = [(b, i) for b, r in enumerate(runs) for i in range(len(r))]
        rng.shuffle(order)
        self.max_pages = max(1, max((len(r) for r in runs), default=1)) + 1
        self.table = np.full((len(lens), self.max_pages), -5, np.int32)
        at = 1
        for b, i in order:
            self.table[b, i] = at
            at += runs[b][i]
        self.pages = at + 1
        self.k, self.v, self.scale = [], [], []                  # scale: 2^ev of each token's block of V
        self.cache = [np.full((self.pages, hkv, P, 128), 0x7F, np.uint8) for _ in range(2)]
        self.exps = [np.full((self.pages, hkv, P // 16), 255, np.uint8) for _ in range(2)]
        for b, L in enumerate(lens):
            slots = fp4_ref.slots_of(self.table[b], L, P, own[b])
            for i, keep in enumerate((self.k, self.v)):
                x = fp4_ref.rows(rng, L, hkv, spread)
                x = x * (np.exp(0.7 * rng.standard_normal((L, 1, 1))) if sizes is None or i == 0 else sizes(rng, L))
                fp8b_ref.append(self.cache[i], self.exps[i], x.astype(np.float32), slots)
                keep.append(fp8b_ref.read(self.cache[i], self.exps[i], slots))
            s = slots.astype(np.int64)
            self.scale.append(np.exp2(self.exps[1][s // P, :, s % P // 16].astype(np.float64) - 127))
        self.psd = None if page_sizes is None else _dev(np.array(page_sizes, np.int32), dev)
        if hidden:                                               # (window, sinks, first query's position of b)
            window, sinks, pos = hidden
            for b in range(len(lens)):
                for i in range(self.max_pages):
                    t = np.arange(i * own[b], min((i + 1) * own[b], lens[b]))
                    if not ((t > pos[b] - window) | (t < sinks)).any():
                        self.table[b, i] = 1 << 30
        self.args = [_dev(x, dev) for x in (*self.cache, *self.exps)]
        self.tabled, self.lensd = _dev(self.table, dev), _dev(np.array(lens, np.int32), dev)

    def queries(self, rows, hq, spread=1.0):
        q = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(self.rng.standard_normal((rows, hq, 128)) * spread))
        return q, _dev(q, self.dev).to(torch.bfloat16)


def _check(got, ref, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, float(np.abs(got - ref).max()), int(bad.sum()), np.argwhere(bad)[:3].tolist())


def _raw(pkv, c, qd, bit, **kw):
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    got = pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled, c.lensd, device_error=e, seq_page_sizes=c.psd,
                                    **{"max_seq_len": max(max(c.lens), 1), "out_dtype": torch.float32, **kw})
    torch.cuda.synchronize()
    assert int(e.item()) == bit
    return got


def _decode(pkv, c, q, qd, window=0, sinks=0, out_dtype=torch.float32, err=0, sm=SM, **kw):
    got = _raw(pkv, c, qd, err, out=torch.full(qd.shape, 9.0, dtype=out_dtype, device=c.dev), sm_scale=sm, window=window,
               sinks=sinks, **kw)
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
    lens = [2900, 1, 0, 519, 2048]
    c = Cache(5, lens, 2, 16, cuda_device)
    q, qd = c.queries(len(lens), 12)
    _decode(pkv, c, q, qd, max_ctas=max_ctas)
    _decode(pkv, c, q, qd, 700, 9, max_ctas=max_ctas)


def test_decode_long_chain(pkv, cuda_device):
    """One worker over a long sequence: its accumulator is folded."""
    c = Cache(6, [20000], 1, 64, cuda_device)
    q, qd = c.queries(1, 8)
    for out_dtype in (torch.float32, torch.bfloat16):
        _decode(pkv, c, q, qd, max_ctas=1, out_dtype=out_dtype)
        _decode(pkv, c, q, qd, out_dtype=out_dtype)


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
    c = Cache(31, [int(x) for x in rng.choice([0, 1, 20, 64, 90], B)], 1, 16, cuda_device)
    q, qd = c.queries(B, G)
    a = _decode(pkv, c, q, qd, window, sinks, max_ctas=max_ctas)
    assert torch.equal(_decode(pkv, c, q, qd, window, sinks, max_ctas=max_ctas), a)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,G,window,sinks", [([2100, 2090, 2110, 2080], 4, 0, 0), ([130, 160, 150, 129], 8, 0, 0),
                                                 ([2100, 2090, 2110, 2080], 3, 500, 9), ([2100, 100, 2110, 1], 4, 0, 0)])
def test_decode_sequences_of_like_length(pkv, cuda_device, lens, G, window, sinks, out_dtype):
    """A list whose segments get a CTA each (256 of them, four sequences' pages by turns),
    and one of as many whose lengths differ."""
    c = Cache(33, lens, 1, 16, cuda_device)
    rows = [i % 4 for i in range(256)]
    q, qd = c.queries(256, G)
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    call = dict(out_dtype=out_dtype, max_seq_len=max(lens), max_ctas=1 << 20, window=window, sinks=sinks, device_error=e)
    got = pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled[rows].contiguous(), c.lensd[rows].contiguous(), **call)
    for i in range(0, 256, 5):
        b, x = rows[i], q[i].astype(np.float64)
        ref = fp4_ref.attend(x, c.k[b], c.v[b], lens[b] - 1, window, sinks, SM)
        tol = _tight_decode(c, b, x, lens[b] - 1, window, sinks, SM) if out_dtype == torch.float32 else \
            fp4_ref.attention_tolerance(x, c.k[b], c.v[b], ref, SM, True)
        _check(got[i], ref, tol, (i, lens[b]))
    again = pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled[rows].contiguous(), c.lensd[rows].contiguous(), **call)
    assert torch.equal(got, again) and int(e.item()) == 0


@pytest.mark.parametrize("spread", [30.0, 1e-4, 1e4])
def test_decode_large_and_small_scores(pkv, cuda_device, spread):
    """Scores from almost equal to one that takes all the weight, rising and
    falling along the sequence."""
    c = Cache(7, [1, 40, 333, 1500], 2, 16, cuda_device)
    q, qd = c.queries(4, 8, spread)
    for sm in (SM / max(1.0, spread / 30), -SM / max(1.0, spread / 30)):
        _decode(pkv, c, q, qd, sm=sm)
        _decode(pkv, c, q, qd, 100, 4, sm=sm)


# V's size over the tokens: rising and falling by 2^30, one token far above the
# others, one far below, and sizes at both ends of what blocks can have.
SIZES = {
    "rising": lambda rng, L: np.exp2(np.linspace(-15, 15, L)).reshape(L, 1, 1),
    "falling": lambda rng, L: np.exp2(np.linspace(15, -15, L)).reshape(L, 1, 1),
    "one large": lambda rng, L: np.where(np.arange(L) == L // 3, 2.0 ** 17, 1.0).reshape(L, 1, 1),
    "mixed": lambda rng, L: np.exp2(rng.uniform(-12, 12, (L, 1, 1))),
    "huge": lambda rng, L: np.full((L, 1, 1), 2.0 ** 100),
    "tiny": lambda rng, L: np.full((L, 1, 1), 2.0 ** -100),
    "zeros": lambda rng, L: (np.arange(L) // 16 % 2).reshape(L, 1, 1),
}


def _tight_decode(c, b, q, p, window, sinks, sm):
    """fp4_tight's tolerance, and what small contributions lose.

    P = 2^(s + ev - n) goes to the tensor cores as h = f16(P) and f16(P - h), which are
    off by 2^-25 together at most where P or its rest is below 2^-14.  The reference n is
    12 below the largest s + ev when it is set and moves only upwards, so the largest P is
    at least 2^12 and 2^-25 is 2^-37 of it: a key whose weight is w and whose code is v 2^-ev
    moves the output by at most 2^-37 max(w 2^ev) |v| 2^-ev.
    """
    k, v, scale = c.k[b], c.v[b], c.scale[b]
    g = q.shape[0] // k.shape[1]
    t = fp4_ref.visible(p, window, sinks)
    s = np.einsum("hd,thd->ht", q, np.repeat(k[t], g, 1)) * sm
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    top = (w * np.repeat(scale[t], g, 1).T).max(1)
    codes = np.repeat((np.abs(v[t]) / scale[t][..., None]).sum(0), g, 0)
    return fp4_tight.tolerance(q, k, v, p, window, sinks, sm) + 2.0 ** -37 * top[:, None] * codes


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("max_ctas", [0, 2])
def test_decode_blocks_of_different_sizes(pkv, cuda_device, sizes, max_ctas):
    """An fp32 output is as near as its own terms allow (sum w |v|), whatever the
    blocks' scales are: weights that meet small values are not lost to those that
    meet large ones."""
    c = Cache(13, [1, 40, 333, 1500], 2, 16, cuda_device, sizes=SIZES[sizes])
    q, qd = c.queries(4, 8, 2.0)
    for window, sinks in ((0, 0), (90, 5)):
        got = _raw(pkv, c, qd, 0, window=window, sinks=sinks, max_ctas=max_ctas)
        for b, L in enumerate(c.lens):
            x = q[b].astype(np.float64)
            ref = fp4_ref.attend(x, c.k[b], c.v[b], L - 1, window, sinks, SM)
            _check(got[b], ref, _tight_decode(c, b, x, L - 1, window, sinks, SM), (sizes, b, window))


def _at_the_ends(pkv, dev, e, out_dtype, run):
    """run(cache) over V of the size 2^e (an end of what blocks can hold), and what it
    gives over the same V at 1: outputs 2^e apart, exactly but for the last rounding."""
    got, codes = [], []
    for size in (2.0 ** e, 1.0):
        c = Cache(34, [40, 700], 2, 16, dev, sizes=lambda rng, L: np.full((L, 1, 1), size))
        got.append(run(c).double().cpu().numpy())
        codes.append(c.cache[1])
    assert (codes[0] == codes[1]).all()                          # no block's exponent has met its end
    want = got[1] * 2.0 ** e
    assert np.isfinite(got[0]).all() and (got[0] != 0).any()
    # the codes are the same, and the size enters by exact factors: the results are the same but for fp32's
    # (bf16's) smallest step below its normal numbers
    least = 2.0 ** (-133 if out_dtype == torch.bfloat16 else -149)
    bad = ~(np.abs(got[0] - want) <= least)
    assert not bad.any(), (int(bad.sum()), got[0][bad][:4], want[bad][:4])


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [-110, 120])
@pytest.mark.parametrize("max_ctas", [0, 1, 5])
def test_decode_at_the_ends_of_the_exponents(pkv, cuda_device, e, max_ctas, out_dtype):
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(3)).to(cuda_device).bfloat16()
    _at_the_ends(pkv, cuda_device, e, out_dtype, lambda c: _raw(pkv, c, q, 0, out_dtype=out_dtype, max_ctas=max_ctas))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [-110, 120])
def test_prefill_at_the_ends_of_the_exponents(pkv, cuda_device, e, out_dtype):
    q = torch.randn(90, 8, 128, generator=torch.Generator().manual_seed(4)).to(cuda_device).bfloat16()
    cu = torch.tensor([0, 30, 90], dtype=torch.int32, device=cuda_device)
    _at_the_ends(pkv, cuda_device, e, out_dtype, lambda c: pkv.paged_prefill_fp8b(
        q, cu, *c.args, c.tabled, c.lensd, 60, max_kv_len=700, out_dtype=out_dtype))


def test_decode_page_sizes_per_sequence(pkv, cuda_device):
    lens = [700, 33, 1, 256, 90]
    c = Cache(8, lens, 2, 16, cuda_device, page_sizes=[64, 16, 256, 128, 32])
    q, qd = c.queries(5, 8)
    _decode(pkv, c, q, qd)
    _decode(pkv, c, q, qd, 50, 3)
    c.psd[1] = 24
    got = _raw(pkv, c, qd, pkv.DEVERR_PAGESIZE)
    assert (got[1] == 0).all()


def _as_before(c, q, got, full, b, max_ctas):
    """Sequence b's rows, whose own tokens have not changed: the same bits from its
    cluster; from the list, whose cuts follow every sequence's length, the same up
    to the order of their sums."""
    if max_ctas == 0:
        assert torch.equal(got[b], full[b])
    else:
        x, L = q[b].astype(np.float64), c.lens[b]
        ref = full[b].double().cpu().numpy()
        _check(got[b], ref, 2 * _tight_decode(c, b, x, L - 1, 0, 0, SM), ("as before", b))


@pytest.mark.parametrize("max_ctas", [0, 3])
def test_decode_bad_pages_and_lengths(pkv, cuda_device, max_ctas):
    """A page outside the pool reads as zeros (score 0, value 0); lengths are
    clamped; both are flagged."""
    c = Cache(9, [100, 64], 2, 16, cuda_device)
    q, qd = c.queries(2, 8)
    kw = dict(max_ctas=max_ctas)
    c.tabled[0, 2] = c.pages
    c.k[0][32:48] = 0
    c.v[0][32:48] = 0
    _decode(pkv, c, q, qd, err=pkv.DEVERR_PAGE, **kw)
    _decode(pkv, c, q, qd, 20, 4, **kw)                          # not seen there: not looked at
    c.tabled[0, 2] = -1
    _decode(pkv, c, q, qd, err=pkv.DEVERR_PAGE, **kw)
    c.tabled[0, 2] = 3
    c.lensd[1] = -3
    got = _raw(pkv, c, qd, pkv.DEVERR_SEQLEN, **kw)
    assert (got[1] == 0).all()
    c.lensd[1] = 64
    full = _raw(pkv, c, qd, 0, **kw)
    c.lensd[1] = 2 ** 31 - 1
    # clamped to 100 tokens, of which the table has pages for 64: the others read as zeros
    got = _raw(pkv, c, qd, pkv.DEVERR_SEQLEN | pkv.DEVERR_PAGE, max_seq_len=64 + 36, **kw)
    _as_before(c, q, got, full, 0, max_ctas)
    c.lensd[1] = 65
    got = _raw(pkv, c, qd, pkv.DEVERR_SEQLEN, max_seq_len=64, **kw)
    _as_before(c, q, got, full, 1, max_ctas)


@pytest.mark.parametrize("max_ctas", [0, 2])
def test_decode_nan_codes(pkv, cuda_device, max_ctas):
    """A NaN of V in sight is NaN in its dim; out of sight it is not seen, in the
    window's and the sinks' own blocks either; a NaN in K takes the whole row."""
    c = Cache(10, [200], 1, 16, cuda_device)
    q, qd = c.queries(1, 4)
    kw = dict(max_ctas=max_ctas)
    base = _decode(pkv, c, q, qd, 55, 3, **kw)
    slot = fp4_ref.slots_of(c.table[0], 200, 16)
    for t in (3, 15, 100, 144):                                  # 145 is the first one of the window
        c.args[1].view(-1, 128)[int(slot[t]), 77] = 0xFF
        c.args[0].view(-1, 128)[int(slot[t])] = 0x7F
    assert torch.equal(_raw(pkv, c, qd, 0, window=55, sinks=3, **kw), base)
    c.args[0].copy_(_dev(c.cache[0], c.dev))
    got = _raw(pkv, c, qd, 0, **kw)
    assert torch.isnan(got[..., 77]).all() and int(torch.isnan(got).sum()) == 4
    c.args[0].view(-1, 128)[int(slot[100]), 5] = 0xFF
    assert torch.isnan(_raw(pkv, c, qd, 0, **kw)).all()


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
        ws = torch.empty(pkv.pkv_decode_fp8b_workspace_size(len(lens), 3, 1, max_seq_len=900), dtype=torch.uint8,
                         device=cuda_device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled, c.lensd, out=out, workspace=ws, max_seq_len=900, window=w,
                                      sinks=2)
        outs.append(out)
        graphs.append((g, ws))
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.paged_gqa_decode_fp8b(qd, *c.args, c.tabled, c.lensd, out_dtype=torch.float32, max_seq_len=900, stream=side)
    side.synchronize()
    assert torch.equal(got, outs[1])


def test_decode_workspace_needs_no_initialisation(pkv, cuda_device):
    lens = [4000, 17, 0]
    c = Cache(12, lens, 2, 16, cuda_device)
    q, qd = c.queries(3, 4)
    n = pkv.pkv_decode_fp8b_workspace_size(3, 4, 2, max_seq_len=4000)
    a, b = (_raw(pkv, c, qd, 0, workspace=torch.full((n,), v, dtype=torch.uint8, device=cuda_device)) for v in (0, 0xFF))
    assert torch.equal(a, b) and not torch.isnan(a).any()
    with pytest.raises(pkv.PkvError):
        _raw(pkv, c, qd, 0, workspace=torch.empty(max(n - 256, 0), dtype=torch.uint8, device=cuda_device))


# ---------------------------------------------------------------- prefill
def _tight(q, k, v, p, window, sinks, sm):
    """fp4_tight's tolerance, and what small weights lose.

    A weight P = 2^(score - m) goes to the tensor cores as f16(h) + f16(P - h), h being P
    with 11 significant bits.  Both conversions round to multiples of 2^-24 where they
    get below 2^-14, so P is off by at most 2 x 2^-25 then.  The reference m is 12 below the
    largest score when it is set and moves only upwards, so the largest P is at least
    2^12, and 2^-24 is 2^-36 of the largest weight, for each key: 2^-36 w_max sum |v|.
    (Decode refers weights to the largest contribution instead.)

    Where CTAs share a row's keys, n of them, each part's sums are weighted and added, of
    the outputs and of the weights: the exponential (2^-22), its argument's rounding (m - M
    is off by 2^-24 of itself, and 2^(m - M) |m - M| ln 2 < 1), the product and n additions
    (2^-24 each), twice: 2 (n + 6) 2^-24 sum w |v|.  A part has two key tiles or more.
    """
    Hq, g = q.shape[0], q.shape[0] // k.shape[1]
    t = fp4_ref.visible(p, window, sinks)
    s = np.einsum("hd,thd->ht", q, np.repeat(k[t], g, 1)) * sm
    w = np.exp(s - s.max(1, keepdims=True))
    lost = 2.0 ** -36 / w.sum(1)[:, None] * np.repeat(np.abs(v[t]).sum(0), g, 0)
    parts = (p // 128 + 1) // 2
    if parts > 1:
        lost = lost + 2 * (parts + 6) * 2.0 ** -24 / w.sum(1)[:, None] * np.einsum("ht,thd->hd", w, np.abs(np.repeat(v[t], g, 1)))
    return fp4_tight.tolerance(q, k, v, p, window, sinks, sm) + lost


def _prefill(pkv, c, ns, hq, window=0, sinks=0, out_dtype=torch.float32, q_spread=1.0, sm=SM, sample=40, total=0, err=0,
             pad_rows=3, skip=(), tight=False, bound=0):
    cu = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    q, qd = c.queries(int(cu[-1]) + pad_rows, hq, q_spread)
    out = torch.full(qd.shape, 9.0, dtype=out_dtype, device=c.dev)
    e = torch.zeros(1, dtype=torch.int32, device=c.dev)
    pkv.paged_prefill_fp8b(qd, _dev(cu, c.dev), *c.args, c.tabled, c.lensd, max(max(ns), 1), out=out,
                           max_kv_len=max(max(c.lens), 1, bound), sm_scale=sm, device_error=e, window=window, sinks=sinks,
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
            tol = _tight(x, c.k[b], c.v[b], p, window, sinks, sm) if tight else \
                fp4_ref.attention_tolerance(x, c.k[b][:p + 1], c.v[b][:p + 1], ref, sm, bf16)
            _check(out[cu[b] + r], ref, tol, ("prefill", b, L, n, int(r), window, sinks))
    return qd, out


@pytest.mark.parametrize("hkv,G,P", [(1, 8, 16), (2, 4, 32), (3, 1, 64), (2, 7, 128), (1, 3, 256), (2, 5, 16),
                                     (1, 6, 16), (8, 2, 16)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_ragged(pkv, cuda_device, hkv, G, P, out_dtype):
    """Chunks of no, one and many queries; whole sequences; odd lengths."""
    lens, ns = [1, 50, 300, 128, 17, 129, 0, 385], [1, 0, 45, 128, 17, 1, 0, 130]
    c = Cache(hkv * 10 + G, lens, hkv, P, cuda_device)
    _prefill(pkv, c, ns, hkv * G, out_dtype=out_dtype, sample=12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 20), (100, 4), (128, 128), (129, 0), (300, 140), (5000, 4)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_window(pkv, cuda_device, window, sinks, out_dtype):
    lens, ns = [700, 1, 300, 1000], [70, 1, 300, 33]
    c = Cache(window + sinks, lens, 2, 16, cuda_device, hidden=(window, sinks, [L - n for L, n in zip(lens, ns)]))
    _prefill(pkv, c, ns, 8, window, sinks, out_dtype, sample=10)


@pytest.mark.parametrize("sizes", ["one large", "mixed", "huge", "tiny", "zeros"])
def test_prefill_blocks_of_different_sizes(pkv, cuda_device, sizes):
    """As near as the outputs' own terms allow, for blocks of like size."""
    c = Cache(14, [40, 333, 900], 2, 16, cuda_device, sizes=SIZES[sizes])
    wide = sizes in ("one large", "mixed")
    _prefill(pkv, c, [40, 33, 20], 8, q_spread=2.0, tight=not wide)
    _prefill(pkv, c, [40, 33, 20], 8, 90, 5, q_spread=2.0, tight=not wide)
    _prefill(pkv, c, [40, 33, 20], 8, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_long_context(pkv, cuda_device, out_dtype):
    """References taken by a cluster of CTAs; rows of many key tiles."""
    c = Cache(15, [18000, 5000], 1, 64, cuda_device)
    _prefill(pkv, c, [5, 130], 4, out_dtype=out_dtype, sample=6, total=23000)
    _prefill(pkv, c, [5, 130], 4, 6000, 70, out_dtype=out_dtype, sample=6)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
def test_prefill_nan_codes(pkv, cuda_device, out_dtype, window, sinks):
    """A NaN of V reaches the queries that see it, in its dim; the others' rows
    are as without it."""
    L, n, at = 300, 200, {110: 5, 130: 64, 250: 127, 251: 5}
    c = Cache(16, [L], 1, 16, cuda_device)
    cu = torch.tensor([0, n], dtype=torch.int32, device=cuda_device)
    q, qd = c.queries(n, 3)

    def run():
        return pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, n, max_kv_len=L, out_dtype=out_dtype,
                                      window=window, sinks=sinks)

    base = run()
    slot = fp4_ref.slots_of(c.table[0], L, 16)
    for t, d in at.items():
        c.args[1].view(-1, 128)[int(slot[t]), d] = 0xFF
    got = run()
    want = torch.zeros_like(got, dtype=torch.bool)
    for r in range(n):
        for t, d in at.items():
            if t in fp4_ref.visible(L - n + r, window, sinks):
                want[r, :, d] = True
    assert torch.equal(torch.isnan(got), want)
    # (codes beside the NaN are still read with the same scales)
    assert torch.equal(got[~want.any(2).any(1)], base[~want.any(2).any(1)])
    c.args[0].view(-1, 128)[int(slot[200]), 9] = 0x7F
    seen = torch.tensor([200 in fp4_ref.visible(L - n + r, window, sinks) for r in range(n)], device=cuda_device)
    got = run()
    assert torch.isnan(got[seen]).all() and torch.equal(torch.isnan(got[~seen]), want[~seen])


# Few rows over a long past: CTAs share a query tile's keys.  Lengths around the parts' ends (4 key
# tiles of 128 in the longest sequence, 2 at least in others: of 897 tokens' 256 queries the first
# ones see nothing of the last part), a sequence with one part, one of no tokens, more parts than lanes.
FEW_ROWS = [([1024], [1], 1, 1), ([1025], [129], 2, 8), ([897, 4096, 130, 3, 0, 2049], [256, 1, 130, 3, 0, 200], 1, 1),
            ([2000, 1100], [64, 0], 8, 4), ([1500, 3100], [40, 33], 3, 5), ([20000], [17], 1, 2)]


@pytest.mark.parametrize("lens,ns,hkv,G", FEW_ROWS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1200, 0), (1100, 300)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_few_rows_over_a_long_past(pkv, cuda_device, lens, ns, hkv, G, window, sinks, out_dtype):
    c = Cache(len(lens) + max(lens), lens, hkv, 16, cuda_device)
    _prefill(pkv, c, ns, hkv * G, window, sinks, out_dtype, sample=8)
    if window == 0:                                              # a bound of so many keys that bf16 calls read the cache itself
        _prefill(pkv, c, ns, hkv * G, window, sinks, out_dtype, sample=8, bound=200000)


@pytest.mark.parametrize("G,P,page_sizes", [(8, 16, None), (4, 64, None), (5, 16, [16, 64, 16, 256, 32, 16, 128, 16])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3000, 0), (2900, 140)])
def test_prefill_from_the_cache_itself(pkv, cuda_device, G, P, page_sizes, window, sinks):
    """Bounds that make bf16 calls widen in the attention; pages behind the window are never looked at."""
    lens, ns = [4000, 1, 1, 3500, 1, 17, 0, 1100], [30, 1, 0, 9, 1, 17, 0, 32]
    c = Cache(25 + G, lens, 8, P, cuda_device, page_sizes=page_sizes,
              hidden=(window, sinks, [L - n for L, n in zip(lens, ns)]) if window else None)
    _prefill(pkv, c, ns, 8 * G, window, sinks, torch.bfloat16, sample=4, bound=0 if window else 200000)


@pytest.mark.parametrize("sizes", ["one large", "mixed", "huge", "tiny", "zeros"])
def test_prefill_from_the_cache_itself_of_different_sizes(pkv, cuda_device, sizes):
    """Scales outside f16's and bf16's, of K and of V."""
    c = Cache(26, [1300, 700], 2, 16, cuda_device, sizes=SIZES[sizes])
    _prefill(pkv, c, [33, 20], 8, q_spread=2.0, out_dtype=torch.bfloat16, bound=200000)
    fixed = c.exps[0].copy()
    for up in (13, 15, 100):                                      # K's exponents 2^up higher, the scale as much lower
        c.args[2].copy_(torch.from_numpy(np.where(fixed == 255, 255, fixed.astype(np.int64) + up).clip(0, 255).astype(np.uint8)))
        keep = [k.copy() for k in c.k]
        c.k = [k * 2.0 ** up for k in keep]
        _prefill(pkv, c, [33, 20], 8, q_spread=2.0, out_dtype=torch.bfloat16, bound=200000, sm=SM * 2.0 ** -up)
        c.k = keep


def test_prefill_from_the_cache_itself_bad_pages(pkv, cuda_device):
    c = Cache(27, [1400, 64], 2, 16, cuda_device)
    c.tabled[0, 2] = c.pages
    for x in (c.k, c.v):
        x[0][32:48] = 0
    _prefill(pkv, c, [30, 10], 8, out_dtype=torch.bfloat16, err=pkv.DEVERR_PAGE, bound=200000)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_parts_of_a_long_context(pkv, cuda_device, out_dtype):
    """So many sequences that the longest one's parts would be above 128 key tiles: there are more of them."""
    c = Cache(21, [1] * 30 + [40000] + [200] * 39, 1, 64, cuda_device)
    _prefill(pkv, c, [1] * 30 + [5] + [7] * 39, 2, out_dtype=out_dtype, sample=2)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window,sinks,bound", [(0, 0, 2100), (1300, 130, 2100), (0, 0, 200000)])
def test_prefill_few_rows_nan_codes(pkv, cuda_device, out_dtype, window, sinks, bound):
    """NaNs of V and of K in several parts of the keys."""
    L, n, at = 2100, 80, {129: 5, 700: 64, 1990: 127, 2060: 0, 2099: 5}
    c = Cache(22, [L], 1, 16, cuda_device)
    cu = torch.tensor([0, n], dtype=torch.int32, device=cuda_device)
    q, qd = c.queries(n, 3)

    def run():
        return pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, n, max_kv_len=bound, out_dtype=out_dtype,
                                      window=window, sinks=sinks)

    def seen(t):
        return torch.tensor([t in fp4_ref.visible(L - n + r, window, sinks) for r in range(n)], device=cuda_device)

    base = run()
    slot = fp4_ref.slots_of(c.table[0], L, 16)
    for t, d in at.items():
        c.args[1].view(-1, 128)[int(slot[t]), d] = 0xFF
    got = run()
    want = torch.zeros_like(got, dtype=torch.bool)
    for t, d in at.items():
        want[seen(t), :, d] = True
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got[~want], base[~want])
    for t in (805, 2080):
        before = c.args[0].view(-1, 128)[int(slot[t]), 9].clone()
        c.args[0].view(-1, 128)[int(slot[t]), 9] = 0x7F
        bad = seen(t)
        got = run()
        assert torch.isnan(got[bad]).all() and torch.equal(torch.isnan(got[~bad]), want[~bad])
        c.args[0].view(-1, 128)[int(slot[t]), 9] = before


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_prefill_few_rows_captured(pkv, cuda_device, out_dtype):
    """Nothing of the workspace is read that the call has not written; a replay after the lengths have changed."""
    lens, ns = [897, 3000, 700, 90], [256, 20, 1, 90]
    c = Cache(23, lens, 2, 16, cuda_device)
    cu = _dev(np.concatenate(([0], np.cumsum(ns))).astype(np.int32), cuda_device)
    _, qd = c.queries(int(cu[-1]), 8)
    n = pkv.pkv_prefill_fp8b_workspace_size(4, 2, 256, 3000)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda_device)
    got = torch.empty(qd.shape, dtype=out_dtype, device=cuda_device)

    def call(out, **kw):
        return pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, 256, out=out, max_kv_len=3000, **kw)

    want = call(torch.empty_like(got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(got, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not torch.isnan(want).any()
    c.lensd[1] = 1000
    c.lensd[2] = 1
    g.replay()
    ws.fill_(0xFF)
    assert torch.equal(got, call(torch.empty_like(got)))
    with pytest.raises(pkv.PkvError):
        call(got, workspace=ws[:n - 512])


def test_prefill_bad_input(pkv, cuda_device):
    c = Cache(17, [100, 64, 90], 2, 16, cuda_device)
    c.tabled[0, 2] = c.pages
    c.k[0][32:48] = 0
    c.v[0][32:48] = 0
    _prefill(pkv, c, [30, 10, 5], 8, err=pkv.DEVERR_PAGE)
    c.tabled[0, 2] = 1
    c.lensd[1] = 5                                               # fewer tokens than queries
    _prefill(pkv, c, [0, 10, 5], 8, err=pkv.DEVERR_SEQLEN, skip=(1,))
    c.lensd[1] = 2 ** 31 - 1
    _prefill(pkv, c, [0, 10, 5], 8, err=pkv.DEVERR_SEQLEN, skip=(1,))
    c.lensd[1] = 64
    # more keys than the workspace was said to need: the regions behind its end are flagged, their rows stay
    c = Cache(17, [1000, 64], 2, 16, cuda_device)
    _prefill(pkv, c, [30, 10], 8, err=pkv.DEVERR_SEQLEN, total=128, skip=(0, 1))


def test_prefill_page_sizes_and_streams(pkv, cuda_device):
    lens, ns = [700, 33, 1, 256, 90], [40, 33, 1, 7, 20]
    c = Cache(18, lens, 2, 16, cuda_device, page_sizes=[64, 16, 256, 128, 32])
    qd, out = _prefill(pkv, c, ns, 8, sample=5)
    cu = _dev(np.concatenate(([0], np.cumsum(ns))).astype(np.int32), cuda_device)
    n = pkv.pkv_prefill_fp8b_workspace_size(5, 2, 40, 700)
    ws, got = torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda_device), torch.full_like(out, 9.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, 40, out=got, max_kv_len=700, workspace=ws,
                               seq_page_sizes=c.psd)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pkv.paged_prefill_fp8b(qd, cu, *c.args, c.tabled, c.lensd, 40, out_dtype=torch.float32, max_kv_len=700,
                                   seq_page_sizes=c.psd, stream=side)
    side.synchronize()
    assert torch.equal(other[:int(cu[-1])], out[:int(cu[-1])])


# ---------------------------------------------------------------- together
def test_a_request_from_prompt_to_release(pkv, cuda_device):
    """Plan, append, prefill, then captured decode steps (plan, append, decode in
    one graph), then release: the outputs are those over the rows that came in."""
    rng = np.random.default_rng(19)
    B, H, G, P, steps, pages = 5, 2, 4, 16, 37, 60
    dev = cuda_device
    past = torch.zeros(B, dtype=torch.int32, device=dev)
    table = torch.full((B, 12), -1, dtype=torch.int32, device=dev)
    pool = pkv.page_pool(pages, dev, rng.permutation(pages))
    free = pool.clone()
    (kc, ke), (vc, ve) = (pkv.fp8b_cache(pages, H, P, dev) for _ in range(2))
    e = torch.zeros(1, dtype=torch.int32, device=dev)
    ns = [33, 1, 80, 16, 7]
    new = torch.tensor(ns, dtype=torch.int32, device=dev)
    lens, cu, slots, pos = pkv.plan_pages(past, new, table, pool, P, max_tokens=150, device_error=e)
    rows = [fp4_ref.rows(rng, 150, H) for _ in range(2)]
    k, v = (_dev(x, dev).to(torch.bfloat16) for x in rows)
    pkv.kv_append_fp8b(k, v, slots, kc, vc, ke, ve, e)
    q = _dev(rng.standard_normal((150, H * G, 128)).astype(np.float32), dev).to(torch.bfloat16)
    out = pkv.paged_prefill_fp8b(q, cu, kc, vc, ke, ve, table, lens, 80, out_dtype=torch.float32, max_kv_len=192, device_error=e)
    assert pos[:sum(ns)].tolist() == [i for n in ns for i in range(n)]

    def reference(x, b, p):
        s = fp4_ref.slots_of(table[b].cpu().numpy(), p + 1, P)
        kv = [fp8b_ref.read(c.cpu().numpy(), y.cpu().numpy(), s) for c, y in ((kc, ke), (vc, ve))]
        ref = fp4_ref.attend(x, *kv, p, 0, 0, SM)
        return ref, fp4_tight.tolerance(x, *kv, p, 0, 0, SM)

    for b, n in enumerate(ns):
        x = q[int(cu[b]) + n - 1].double().cpu().numpy()
        _check(out[int(cu[b]) + n - 1], *reference(x, b, n - 1), ("prefill", b))
    one = torch.ones(B, dtype=torch.int32, device=dev)
    kd, vd = (torch.empty((B, H, 128), dtype=torch.bfloat16, device=dev) for _ in range(2))
    qd, od = torch.empty((B, H * G, 128), dtype=torch.bfloat16, device=dev), torch.empty((B, H * G, 128), device=dev)
    cu1, slots1 = torch.empty(B + 1, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int64, device=dev)
    pos1 = torch.empty(B, dtype=torch.int32, device=dev)
    ws = torch.empty(pkv.pkv_decode_fp8b_workspace_size(B, H * G, H, max_seq_len=192), dtype=torch.uint8, device=dev)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.plan_pages(lens, one, table, pool, P, seq_lens=lens, cu_q=cu1, slot_mapping=slots1, positions=pos1, device_error=e)
        pkv.kv_append_fp8b(kd, vd, slots1, kc, vc, ke, ve, e)
        pkv.paged_gqa_decode_fp8b(qd, kc, vc, ke, ve, table, lens, out=od, workspace=ws, max_seq_len=192, device_error=e)
    for i in range(steps):
        for x in (kd, vd, qd):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32) * 2.0 ** (i % 5)))
        g.replay()
        if i % 9 == 0 or i == steps - 1:
            for b, n in enumerate(ns):
                x = qd[b].double().cpu().numpy()
                _check(od[b], *reference(x, b, n + i), ("decode", b, i))
    assert lens.tolist() == [n + steps for n in ns] and int(e.item()) == 0
    pkv.release_pages(lens, table, pool, P, device_error=e)
    n = int(pool[0])
    assert n == int(free[0]) and sorted(pool[4:4 + n].tolist()) == sorted(free[4:4 + n].tolist())
    assert int(e.item()) == 0


def test_calls_behind_copies_fills_and_other_streams(pkv, cuda_device):
    """Each call, brought onto the GPU before what is ahead of it has ended, waits for that: kernels
    of its own kind, copies, fills and another stream's work, captured; as with a synchronisation
    between any two of them."""
    dev, B, H, G, P, n, pages = cuda_device, 40, 4, 4, 16, 100, 300
    gen = torch.Generator(device=dev).manual_seed(24)
    pool0 = pkv.page_pool(pages, dev)
    past0, new = torch.zeros(B, dtype=torch.int32, device=dev), torch.full((B,), n, dtype=torch.int32, device=dev)
    new[3] = 0
    T = B * n
    src = [torch.empty((T, H, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    qsrc = torch.empty((T, H * G, 128), dtype=torch.bfloat16, device=dev)
    k, v, q, qd = *(torch.empty_like(x) for x in src), torch.empty_like(qsrc), torch.empty((B, H * G, 128), dtype=torch.bfloat16, device=dev)
    (kc, ke), (vc, ve) = (pkv.fp8b_cache(pages, H, P, dev) for _ in range(2))
    table, pool, past = torch.empty((B, 8), dtype=torch.int32, device=dev), pool0.clone(), past0.clone()
    lens, cu = torch.empty_like(past0), torch.empty(B + 1, dtype=torch.int32, device=dev)
    slots, pos = torch.empty(T, dtype=torch.int64, device=dev), torch.empty(T, dtype=torch.int32, device=dev)
    e = torch.zeros(1, dtype=torch.int32, device=dev)
    back = [torch.empty_like(k) for _ in range(2)]
    od, op = torch.empty((B, H * G, 128), device=dev), torch.empty_like(q)
    wd = torch.empty(pkv.pkv_decode_fp8b_workspace_size(B, H * G, H, max_seq_len=128), dtype=torch.uint8, device=dev)
    wp = torch.empty(pkv.pkv_prefill_fp8b_workspace_size(B, H, n, 128), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream(dev)

    def on_the_side():
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            v.copy_(src[1])
            od.fill_(7.0)
        torch.cuda.current_stream(dev).wait_stream(side)

    steps = [lambda: pool.copy_(pool0), lambda: past.copy_(past0), lambda: table.fill_(-1), lambda: e.zero_(),
             lambda: pkv.plan_pages(past, new, table, pool, P, seq_lens=lens, cu_q=cu, slot_mapping=slots, positions=pos,
                                    device_error=e),
             lambda: k.copy_(src[0]), on_the_side,
             lambda: pkv.kv_append_fp8b(k, v, slots, kc, vc, ke, ve, e),
             lambda: pkv.kv_read_fp8b(slots, kc, vc, ke, ve, *back, device_error=e),
             lambda: q.copy_(qsrc), lambda: op.zero_(),
             lambda: pkv.paged_prefill_fp8b(q, cu, kc, vc, ke, ve, table, lens, n, out=op, workspace=wp, max_kv_len=128, device_error=e),
             lambda: qd.copy_(qsrc[:B]),
             lambda: pkv.paged_gqa_decode_fp8b(qd, kc, vc, ke, ve, table, lens, out=od, workspace=wd, max_seq_len=128, device_error=e),
             lambda: pkv.release_pages(lens, table, pool, P, device_error=e),
             lambda: pkv.plan_pages(past, new, table, pool, P, seq_lens=lens, cu_q=cu, slot_mapping=slots, positions=pos,
                                    device_error=e)]
    results = (table, pool, lens, cu, slots, pos, e, *back, op, od)

    def fresh(seed):
        gen.manual_seed(seed)
        for x in (*src, qsrc):
            x.normal_(generator=gen)

    def apart():
        for step in steps:
            step()
            torch.cuda.synchronize()
        return [x.clone() for x in results]

    fresh(0)
    apart()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            for step in steps:
                step()
    for seed in range(1, 5):
        fresh(seed)
        want = apart()
        fresh(seed + 100)
        apart()
        fresh(seed)
        g.replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(results, want)):
            assert torch.equal(x, y), i
    assert int(e.item()) == 0
