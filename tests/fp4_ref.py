"""Plain 64-bit forms of the 4-bit cache and of the attention over it (NumPy),
for the tests: no code of the library, no CUDA.

A row of 128 values is 8 blocks of 16 E2M1 codes with one E4M3 scale each; a
tile of 1152 bytes holds 16 tokens of a kv head, 64 bytes of codes a token,
then 8 scales a token.
"""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    c = np.arange(256)
    ex, m = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (ex - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def nearest(grid, x):
    """Index of the grid value nearest to x >= 0, ties to the even index,
    saturating at the last one."""
    i = np.clip(np.searchsorted(grid, x, side="left"), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((lo < hi) | ((lo == hi) & ((i - 1) % 2 == 0)), i - 1, i)


def quantise(x: np.ndarray, scale: np.ndarray):
    """fp32 rows [T, H, 128], scales fp32 [H] -> codes uint8 [T, H, 128] (one
    code a byte) and block scales uint8 [T, H, 8]."""
    T, H, _ = x.shape
    b = x.reshape(T, H, 8, 16).astype(np.float32)
    k = scale.astype(np.float32).reshape(1, H, 1)
    nan = np.isnan(b).any(-1)
    amax = np.abs(np.where(np.isnan(b), 0, b)).max(-1)
    with np.errstate(all="ignore"):
        ratio = amax / (np.float32(6.0) * k)                    # fp32, IEEE
        s = nearest(e4m3_values()[:127], ratio.astype(np.float64)).astype(np.uint8)
        step = e4m3_values()[s].astype(np.float32) * k
        q = (b / np.where(step > 0, step, 1)[..., None]).astype(np.float32)
    mag = nearest(E2M1, np.abs(np.where(np.isnan(q), 0, q)).astype(np.float64)).astype(np.uint8)
    c = mag | (np.signbit(b).astype(np.uint8) << 3)
    dead = nan | (s == 0)
    c[dead] = 0
    s[nan] = 0x7F
    return c.reshape(T, H, 128), s


def write(pool: np.ndarray, codes, scales, slots):
    """Codes and scales of T tokens into a pool [pages, H, P, 72] (in place)."""
    pages, H, P, _ = pool.shape
    tiles = pool.reshape(pages, H, P // 16, 1152)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= pages * P:
            continue
        pg, r = divmod(int(slot), P)
        i = r % 16
        tiles[pg, :, r // 16, 64 * i:64 * i + 64] = packed[t]
        tiles[pg, :, r // 16, 1024 + 8 * i:1024 + 8 * i + 8] = scales[t]


def block_values(pool: np.ndarray, slots):
    """e * s of the rows at the slots, fp64 [T, H, 128] (exact); slots outside
    the pool give zeros."""
    pages, H, P, _ = pool.shape
    tiles = pool.reshape(pages, H, P // 16, 1152)
    out = np.zeros((len(slots), H, 128))
    e4 = e4m3_values()
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= pages * P:
            continue
        pg, r = divmod(int(slot), P)
        i = r % 16
        c = tiles[pg, :, r // 16, 64 * i:64 * i + 64]
        s = e4[tiles[pg, :, r // 16, 1024 + 8 * i:1024 + 8 * i + 8]]
        n = np.stack((c & 15, c >> 4), -1).reshape(H, 8, 16)
        e = E2M1[n & 7] * np.where(n >= 8, -1.0, 1.0)
        out[t] = (e * s[..., None]).reshape(H, 128)
    return out


def slots_of(table_row, n, P, page_size=None):
    """Slots of a sequence's first n tokens; page_size: its own page size."""
    pb = page_size or P
    t = np.arange(n)
    return np.asarray(table_row, np.int64)[t // pb] * P + t % pb


def visible(p, window, sinks):
    """Tokens a query at position p sees."""
    t = np.arange(p + 1)
    return t if window == 0 else t[(t > p - window) | (t < sinks)]


def attend(q, k, v, p, window, sinks, sm_scale):
    """q [Hq, 128] at position p, k and v [L, H, 128] in 64 bits -> [Hq, 128]."""
    Hq, H = q.shape[0], k.shape[1]
    t = visible(p, window, sinks)
    if t.size == 0:
        return np.zeros((Hq, 128))
    kr, vr = np.repeat(k[t], Hq // H, 1), np.repeat(v[t], Hq // H, 1)
    s = np.einsum("hd,thd->ht", q, kr) * sm_scale
    w = np.exp(s - s.max(1, keepdims=True))
    return np.einsum("ht,thd->hd", w / w.sum(1, keepdims=True), vr)


def attention_tolerance(q, k, v, ref, sm_scale, bf16):
    """How far an output may be from the 64-bit one, element by element.

    Scores are fp32 sums of exact products: with S the largest |sm_scale|
    sum |q k| a score is off by at most 10 roundings of 2^-23 S (8 chained
    products of 16, the sum of two chains, the scale), its weight by that
    relative amount twice (numerator and normaliser).  Weights: 2^-21 for the
    exponential and its argument's rounding, 2^-15 for chains of at most 256
    truncating fp32 additions (256 x 2^-23).  All of it moves the output by at
    most twice the largest |v|.  A bf16 output adds the weights' rounding to
    f16 (2^-11, again twice the largest |v|) and its own 2^-8 of the value.
    """
    g = q.shape[-2] // k.shape[-2]
    vmax = np.abs(v).max(initial=0.0)
    # a bound on |scores|, so of the size of sm_scale: a negative one turns the scores' sign, not their error's
    S = abs(sm_scale) * np.abs(np.einsum("...hd,thd->...ht", np.abs(q), np.repeat(np.abs(k), g, 1))).max(initial=0.0)
    rel = 2 * 10 * 2.0 ** -23 * S + 2.0 ** -21 + 2.0 ** -15
    tol = 2 * vmax * rel + 2.0 ** -23 * np.abs(ref)
    if bf16:
        tol = tol + 2 * vmax * 2.0 ** -11 + 2.0 ** -8 * np.abs(ref)
    return tol + 1e-30


def rows(rng, T, H, spread=1.0):
    """Rows like a model's K and V: each head its own spread, one value in 200
    eight times larger; fp32 [T, H, 128]."""
    sigma = rng.uniform(0.5, 2.0, (1, H, 1)) * spread
    x = rng.standard_normal((T, H, 128)) * sigma
    return (x * np.where(rng.random(x.shape) < 0.005, 8.0, 1.0)).astype(np.float32)


def scale_of(x) -> np.ndarray:
    return np.maximum(np.abs(x).max((0, 2)) / np.float32(448), 1e-12).astype(np.float32)


def to_bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16_bits(b: np.ndarray) -> np.ndarray:
    return (b.astype(np.uint32) << 16).view(np.float32)


SM = 1.0 / math.sqrt(128.0)
