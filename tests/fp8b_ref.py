"""Plain 64-bit forms of the block-scaled FP8 cache and of the page plan (NumPy),
for the tests: no code of the library, no CUDA.

16 tokens of a kv head are a block: 16 rows of 128 E4M3 codes and one byte x; a
value is code * 2^(x - 127).
"""
import numpy as np

from tests import fp4_ref

GRID = fp4_ref.e4m3_values()[:127]
SM = fp4_ref.SM


def e4m3(x):
    """Codes of 64-bit values: nearest, ties to even, saturating; NaN 0x7F."""
    nan = np.isnan(x)
    a = np.minimum(np.abs(np.where(nan, 0, x)), 448.0)
    c = fp4_ref.nearest(GRID, a).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(nan, 0x7F, c).astype(np.uint8)


def values(codes, x):
    """Codes [..., 128] with bytes x [...] as 64-bit values."""
    return fp4_ref.e4m3_values()[codes] * np.exp2(x.astype(np.float64) - 127)[..., None]


def exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within -117 .. 119."""
    e = -117
    while e < 119 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(cache, exps, rows, slots):
    """Rows [T, H, 128] (any float type) into cache [pages, H, P, 128] and exps
    [pages, H, P / 16], in place."""
    pages, H, P, _ = cache.shape
    blocks = {}
    for t, s in enumerate(slots):
        if 0 <= s < pages * P:
            blocks.setdefault(int(s) // 16, []).append((int(s) % 16, t))
    for n, members in blocks.items():
        pg, i = divmod(n, P // 16)
        for h in range(H):
            new = rows[[t for _, t in members], h].astype(np.float64)
            fin = np.abs(new[np.isfinite(new)])
            e = exponent(fin.max(initial=0.0))
            block = cache[pg, h, 16 * i:16 * i + 16]
            if not any(r == 0 for r, _ in members):
                was = int(exps[pg, h, i]) - 127
                if e > was:
                    keep = [r for r in range(16) if r not in [m for m, _ in members]]
                    block[keep] = same_sign_nan(block[keep], e4m3(fp4_ref.e4m3_values()[block[keep]] * 2.0 ** (was - e)))
                e = max(e, was)
            exps[pg, h, i] = e + 127
            for (r, _), x in zip(members, new):
                block[r] = e4m3(x * 2.0 ** -e)


def same_sign_nan(old, new):
    return np.where((old & 0x7F) == 0x7F, 0x7F, new).astype(np.uint8)


def same(a, b):
    """Bytes of codes alike, a NaN of either sign being one."""
    nan = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
    return bool(((a == b) | nan).all())


def read(cache, exps, slots):
    """Values at the slots, [T, H, 128]; zeros for those outside the pool."""
    pages, H, P, _ = cache.shape
    out = np.zeros((len(slots), H, 128))
    for t, s in enumerate(slots):
        if 0 <= s < pages * P:
            pg, r = divmod(int(s), P)
            out[t] = values(cache[pg, :, r], exps[pg, :, r // 16])
    return out


def plan(past, new, table, free, P, rows, pages):
    """What plan_pages does, on lists and arrays: (seq_lens, cu_q, slots,
    positions, error bits); table [B, max_pages] and the list `free` in place."""
    B, cap = table.shape[0], table.shape[1] * P
    slots, positions = np.full(rows, -1, np.int64), np.zeros(rows, np.int32)
    none = (np.array(past, np.int32), np.zeros(B + 1, np.int32), slots, positions)
    if any(p < 0 or n < 0 or p + n > cap for p, n in zip(past, new)) or sum(new) > rows:
        return (*none, 4)
    if sum(-(-(p + n) // P) + (-p // P) for p, n in zip(past, new)) > len(free):
        return (*none, 64)
    err, cu = 0, [0]
    for b, (p, n) in enumerate(zip(past, new)):
        for i in range(-(-p // P), -(-(p + n) // P)):
            table[b, i] = free.pop()
            err |= 0 if 0 <= table[b, i] < pages else 2
        for j in range(n):
            pg = int(table[b, (p + j) // P])
            if 0 <= pg < pages:
                slots[cu[-1] + j] = pg * P + (p + j) % P
            else:
                err |= 2
            positions[cu[-1] + j] = p + j
        cu.append(cu[-1] + n)
    return np.array([p + n for p, n in zip(past, new)], np.int32), np.array(cu, np.int32), slots, positions, err


def release(lens, keep, table, free, P, pages):
    """What release_pages does; the error bits."""
    keep = [0] * len(lens) if keep is None else keep
    cap = table.shape[1] * P
    if any(k < 0 or n < k or n > cap for n, k in zip(lens, keep)):
        return 4
    back = [int(table[b, i]) for b, (n, k) in enumerate(zip(lens, keep)) for i in range(-(-k // P), -(-n // P))]
    if len(free) + len(back) > pages:
        return 64
    free.extend(reversed(back))
    return 2 if any(not 0 <= p < pages for p in back) else 0
