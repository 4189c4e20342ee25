"""What an fp32 output of the 4-bit attention may be off by, from the paths'
own roundings, and a CPU model of what they would be without them."""
import numpy as np

from tests import fp4_ref

# Both kernels add the products with V in chains of 64 tensor-core additions (two
# f16 parts of a weight: 16 units of 2 tiles in decode, 4 key tiles of 8 steps in
# prefill) before the sum is folded into fp32.
CHAIN = 64


def tolerance(q, k, v, p, window, sinks, sm):
    """[Hq, 128]: how far an fp32 output at position p may be from 64 bits.

    With A = sum w |v| (element by element) and S = sm sum |q k| (the largest
    of a head's visible tokens):
      chain     CHAIN truncating additions, each less than 2^-23 of a partial
                sum, and partial sums are at most A:                CHAIN 2^-23 A
      parts     a weight as two f16 parts                           2^-21 A
      folds     fp32 sums, their rescaling and the joins of pieces, the
                normaliser's own sums: 16 roundings of 2^-24        2^-20 A
      weights   a weight is off by the rounding of its exponent (2^-21 of log2
                units under 16 of them, so 2^-21 of it), the exponential (2^-22)
                and its score: 8 chained sums of 16 products (2^-23 S each),
                4 roundings of factors (2^-24 S each), and q's components below
                2^-17 of the row's largest (2^-25 of that each, times |k|); all
                of it in numerator and normaliser                   2 delta A
    and the result's rounding, 2^-24 of it.
    """
    Hq, H = q.shape[0], k.shape[1]
    t = fp4_ref.visible(p, window, sinks)
    kr, vr = np.repeat(k[t], Hq // H, 1), np.repeat(v[t], Hq // H, 1)
    s = np.einsum("hd,thd->ht", q, kr) * sm
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    A = np.einsum("ht,thd->hd", w, np.abs(vr))
    S = (abs(sm) * np.einsum("hd,thd->ht", np.abs(q), np.abs(kr))).max(1)
    lost = 2.0 ** -25 * np.abs(q).max(1) * abs(sm) * np.abs(kr).sum(2).max(0)
    delta = 2.0 ** -21 + 2.0 ** -22 + (8 * 2.0 ** -23 + 4 * 2.0 ** -24) * S + lost
    rel = CHAIN * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -20 + 2 * delta
    return rel[:, None] * A + 2.0 ** -24 * np.abs(fp4_ref.attend(q, k, v, p, window, sinks, sm)) + 1e-30


def chained(q, k, v, p, window, sinks, sm, parts=2, fold=CHAIN, lift=12):
    """The output as the kernels' roundings give it: a weight in `parts` f16
    parts, 16 tokens an addition, truncated to fp32, `fold` additions a chain
    (0: one chain).  Everything else in 64 bits."""
    Hq, H = q.shape[0], k.shape[1]
    t = fp4_ref.visible(p, window, sinks)
    kr, vr = np.repeat(k[t], Hq // H, 1), np.repeat(v[t], Hq // H, 1)
    s = np.einsum("hd,thd->ht", q, kr) * sm
    w = np.exp(s - s.max(1, keepdims=True)) * 2.0 ** lift
    left, terms = w.copy(), []
    for _ in range(parts):
        part = left.astype(np.float16).astype(np.float64)
        left = left - part
        terms.append(part)
    pad = -len(t) % 16
    vr = np.pad(vr, ((0, pad), (0, 0), (0, 0))).reshape(-1, 16, Hq, 128)
    sums = [np.einsum("hnt,nthd->nhd", np.pad(x, ((0, 0), (0, pad))).reshape(Hq, -1, 16), vr) for x in terms]
    total, acc, n = 0.0, np.zeros((Hq, 128)), 0
    for i in range(len(vr)):
        for x in sums:
            acc = _truncate(acc + x[i])
            n += 1
            if n == fold:
                total, acc, n = total + acc, np.zeros_like(acc), 0
    return (total + acc) / w.sum(1, keepdims=True)


def _truncate(x):
    y = x.astype(np.float32)
    over = np.abs(y.astype(np.float64)) > np.abs(x)
    return np.where(over, np.nextafter(y, np.float32(0)), y).astype(np.float64)
