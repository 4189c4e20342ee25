"""What is timed of the block-scaled FP8 cache and of the page plan that feeds it:
tables and slots built on the GPU from request lengths, writing the cache, reading
it back, and the decode and prefill attention over it.

The cache.  K and V rows of 128 values are held as E4M3 codes; 16 consecutive
tokens of a kv head (a block) share a power of two, 2^(x - 127) with one byte x.
Codes are uint8 [pages][kv heads][page size][128], bytes x uint8 [pages][kv
heads][page size / 16].  There is no scale to calibrate:

  write    a block's x comes from the largest new value in it: the smallest power
           of two with which that value is within 448.  A call that writes a
           block's row 0 begins the block; one that adds rows to it keeps the
           larger of the two x and, where it grows, rounds the block's rows to it.
           Then the rows written, and those that shared a block with them, are
           read back (what is held in 8 bits is compared as the values it stands for)
  read     value = code * 2^(x - 127) for a list of slots
  decode   one query per sequence at position L - 1
  prefill  n queries per sequence at positions L - n .. L - 1, causal
  plan     a step's pages, tables and slots: sequence b holds past[b] tokens and
           brings new[b].  Its missing pages come from the end of a list of free
           ones, in the order of sequences and positions; every new token gets its
           slot (page * page size + row) and position, rows behind the last token
           slot -1 and position 0.  Then the same pages go back, last one first,
           so that the list is as it was.

A window of W tokens and S sinks leave a query at position p the tokens t <= p
with t > p - W or t < S (W = 0: all t <= p).
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _case(name, kind, **kw):
    c = {"kind": kind, "page": 16, "hkv": 8, "shape_seed": 1}
    if name:
        c["name"] = name
    c.update(kw)
    return c


def listed():
    return [
        # a decode step of a batch of 64 between 512 and 131072 tokens: one slot each, a page for some
        _case("plan_step_b64", "plan", batch=64, past_lo=512, past_hi=131072, new_lo=1, new_hi=1, pad=0),
        # a serving step of 1021 requests, ragged prompts and running ones, padded to a fixed number of rows
        _case("plan_prompts_b1021_p32", "plan", page=32, batch=1021, past_lo=0, past_hi=2000, new_lo=1, new_hi=1500,
              pad=777),
        # one decode step of a batch of 64: a token each into a block that others have begun
        _case("write_step_b64", "write", batch=64, past_lo=1, past_hi=4096, new_lo=1, new_hi=1, in_dtype="bf16",
              out_dtype="bf16", skip=0),
        # ragged chunks of fp32 rows with an odd number of heads that start inside blocks, some tokens not written
        _case("write_f32_ragged_5heads_p32", "write", hkv=5, page=32, batch=7, past_lo=1, past_hi=300, new_lo=40,
              new_hi=400, in_dtype="f32", out_dtype="f32", skip=7),
        # a 16K chunk of a long prompt joining the cache
        _case("write_chunk_16k", "write", batch=1, past_lo=16384, past_hi=16384, new_lo=16384, new_hi=16384,
              in_dtype="bf16", out_dtype="bf16", skip=0),
        # a whole 128K context read back
        _case("read_128k_p64", "read", tokens=131072, page=64, out_dtype="bf16", skip=0),
        # two short sequences on one kv head: latency, fp32 output
        _case("decode_tiny_b2", "decode", hq=8, hkv=1, batch=2, len_lo=37, len_hi=100, window=0, sinks=0,
              out_dtype="f32"),
        # an 8B layer, batch 32 at 4K
        _case("decode_8b_b32_4k", "decode", hq=32, batch=32, len_lo=4096, len_hi=4096, window=0, sinks=0,
              out_dtype="bf16"),
        # a 70B layer at 128K that keeps 4 first tokens and the last 4096
        _case("decode_70b_b4_128k_w4096_s4", "decode", hq=64, batch=4, len_lo=127984, len_hi=127984, window=4096,
              sinks=4, out_dtype="bf16"),
        # 70B geometry, a mixed batch of 64 sequences of 512 to 131072 tokens
        _case("decode_mixed_b64", "decode", hq=64, batch=64, len_lo=512, len_hi=131072, window=0, sinks=0,
              out_dtype="bf16"),
        # short ragged chunks, three query heads a kv head, fp32 output
        _case("prefill_ragged_b3", "prefill", hq=6, hkv=2, batch=3, q_lo=1, q_hi=130, past_lo=0, past_hi=700,
              window=0, sinks=0, out_dtype="f32"),
        # the last 4K chunk of a 16K prompt, 70B geometry
        _case("prefill_70b_4k_of_16k", "prefill", hq=64, batch=1, q_lo=4096, q_hi=4096, past_lo=12288, past_hi=12288,
              window=0, sinks=0, out_dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["plan", "write", "read", "decode", "prefill"])
    c = {"page": rng.choice([16, 16, 32, 64, 128, 256]), "shape_seed": rng.randrange(1 << 30)}
    if kind == "plan":
        batch = _log(rng, 1, 2048)
        a, b = _log(rng, 1, 200000 // batch), _log(rng, 1, 200000 // batch)
        p, r = rng.choice([0, _log(rng, 1, 500000 // batch)]), _log(rng, 1, 500000 // batch)
        c.update(batch=batch, new_lo=min(a, b), new_hi=max(a, b), past_lo=min(p, r), past_hi=max(p, r),
                 pad=rng.choice([0, 0, _log(rng, 1, 5000)]))
        return _case(None, kind, **c)
    if kind == "read":
        hkv = rng.randint(1, 16)
        c.update(hkv=hkv, tokens=_log(rng, 1, 131072 * 8 // hkv), out_dtype=rng.choice(["bf16", "f32"]),
                 skip=rng.choice([0, 0, 5, 9]))
        if c["out_dtype"] == "f32":
            c["tokens"] = max(1, c["tokens"] // 2)
        return _case(None, kind, **c)
    if kind == "write":
        hkv = rng.randint(1, 16)
        batch = _log(rng, 1, 256)
        most = max(1, 16384 * 4 // hkv // batch)
        a, b = _log(rng, 1, most), _log(rng, 1, most)
        p, r = rng.choice([0, _log(rng, 1, 4096)]), _log(rng, 1, 4096)
        c.update(hkv=hkv, batch=batch, new_lo=min(a, b), new_hi=max(a, b), past_lo=min(p, r), past_hi=max(p, r),
                 in_dtype=rng.choice(["bf16", "f32"]), out_dtype=rng.choice(["bf16", "f32"]),
                 skip=rng.choice([0, 0, 5, 9]))
        return _case(None, kind, **c)
    group = rng.randint(1, 8)
    hkv = rng.randint(1, 8)
    windowed = rng.random() < 0.4
    c.update(hkv=hkv, hq=hkv * group, out_dtype=rng.choice(["bf16", "bf16", "f32"]),
             window=_log(rng, 1, 8192) if windowed else 0, sinks=rng.choice([0, 1, 4, 20, 128]) if windowed else 0)
    if kind == "decode":
        batch = _log(rng, 1, 64)
        a, b = _log(rng, 1, 60000), _log(rng, 1, 60000)
        c.update(batch=batch, len_lo=min(a, b), len_hi=max(a, b))
    else:
        batch = _log(rng, 1, 8)
        a, b = _log(rng, 1, 2048 // batch), _log(rng, 1, 2048 // batch)
        p, r = rng.choice([0, _log(rng, 1, 14000)]), _log(rng, 1, 14000)
        c.update(batch=batch, q_lo=min(a, b), q_hi=max(a, b), past_lo=min(p, r), past_hi=max(p, r))
    return _case(None, kind, **c)


def _between(rng, lo, hi):
    return lo if lo == hi else int(round(math.exp(rng.uniform(math.log(max(lo, 0.5)), math.log(hi)))))


def _shapes(case):
    """Tokens that the case's sequences hold before the call, and those they bring."""
    rng = random.Random(case["shape_seed"])
    past, new = [], []
    for _ in range(case["batch"]):
        if case["kind"] == "decode":
            past.append(_between(rng, case["len_lo"], case["len_hi"]) - 1)
            new.append(1)
        elif case["kind"] == "prefill":
            new.append(_between(rng, case["q_lo"], case["q_hi"]))
            past.append(0 if case["past_hi"] == 0 else _between(rng, case["past_lo"], case["past_hi"]))
        else:
            new.append(_between(rng, case["new_lo"], case["new_hi"]))
            past.append(0 if case["past_hi"] == 0 else _between(rng, case["past_lo"], case["past_hi"]))
    return past, new


def _visible(p, window, sinks):
    """How many tokens a query at position p sees."""
    if window == 0 or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(case):
    h, page = case["hkv"], case["page"]
    if case["kind"] == "read":
        t = case["tokens"] - (case["tokens"] // case["skip"] if case["skip"] else 0)
        rows = 2 * t * h                                        # of K and of V
        b = rows * (D + D * (2 if case["out_dtype"] == "bf16" else 4)) + rows // BLOCK + 8 * case["tokens"]
        return {"bytes": b, "flops": rows * D}
    past, new = _shapes(case)
    if case["kind"] == "plan":
        pages = sum((p + n + page - 1) // page - (p + page - 1) // page for p, n in zip(past, new))
        rows = sum(new) + case["pad"]
        # lengths in and out, a slot and a position a row, each page: read from the list, written to the table,
        # read from there and written to the list
        return {"bytes": 16 * len(new) + 12 * rows + 16 * pages, "flops": 4 * rows}
    if case["kind"] == "write":
        t = sum(new)
        t -= t // case["skip"] if case["skip"] else 0
        back = t + sum(p % BLOCK for p in past)
        rows, rows_back = 2 * t * h, 2 * back * h
        b = rows * (D * (2 if case["in_dtype"] == "bf16" else 4) + D) + rows // BLOCK + 8 * t
        b += rows_back * (D + D * (2 if case["out_dtype"] == "bf16" else 4)) + rows_back // BLOCK + 8 * back
        return {"bytes": b, "flops": rows * D * 3 + rows_back * D}
    w, s, hq = case["window"], case["sinks"], case["hq"]
    osz = 2 if case["out_dtype"] == "bf16" else 4
    pairs = keys = 0
    for p0, n in zip(past, new):
        pairs += sum(_visible(p, w, s) for p in range(p0, p0 + n))
        first = 0 if w == 0 else max(0, p0 - w + 1)
        keys += p0 + n - first + min(s, first)
    return {"bytes": keys * h * (2 * D + 2 / BLOCK) + sum(new) * hq * D * (2 + osz), "flops": 4 * D * hq * pairs}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _rows(gen, sigma, tokens):
    """K or V rows [tokens, heads, 128]: normal values of each head's own
    spread and each token's own size, one value in 200 eight times larger."""
    x = torch.randn((tokens, sigma.numel(), D), generator=gen, device="cuda")
    x *= sigma.view(1, -1, 1)
    x *= torch.exp(0.7 * torch.randn((tokens, 1, 1), generator=gen, device="cuda"))
    x *= 1.0 + 7.0 * (torch.rand(x.shape, generator=gen, device="cuda") < 0.005)
    return x


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within -117 .. 119 (448 is 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 8 - (m <= 0.875).int(), -117).clamp_(-117, 119)


def _two_to(e):
    """2^e in fp32, e >= -126 (differences below it stand for nothing that is left)."""
    return ((e.int().clamp(min=-126) + 127) << 23).view(torch.float32)


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _blocks(cache):
    pages, h, page, _ = cache.shape
    return cache.view(pages, h, page // BLOCK, BLOCK, D)


def _fill(gen, cache, exps, sigma):
    """A pool filled with quantised rows, a part at a time."""
    blocks = _blocks(cache)
    pages, h, page, _ = cache.shape
    step = max(1, (1 << 19) // (h * page))
    for p0 in range(0, pages, step):
        n = min(step, pages - p0)
        x = _rows(gen, sigma, n * page).view(n, page // BLOCK, BLOCK, h, D).permute(0, 3, 1, 2, 4)
        e = _exponent(x.abs().amax((-1, -2)))
        blocks[p0:p0 + n] = _codes(x / _two_to(e)[..., None, None])
        exps[p0:p0 + n] = (e + 127).to(torch.uint8)


def _spread(gen, hkv):
    return 0.5 + 1.5 * torch.rand(hkv, generator=gen, device="cuda")


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_plan(case, gen):
    page = case["page"]
    past, new = _shapes(case)
    held = [(p + page - 1) // page for p in past]
    all_pages = [(p + n + page - 1) // page for p, n in zip(past, new)]
    total = sum(all_pages)
    pages = total + total // 4 + 1
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(past), max(all_pages)), -1, dtype=torch.int32, device="cuda")
    first = np.concatenate(([0], np.cumsum(held)))
    row = torch.from_numpy(np.repeat(np.arange(len(past)), held)).cuda()
    col = torch.from_numpy(np.arange(first[-1]) - np.repeat(first[:-1], held)).cuda()
    table[row, col] = perm[:int(first[-1])]
    pool = torch.zeros(4 + pages, dtype=torch.int32, device="cuda")
    pool[0] = pages - int(first[-1])
    pool[4:4 + pages - int(first[-1])] = perm[int(first[-1]):]
    rows = sum(new) + case["pad"]
    return {"past": _int32(past), "new": _int32(new), "tokens": sum(new), "taken": total - sum(held),
            "held": int(first[-1]), "pages": pages, "block_table": table, "pool": pool,
            "seq_lens": torch.zeros(len(past), dtype=torch.int32, device="cuda"),
            "cu_q": torch.zeros(len(past) + 1, dtype=torch.int32, device="cuda"),
            "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"),
            "positions": torch.zeros(rows, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    page, h, kind = case["page"], case["hkv"], case["kind"]
    st = {"case": case}
    if kind == "plan":
        st.update(_prepare_plan(case, gen))
        return st
    st["out_dtype"] = DTYPES[case["out_dtype"]]
    sigma = {"k": _spread(gen, h), "v": _spread(gen, h)}
    past, new = ([0], [case["tokens"]]) if kind == "read" else _shapes(case)
    lens = [p + n for p, n in zip(past, new)]
    per = [(L + page - 1) // page for L in lens]
    pages = sum(per) + sum(per) // 4 + 1
    perm = torch.randperm(pages, generator=gen, device="cuda")
    if kind in ("read", "write"):
        first = np.cumsum([0] + per)
        slots, back = [], []
        for b, (p, n) in enumerate(zip(past, new)):
            # positions whose block the new ones share, then the new ones
            pos = torch.arange(p // BLOCK * BLOCK, p + n, device="cuda")
            s = perm[int(first[b]) + pos // page] * page + pos % page
            slots.append(s[p % BLOCK:])
            back.append(s[:p % BLOCK])
        slots, old = torch.cat(slots), torch.cat(back)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1          # padding tokens
        st.update(slots=slots, back=torch.cat((old, slots)) if kind == "write" else slots)
    else:
        table = torch.zeros((len(lens), max(per)), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = perm[at:at + n].to(torch.int32)
            at += n
        rows = sum(new)
        q = torch.randn((rows, case["hq"], D), generator=gen, device="cuda").to(torch.bfloat16)
        st.update(lens=lens, qs=new, q=q, block_table=table, seq_lens=_int32(lens),
                  out=torch.zeros((rows, case["hq"], D), dtype=st["out_dtype"], device="cuda"))
        if kind == "prefill":
            st["cu_q"] = _int32(np.concatenate(([0], np.cumsum(new))))
    for x in ("k", "v"):
        st[x + "_cache"] = torch.empty((pages, h, page, D), dtype=torch.uint8, device="cuda")
        st[x + "_exp"] = torch.empty((pages, h, page // BLOCK), dtype=torch.uint8, device="cuda")
        _fill(gen, st[x + "_cache"], st[x + "_exp"], sigma[x])
        if kind == "write":
            st[x + "_new"] = _rows(gen, sigma[x], st["slots"].numel()).to(DTYPES[case["in_dtype"]])
        if kind in ("read", "write"):
            st[x + "_out"] = torch.zeros((st["back"].numel(), h, D), dtype=st["out_dtype"], device="cuda")
    if own and kind in ("decode", "prefill"):
        import paged_fp8_kv_03_gb300 as pkv
        if kind == "decode":
            n = pkv.pkv_decode_fp8b_workspace_size(len(lens), case["hq"], h, page_size=page, max_seq_len=max(lens))
        else:
            n = pkv.pkv_prefill_fp8b_workspace_size(len(lens), h, max(new), max(lens), sum(lens), case["window"],
                                                    case["sinks"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _run_own(st):
    import paged_fp8_kv_03_gb300 as pkv
    case, kind = st["case"], st["case"]["kind"]
    if kind == "plan":
        pkv.plan_pages(st["past"], st["new"], st["block_table"], st["pool"], case["page"],
                       seq_lens=st["seq_lens"], cu_q=st["cu_q"], slot_mapping=st["slots"], positions=st["positions"])
        pkv.release_pages(st["seq_lens"], st["block_table"], st["pool"], case["page"], keep_lens=st["past"])
        return st["block_table"], st["seq_lens"], st["cu_q"], st["slots"], st["positions"], st["pool"]
    cache = (st["k_cache"], st["v_cache"], st["k_exp"], st["v_exp"])
    if kind in ("write", "read"):
        if kind == "write":
            pkv.kv_append_fp8b(st["k_new"], st["v_new"], st["slots"], *cache)
        return pkv.kv_read_fp8b(st["back"], *cache, k_out=st["k_out"], v_out=st["v_out"])
    if kind == "decode":
        return pkv.paged_gqa_decode_fp8b(st["q"], *cache, st["block_table"], st["seq_lens"], out=st["out"],
                                         workspace=st["workspace"], max_seq_len=max(st["lens"]),
                                         window=case["window"], sinks=case["sinks"])
    return pkv.paged_prefill_fp8b(st["q"], st["cu_q"], *cache, st["block_table"], st["seq_lens"], max(st["qs"]),
                                  out=st["out"], max_kv_len=max(st["lens"]), max_total_kv=sum(st["lens"]),
                                  workspace=st["workspace"], window=case["window"], sinks=case["sinks"])


def _run_plan(st):
    page, past, new, pool, table = st["case"]["page"], st["past"], st["new"], st["pool"], st["block_table"]
    free = pool[4:]
    dev = past.device
    lens = past + new
    st["seq_lens"].copy_(lens)
    st["cu_q"][1:] = torch.cumsum(new, 0)
    held = (past + page - 1) // page
    add = (lens + page - 1) // page - held
    first = torch.cumsum(add, 0) - add                           # of each sequence, among the pages taken
    seqs = torch.arange(past.numel(), device=dev)
    b = torch.repeat_interleave(seqs, add, output_size=st["taken"])
    k = torch.arange(st["taken"], device=dev)
    col = (k - first[b] + held[b]).long()
    table[b, col] = free[(pool[0] - 1 - k).long()]
    pool[0] -= st["taken"]
    b2 = torch.repeat_interleave(seqs, new, output_size=st["tokens"])
    pos = torch.arange(st["tokens"], device=dev) - st["cu_q"][b2] + past[b2]
    st["positions"][:st["tokens"]] = pos.to(torch.int32)
    st["positions"][st["tokens"]:] = 0
    st["slots"][:st["tokens"]] = table[b2, (pos // page).long()].long() * page + pos % page
    st["slots"][st["tokens"]:] = -1
    # and back
    free[(pool[0] + st["taken"] - 1 - k).long()] = table[b, col]
    pool[0] += st["taken"]
    return table, st["seq_lens"], st["cu_q"], st["slots"], st["positions"], pool


def _write(x, slots, cache, exps):
    """fp32 rows [tokens, heads, 128] at slots [tokens] >= 0."""
    pages, h, page, _ = cache.shape
    blocks = _blocks(cache).permute(0, 2, 1, 3, 4)               # [pages, page / 16, heads, 16, 128]
    ids, which = torch.unique(slots // BLOCK, return_inverse=True)
    per = page // BLOCK
    amax = torch.zeros((ids.numel(), h), device=x.device)
    amax.scatter_reduce_(0, which.unsqueeze(1).expand(-1, h), x.abs().amax(-1), "amax")
    row = slots % BLOCK
    begun = torch.zeros(ids.numel(), dtype=torch.bool, device=x.device)
    begun[which[row == 0]] = True
    was = exps[ids // per, :, ids % per].int() - 127
    e = _exponent(amax)
    e = torch.where(begun.unsqueeze(1), e, torch.maximum(e, was))
    tile = blocks[ids // per, ids % per]
    old = tile.view(torch.float8_e4m3fn).float() * _two_to(was - e)[..., None, None]
    tile = torch.where(begun.view(-1, 1, 1, 1), tile, _codes(old))
    tile[which, :, row] = _codes(x / _two_to(e)[which].unsqueeze(-1))
    blocks[ids // per, ids % per] = tile
    exps[ids // per, :, ids % per] = (e + 127).to(torch.uint8)


def _gather(cache, exps, pages, rows):
    """Values of rows, [tokens, heads, 128] fp32."""
    v = cache[pages, :, rows].view(torch.float8_e4m3fn).float()
    return v * _two_to(exps[pages, :, rows // BLOCK].int() - 127).unsqueeze(-1)


def _attend(q, k, v, mask):
    """q [rows, 128], k and v [keys, 128], mask [rows, keys] or None, fp32."""
    s = q @ k.T
    if mask is not None:
        s = s.masked_fill_(~mask, -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True))
    return (s @ v) / s.sum(-1, keepdim=True)


def run(state):
    st = state
    if own:
        return _run_own(st)
    case, kind = st["case"], st["case"]["kind"]
    if kind == "plan":
        return _run_plan(st)
    page = case["page"]
    if kind in ("write", "read"):
        keep = st["back"] >= 0
        at = st["back"].clamp(min=0)
        if kind == "write":
            some = (st["slots"] >= 0).nonzero().flatten()
        for x in ("k", "v"):
            cache, exps = st[x + "_cache"], st[x + "_exp"]
            if kind == "write":
                _write(st[x + "_new"].float()[some], st["slots"][some], cache, exps)
            val = _gather(cache, exps, at // page, at % page).to(st["out_dtype"])
            out = st[x + "_out"]
            out.copy_(torch.where(keep.view(-1, 1, 1), val, out))
        return st["k_out"], st["v_out"]
    h, hq, w, sinks = case["hkv"], case["hq"], case["window"], case["sinks"]
    g = hq // h
    sm = 1.0 / math.sqrt(D)
    q0 = 0
    for b, L in enumerate(st["lens"]):
        n = st["qs"][b]
        first = 0 if w == 0 else max(0, L - n - w + 1)          # before it only sinks are seen
        t = torch.arange(L, device="cuda")
        t = t[(t >= first) | (t < sinks)]
        pg, row = st["block_table"][b, t // page].long(), t % page
        k = _gather(st["k_cache"], st["k_exp"], pg, row)
        v = _gather(st["v_cache"], st["v_exp"], pg, row)
        q = st["q"][q0:q0 + n].float().view(n, h, g, D) * sm
        mask = None
        if n > 1:
            p = torch.arange(L - n, L, device="cuda").view(n, 1, 1)
            m = t.view(1, 1, -1) <= p
            if w:
                m = m & ((t.view(1, 1, -1) > p - w) | (t.view(1, 1, -1) < sinks))
            mask = m.expand(n, g, -1).reshape(n * g, -1)
        for i in range(h):
            o = _attend(q[:, i].reshape(n * g, D), k[:, i], v[:, i], mask)
            st["out"][q0:q0 + n].view(n, h, g, D)[:, i] = o.view(n, g, D).to(st["out_dtype"])
        q0 += n
    return st["out"]


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _e4m3_grid():
    """The 127 values of codes 0 .. 126."""
    return [math.ldexp(c & 7, -9) if c < 8 else math.ldexp(8 + (c & 7), (c >> 3) - 10) for c in range(127)]


def _nearest(x):
    """E4M3's value nearest to x, a tie to the even code, beyond 448 +-448."""
    grid = torch.tensor(_e4m3_grid(), dtype=torch.float64, device=x.device)
    a = x.abs()
    i = torch.searchsorted(grid, a).clamp_(max=126)             # the first value >= a
    lo, hi = (i - 1).clamp_(min=0), i
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.where(x < 0, -grid[pick], grid[pick])


def _exact_rows(cache, exps, slots):
    """Values of the rows at `slots`, [tokens, heads, 128], one by one from their bytes."""
    pages, h, page, _ = cache.shape
    grid = _e4m3_grid() + [math.nan]
    lut = torch.tensor(grid + [-v for v in grid], dtype=torch.float64, device=cache.device)
    heads = torch.arange(h, device=cache.device)
    row = ((slots // page).view(-1, 1) * h + heads) * page + (slots % page).view(-1, 1)
    c = cache.reshape(-1)[row.unsqueeze(-1) * D + torch.arange(D, device=cache.device)]
    x = exps.reshape(-1)[row // BLOCK].double() - 127.0
    return lut[c.long()] * torch.exp2(x).unsqueeze(-1)


def _exact_write(st, x):
    """The values at st["back"] after the write."""
    slots = st["slots"][st["slots"] >= 0].tolist()
    new = st[x + "_new"][st["slots"] >= 0].double()
    back = st["back"][st["back"] >= 0].tolist()
    old = _exact_rows(st[x + "_cache"], st[x + "_exp"], torch.tensor(back, device=new.device))
    was = st[x + "_exp"].permute(0, 2, 1).reshape(-1, new.shape[1]).double() - 127.0
    groups = {}
    for i, s in enumerate(slots):
        groups.setdefault(s // BLOCK, []).append((s, i))
    at = {s: i for i, s in enumerate(slots)}
    ids = {b: n for n, b in enumerate(groups)}
    member = torch.tensor([ids[s // BLOCK] for s in slots], device=new.device)
    top = torch.zeros((len(ids), new.shape[1]), dtype=torch.float64, device=new.device)
    top = top.scatter_reduce(0, member.unsqueeze(1).expand(-1, new.shape[1]), new.abs().amax(-1), "amax")
    e = torch.ceil(torch.log2(top / 448.0).clamp(-200.0, 200.0))
    e = e + (448.0 * torch.exp2(e) < top).double() - (448.0 * torch.exp2(e - 1.0) >= top).double()
    e = e.clamp(-117.0, 119.0)
    begun = torch.tensor([any(s % BLOCK == 0 for s, _ in g) for g in groups.values()], device=new.device)
    kept = was[torch.tensor(list(groups), device=new.device)]
    e = torch.where(begun.unsqueeze(1), e, torch.maximum(e, kept))
    which = torch.tensor([ids.get(s // BLOCK, -1) for s in back], device=new.device)
    source = torch.tensor([at.get(s, -1) for s in back], device=new.device)
    value = torch.where((source >= 0).view(-1, 1, 1), new[source.clamp(min=0)], old)
    step = torch.exp2(e)[which.clamp(min=0)].unsqueeze(-1)
    return torch.where((which >= 0).view(-1, 1, 1), _nearest(value / step) * step, old)


def _exact_plan(case, st):
    page = case["page"]
    past, new = st["past"].tolist(), st["new"].tolist()
    table, pool = st["block_table"].cpu().numpy(), st["pool"].cpu().numpy()
    free = pool[4:4 + pool[0]].tolist()
    slots = np.full(st["slots"].numel(), -1, dtype=np.int64)
    positions = np.zeros(st["slots"].numel(), dtype=np.int32)
    cu = [0]
    for b, (p, n) in enumerate(zip(past, new)):
        for i in range((p + page - 1) // page, (p + n + page - 1) // page):
            table[b, i] = free.pop()
        pos = np.arange(p, p + n)
        slots[cu[-1]:cu[-1] + n] = table[b, pos // page].astype(np.int64) * page + pos % page
        positions[cu[-1]:cu[-1] + n] = pos
        cu.append(cu[-1] + n)
    lens = np.array([p + n for p, n in zip(past, new)], dtype=np.int32)
    parts = (table, lens, np.array(cu, dtype=np.int32), slots, positions, pool)
    return tuple(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in parts)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "plan":
        return _exact_plan(case, st)
    if case["kind"] in ("write", "read"):
        keep = st["back"] >= 0
        res = []
        for x in ("k", "v"):
            full = torch.zeros(st[x + "_out"].shape, dtype=torch.float64, device="cuda")
            if case["kind"] == "write":
                full[keep] = _exact_write(st, x)
            else:
                for a in range(0, keep.numel(), 16384):
                    part = keep[a:a + 16384]
                    full[a:a + 16384][part] = _exact_rows(st[x + "_cache"], st[x + "_exp"],
                                                          st["back"][a:a + 16384][part])
            res.append(full)
        return tuple(res)
    if work(case)["flops"] > 6e12:
        return None
    page, h, hq, w, sinks = case["page"], case["hkv"], case["hq"], case["window"], case["sinks"]
    g = hq // h
    out = torch.empty(st["out"].shape, dtype=torch.float64, device="cuda")
    q0 = 0
    for b, L in enumerate(st["lens"]):
        n = st["qs"][b]
        pos = torch.arange(L, device="cuda")
        slots = st["block_table"][b].long()[pos // page] * page + pos % page
        for i in range(h):
            rows = []
            for x in ("k", "v"):
                cache, exps = st[x + "_cache"][:, i:i + 1], st[x + "_exp"][:, i:i + 1]
                rows.append(_exact_rows(cache.contiguous(), exps.contiguous(), slots)[:, 0])
            k, v = rows
            for r0 in range(0, n, 512):
                r1 = min(n, r0 + 512)
                q = st["q"][q0 + r0:q0 + r1, i * g:(i + 1) * g].double()
                s = torch.einsum("cgd,td->cgt", q, k) / math.sqrt(D)
                p = torch.arange(L - n + r0, L - n + r1, device="cuda").view(-1, 1)
                hide = pos.view(1, -1) > p
                if w:
                    hide |= (pos.view(1, -1) <= p - w) & (pos.view(1, -1) >= sinks)
                s.masked_fill_(hide.unsqueeze(1), -math.inf)
                prob = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
                out[q0 + r0:q0 + r1, i * g:(i + 1) * g] = torch.einsum("cgt,td->cgd", prob, v)
        q0 += n
    return out
