"""Calls of the block-scaled cache and of the page plan directly behind a kernel that lets
the next one in before it writes: whatever they read (lengths, offsets, tables, slots,
pages, the pool), they read it after that kernel has ended, in every kernel of the call."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from paged_fp8_kv_03_gb300 import build as _build

pytestmark = pytest.mark.gpu

B, H, G, P, PAGES, ENTRIES, ROWS, MAX_Q, MAX_KV = 4, 2, 4, 16, 260, 100, 90, 48, 1500
DELAY_NS = 40000


@pytest.fixture(scope="module")
def late_copy(cuda_device, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("late") / "late_copy.so")
    subprocess.run([_build._nvcc(), *_build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o", out,
                    str(_build.ROOT) + "/tests/late_copy.cu"], check=True)
    fn = ctypes.CDLL(out).late_copy
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_ulonglong, ctypes.c_void_p]

    def run(src, dst):
        assert fn(src.data_ptr(), dst.data_ptr(), src.numel() // 16, DELAY_NS, torch.cuda.current_stream().cuda_stream) == 0

    return run


SHAPES = {
    "past": ((B,), torch.int32), "new": ((B,), torch.int32), "lens": ((B,), torch.int32), "cu": ((B + 1,), torch.int32),
    "sizes": ((B,), torch.int32), "table": ((B, ENTRIES), torch.int32), "pool": ((4 + PAGES,), torch.int32),
    "slots": ((ROWS,), torch.int64), "positions": ((ROWS,), torch.int32),
    "k": ((ROWS, H, 128), torch.bfloat16), "v": ((ROWS, H, 128), torch.bfloat16),
    "q": ((ROWS, H * G, 128), torch.bfloat16),
    "kc": ((PAGES, H, P, 128), torch.uint8), "vc": ((PAGES, H, P, 128), torch.uint8),
    "ke": ((PAGES, H, P // 16), torch.uint8), "ve": ((PAGES, H, P // 16), torch.uint8),
}


class Arena:
    """Everything that the calls read, in one piece of memory."""

    def __init__(self, dev):
        at, places = 0, {}
        for name, (shape, dtype) in SHAPES.items():
            n = int(np.prod(shape)) * dtype.itemsize
            places[name] = (at, n)
            at = (at + n + 255) // 256 * 256
        self.bytes = torch.zeros(at, dtype=torch.uint8, device=dev)
        for name, (shape, dtype) in SHAPES.items():
            a, n = places[name]
            setattr(self, name, self.bytes[a:a + n].view(dtype).view(shape))
        self.pools = (self.kc, self.vc, self.ke, self.ve)

    def fill(self, seed, lens, ns):
        """Contents that are valid by themselves: sequences of these lengths, of which the last ns
        tokens are queries (and new ones, of the plan and of the append)."""
        rng = np.random.default_rng(seed)
        pages = [(L + P - 1) // P for L in lens]
        order = rng.permutation(PAGES)
        table = np.full((B, ENTRIES), 0, np.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        cu = np.concatenate(([0], np.cumsum(ns)))
        slots = np.full(ROWS, -1, np.int64)
        for b, (L, n) in enumerate(zip(lens, ns)):
            t = np.arange(L - n, L)
            slots[cu[b]:cu[b + 1]] = table[b, t // P].astype(np.int64) * P + t % P
        codes = [rng.integers(0, 0x7F, (PAGES, H, P, 128)) | (rng.integers(0, 2, (PAGES, H, P, 128)) << 7) for _ in range(2)]
        free = PAGES - at
        pool = np.concatenate(([free, 0, 0, 0], order[at:], np.zeros(at, np.int64)))
        values = {
            "past": np.array(lens) - ns, "new": ns, "lens": lens, "cu": cu, "sizes": [P] * B, "table": table, "pool": pool,
            "slots": slots, "positions": np.zeros(ROWS), "kc": codes[0], "vc": codes[1],
            "ke": rng.integers(118, 126, (PAGES, H, P // 16)), "ve": rng.integers(118, 126, (PAGES, H, P // 16)),
            **{n: rng.standard_normal(SHAPES[n][0]) for n in ("k", "v", "q")},
        }
        for name, x in values.items():
            getattr(self, name).copy_(torch.from_numpy(np.ascontiguousarray(x)))
        return self


STALE = (1, [900, 1100, 20, 300], [10, 40, 8, 1])
FRESH = (2, [1400, 700, 33, 1], [33, 20, 5, 1])

CALLS = {
    "append": lambda pkv, a, out, e, ws: pkv.kv_append_fp8b(a.k, a.v, a.slots, *a.pools, e),
    "read": lambda pkv, a, out, e, ws: pkv.kv_read_fp8b(a.slots, *a.pools, a.k, a.v, device_error=e),
    "plan": lambda pkv, a, out, e, ws: pkv.plan_pages(a.past, a.new, a.table, a.pool, P, seq_lens=a.past, cu_q=a.cu,
                                                      slot_mapping=a.slots, positions=a.positions, device_error=e),
    "release": lambda pkv, a, out, e, ws: pkv.release_pages(a.lens, a.table, a.pool, P, keep_lens=a.new, device_error=e),
}


def _decode(max_ctas=0, **kw):
    return lambda pkv, a, out, e, ws: pkv.paged_gqa_decode_fp8b(
        a.q[:B], *a.pools, a.table, a.lens, out=out[:B], workspace=ws, device_error=e, max_ctas=max_ctas, max_seq_len=MAX_KV,
        seq_page_sizes=a.sizes, **kw)


def _prefill(bound=MAX_KV, max_q=MAX_Q, **kw):
    return lambda pkv, a, out, e, ws: pkv.paged_prefill_fp8b(
        a.q, a.cu, *a.pools, a.table, a.lens, max_q, out=out, max_kv_len=bound, workspace=ws, device_error=e,
        seq_page_sizes=a.sizes, **kw)


def _case(call, dtype, work=None):
    return (call, dtype, work)


CASES = {
    **{name: _case(call, torch.float32) for name, call in CALLS.items()},
    **{f"decode {d} {m} {w}": _case(_decode(m, window=w, sinks=3), t, lambda pkv, m=m: pkv.pkv_decode_fp8b_workspace_size(
        B, H * G, H, max_seq_len=MAX_KV, max_ctas=m))
       for d, t in (("bf16", torch.bfloat16), ("f32", torch.float32)) for m in (0, 5) for w in (0, 200)},
    # a CTA a query tile without and with a window, keys shared among CTAs, the cache read by the attention itself
    **{f"prefill {d} {n} {m} {w}": _case(_prefill(n, m, window=w, sinks=3), t,
                                         lambda pkv, n=n, m=m, w=w: pkv.pkv_prefill_fp8b_workspace_size(B, H, m, n, 0, w, 3))
       for d, t in (("bf16", torch.bfloat16), ("f32", torch.float32))
       for n, m, w in ((MAX_KV, 640, 0), (MAX_KV, MAX_Q, 200), (MAX_KV, MAX_Q, 0), (MAX_KV, MAX_Q, 1200), (200000, MAX_Q, 0))},
}


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_reads_what_a_late_producer_writes(pkv, cuda_device, late_copy, name, captured):
    call, dtype, work = CASES[name]
    dev = cuda_device
    a = Arena(dev)
    stale = a.fill(*STALE).bytes.clone()
    fresh = a.fill(*FRESH).bytes.clone()
    out = torch.full((ROWS, H * G, 128), 9.0, dtype=dtype, device=dev)
    e = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.empty(work(pkv), dtype=torch.uint8, device=dev) if work else None

    def results():
        torch.cuda.synchronize()
        got = (a.bytes.clone(), out.clone(), int(e.item()))
        out.fill_(9.0)
        torch.cuda.synchronize()
        return got

    # (once on either contents, with a synchronisation between producer and call)
    wants = []
    for x in (stale, fresh):
        a.bytes.copy_(x)
        torch.cuda.synchronize()
        call(pkv, a, out, e, ws)
        wants.append(results())
    assert wants[0][2] == 0 and wants[1][2] == 0
    assert not (torch.equal(wants[0][0], wants[1][0]) and torch.equal(wants[0][1], wants[1][1]))
    run = lambda: (late_copy(fresh, a.bytes), call(pkv, a, out, e, ws))
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(5):
        a.bytes.copy_(stale)
        torch.cuda.synchronize()
        run()
        got = results()
        assert got[2] == 0
        assert torch.equal(got[0], wants[1][0]) and torch.equal(got[1], wants[1][1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bound", [MAX_KV, 200000])
def test_prefill_behind_a_plan_of_other_lengths(pkv, cuda_device, bound, dtype):
    """Plan, append and prefill in one graph, whose lengths, offsets and tables are others in every
    replay: as with a synchronisation between any two of the calls."""
    dev = cuda_device
    a = Arena(dev)
    out = torch.empty((ROWS, H * G, 128), dtype=dtype, device=dev)
    e = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.empty(pkv.pkv_prefill_fp8b_workspace_size(B, H, MAX_Q, bound), dtype=torch.uint8, device=dev)
    steps = [lambda: pkv.plan_pages(a.past, a.new, a.table, a.pool, P, seq_lens=a.lens, cu_q=a.cu, slot_mapping=a.slots,
                                    positions=a.positions, device_error=e),
             lambda: _prefill(bound)(pkv, a, out, e, ws),
             lambda: pkv.kv_append_fp8b(a.k, a.v, a.slots, *a.pools, e),
             lambda: pkv.plan_pages(a.past, a.new, a.table, a.pool, P, seq_lens=a.lens, cu_q=a.cu, slot_mapping=a.slots,
                                    positions=a.positions, device_error=e),
             lambda: _prefill(bound)(pkv, a, out, e, ws)]
    a.fill(*STALE)
    for s in steps:
        s()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for s in steps:
            s()
    rng = np.random.default_rng(7)
    for seed in range(3, 11):
        ns = [int(n) for n in rng.integers(0, 22, B)]
        contents = (seed, [int(n + x) for n, x in zip(ns, rng.integers(1, 700, B))], ns)
        got = []
        for apart in (True, False):
            a.fill(*contents)
            out.fill_(9.0)
            torch.cuda.synchronize()
            if apart:
                for s in steps:
                    s()
                    torch.cuda.synchronize()
            else:
                g.replay()
            torch.cuda.synchronize()
            got.append((a.bytes.clone(), out.clone()))
        assert int(e.item()) == 0
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
