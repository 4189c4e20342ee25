"""Kernels that are brought onto the GPU before what is ahead of them has ended: how their
sources read what that may write."""
import os
import re

from paged_fp8_kv_03_gb300 import build

# All of these files' kernels, or the device functions that they share with others.
EARLY = ["rows_fp8b.cu", "pages.cu", "decode_fp8b.cu", "prefill_fp8b.cu", "prefill_direct.cu", "widen_fp8b.cuh", "split.cuh"]
# Instances of kernels that are launched early are among these files' too: there only the scales a
# kv head, which no early kernel takes, may be read so, and what other instances (not kBlocks) read.
SHARED = ["prefill.cuh", "list.cuh"]


def _source(name):
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_read_only_loads_behind_the_wait():
    for name in EARLY:
        assert "__ldg" not in _source(name), name
    for name in SHARED:
        assert all("_scale + h" in line or "kBlocks ? __ldcg(p) : __ldg(p)" in line
                   for line in _source(name).split("\n") if "__ldg" in line), name
    walk = _source("internal.h")
    assert "seq_token_page" in walk and "__ldg" not in walk


def _kernel(text, name):
    """A kernel's body, from its opening brace to the next line that is only a closing one."""
    at = re.search(name + r"\([^{;]*\)\s*\{", text).end()
    return text[at:text.index("\n}\n", at)]


def test_the_wait_comes_before_any_read():
    """Ahead of grid_wait(): nothing but arithmetic on launch indices and sizes."""
    kernels = {"prefill.cu": ["paged_prefill_kernel"], "prefill_fp4.cu": ["paged_prefill_pair_kernel"],
               "prefill_direct.cu": ["paged_prefill_direct_kernel"],
               "prefill_fp8b.cu": ["kv_refs_fp8b_kernel", "kv_widen_fp8b_kernel", "prefill_join_fp8b_kernel"],
               "rows_fp8b.cu": ["kv_append_fp8b_kernel", "kv_read_fp8b_kernel"],
               "pages.cu": ["plan_pages_kernel", "release_pages_kernel"],
               "decode_fp8b.cu": ["paged_gqa_decode_fp8b_kernel", "paged_gqa_decode_fp8b_cluster_kernel"],
               "list.cuh": ["join_kernel", "join_cut_kernel"]}
    inputs = r"cu_q|seq_lens|tile_off|page_sizes|block_table|slots|k_exp|v_exp|v_refs|joins|firsts|a\.pool\b|a\.past|a\.fresh"
    for name, kernel in ((f, k) for f, ks in kernels.items() for k in ks):
        body = _kernel(_source(name), kernel)
        ahead = body[:body.index("grid_wait()")]
        assert not re.search(inputs, ahead) and "__ldg" not in ahead, (kernel, ahead)
