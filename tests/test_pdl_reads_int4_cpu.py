"""The read rule of kernels launched with programmatic dependent launch (nothing of
the kernel before is read ahead of griddepcontrol.wait, nor through __ldg or a const
__restrict__ pointer), over every kernel the library launches so: the list is taken
from the launches, conditional ones among them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "head_latent_attention_10_b200", "csrc")
# kernel: its file, and the words by which its body names memory that other kernels write
KERNELS = {
    "tc_decode64_kernel": ("tc_decode64.cuh", ("seq_lens", "block_table", "q_abs", "scales", "tma_load")),
    "dec_combine_kernel": ("dec_common.cuh", ("plan +", "flags +", "part_o", "part_lse2", "__ldcg")),
    "tc_decode_int4_kernel": ("tc_decode_int4.cuh", ("seq_lens", "block_table", "q_abs", "codes", "scales", "__ldcg")),
    "dec4_clear_kernel": ("tc_decode_int4.cuh", ("*err",)),
    "dec4_combine_kernel": ("tc_decode_int4.cuh", ("__ldcg", "part_o", "part_lse2", "plan +")),
    "tc_gemm_kernel": ("tc_gemm.cuh", ("tma_load", "factor", "epi(")),
    "tc_prefill_kernel": ("tc_prefill.cuh", ("seq_lens", "max_lat", "max_w", "counter", "tma_load")),
}


def src(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def definition(kernel):
    """(parameter list, body) of the kernel."""
    text = src(KERNELS[kernel][0])
    i = re.search(r"\b" + kernel + r"\(", text).end()
    j = text.index("\n{", i)
    return text[i:j], text[j:text.index("\n}\n", j)]


def test_the_list_is_whole():
    abi = src("mla_abi.cu")
    launched = set()
    for m in re.finditer(r"= launch_pdl\(", abi):
        depth, j = 1, m.end()
        while depth and not (depth == 1 and abi[j] == ","):     # the first argument
            depth += (abi[j] in "(<{") - (abi[j] in ")>}")
            j += 1
        names = re.findall(r"\b(\w+_kernel)\b", abi[m.end():j])
        launched |= set(names) if names else {"tc_gemm_kernel"}
        assert names or abi[m.end():j] == "kern"
    assert "auto kern = tc_gemm_kernel<" in abi and launched == set(KERNELS)


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_nothing_is_read_ahead_of_the_wait(kernel):
    body = definition(kernel)[1]
    before = body[:body.index("pdl_wait()")]
    for word in KERNELS[kernel][1]:
        assert word in body and word not in before, word


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_reads_go_through_l2(kernel):
    params, body = definition(kernel)
    assert "__ldg(" not in body
    for p in re.split(r",(?![^<]*>)", params):
        assert not ("const" in p and "__restrict__" in p), p
