"""Codes of waits that run out: each has a name, no two the same one, and a kernel reports its own kind's."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dit_transformer_block_gb300", "csrc")


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_every_code_has_a_number_and_a_name_of_its_own():
    codes = dict(re.findall(r"(ERR_WAIT_\w+) = (0x[0-9a-f]+)", read("h3_ptx.cuh")))
    names = dict(re.findall(r'case (ERR_WAIT_\w+): return "([^"]+)"', read("h3_abi.cu")))
    assert codes.keys() == names.keys()
    assert len(set(codes.values())) == len(codes) and len(set(names.values())) == len(names)


def test_kernels_report_their_own_kind():
    kinds = {"h3_gemm.cu": {"GEMM"}, "h3_fp4_gemm.cu": {"GEMM"}, "h3_blocks.cu": {"POOL", "SCORES"},
             "h3_attention.cu": {"ATTN"}, "h3_attention_tiles.cu": {"ATTN"}, "h3_block_attention.cu": {"ATTN"},
             "h3_paged_attention.cu": {"ATTN"}, "h3_abi.cu": {"GEMM", "ATTN", "POOL", "SCORES", "PROBE"}}
    for name in os.listdir(CSRC):
        if name.endswith(".cu"):
            found = {k for k in re.findall(r"ERR_WAIT_([A-Z]+)", read(name))}
            assert found == kinds.get(name, set()), name
