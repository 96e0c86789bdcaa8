"""Kernels that are launched before the one ahead in the stream has ended read what it may have written with coherent loads (no
GPU needed: the sources are read)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_quant_memory_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


EARLY = ["fq_append.cu", "fq_attention.cu", "fq_extend.cu", "fq_matmul.cuh", "fq_sample.cu"]


def test_the_list_names_every_early_launch_of_the_serving_operators():
    files = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and "launch_overlapped(" in source(f)]
    assert files == EARLY


@pytest.mark.parametrize("name", EARLY)
def test_no_input_takes_the_non_coherent_path(name):
    """__ldg and ld.global.nc are for data that does not change while the kernel lives: here a table in the program alone."""
    text = source(name)
    assert "global.nc" not in text
    assert [m for m in re.findall(r"__ldg\(([^)]*)\)", text) if not m.startswith("&kPowers.")] == []


def test_streamed_inputs_are_read_coherently():
    body = re.search(r"uint4 ld_stream16\(.*?\n}", source("fq_device.cuh"), re.S).group()
    assert "ld.global" in body and ".nc" not in body
