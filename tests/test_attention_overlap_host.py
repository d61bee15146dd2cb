"""Launches of the attention overlap: what one of them writes is never read as
read-only data by another."""
import os
import re

import implicit_gemm_dgrad_gb300 as cdg

CSRC = os.path.join(os.path.dirname(cdg.__file__), "csrc")


def test_only_arguments_of_the_caller_are_read_only():
    for name in ("attention_sm103.cu", "attention_grad_sm103.cu"):
        with open(os.path.join(CSRC, name)) as f:
            assert "__ldg" not in f.read(), name
    with open(os.path.join(CSRC, "attention_device.cuh")) as f:
        loads = re.findall(r"__ldg\((.*)", f.read())
    assert loads and all("offsets" in x for x in loads)
