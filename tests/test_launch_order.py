"""Which kernels let the next one on their stream start early (CPU only: the sources are read).

A product copies its first weights before it waits for the kernels in front of it, so a kernel that writes a weight format,
or a matrix out of one, must not let its successors start."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_split_gb300", "csrc")


def kernels():
    """{name: body} of every __global__ function."""
    found = {}
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", text):
            at = text.index("{", m.end())
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            found[m.group(1)] = text[at:end]
    return found


def calls(body):
    """The lines that let successors start."""
    return [line.split("//")[0].strip() for line in body.splitlines() if "pdl_launch_dependents" in line]


def test_kernels_that_write_weights_hold_their_successors_back():
    every = kernels()
    for name in ("q4_0_quant_kernel", "nf4_quant_kernel", "nf4_dequant_kernel", "nf4_dequant_rows_kernel", "q8_1_dequant_kernel",
                 "kv4_append_kernel", "kv4_read_kernel"):
        assert calls(every[name]) == [], name
