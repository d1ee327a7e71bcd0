"""Shared-memory arrays of narrow elements that a kernel also reads or writes in wider pieces say so in their
declaration: nothing else fixes where the compiler puts them."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "vocabulary_label_bce_b200", "csrc")


def kernels():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = open(os.path.join(CSRC, name)).read()
            for body in re.split(r"(?=\n__global__ |\ntemplate <)", text):
                yield name, body


def test_narrow_arrays_that_are_read_wide_are_aligned():
    seen = 0
    for name, body in kernels():
        for m in re.finditer(r"__shared__ ((?:__align__\(16\) )?)(uint8_t|uint16_t)\s+(\w+)(\[|;)", body):
            var = m.group(3)
            wide = re.search(r"reinterpret_cast<(?!uintptr_t)[\w ]+\*>\(&?" + var + r"\b", body)
            by_hand = re.search(r"reinterpret_cast<uintptr_t>\(" + var + r"\)", body)     # rounded up by the kernel
            if wide and not by_hand:
                seen += 1
                assert m.group(1), f"{name}: {var} is read in wider pieces without an alignment"
    assert seen >= 2
