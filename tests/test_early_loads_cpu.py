"""Kernels that begin before the one in front of them has ended read what is
older past L1 (its lines are only known to be current behind the kernel's own
wait). No run shows a load that breaks the rule for certain, so it is checked in
the sources: what stands in front of the wait, and what is called there."""
import os
import re

import pytest

from w4a8_quantized_gemm_gb300 import builder


def source(name):
    with open(os.path.join(builder.CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def before_the_wait(text, kernel):
    """The kernel's body up to where it waits and lets the next one begin."""
    start = re.search(r"\b%s\(const [\w:]*Params p\) \{" % kernel, text).end()
    return text[start:re.compile(r"griddep_wait\(\);\s*if \(threadIdx\.x == 0\) "
                                 r"griddep_launch_dependents\(\);").search(text, start).start()]


@pytest.mark.parametrize("file,kernel", [
    ("lora.cu", "lora_expand_kernel"), ("experts.cu", "experts_down_kernel"),
    ("experts.cu", "experts_few_down_kernel")])
def test_loads_in_front_of_the_wait_are_past_l1(file, kernel):
    body = before_the_wait(source(file), kernel)
    assert "__ldcg" in body or "FewPicks" in body
    assert not re.search(r"__ldg|\*\s*reinterpret_cast<const", body)


def test_copies_that_prime_the_rings_are_past_l1():
    for file in ("experts.cu", "lora.cu"):
        assert "cp.async.c" in source(file)
        assert "cp.async.ca" not in source(file)


def test_the_adapters_kernel_that_may_be_early_reads_past_l1_throughout():
    text = source("lora.cu")
    body = text[text.index("lora_kernel(const LoraParams p) {"):
                text.index("constexpr int kShrinkWarps")]
    assert "p.beside" in body and "__ldcg" in body
    assert "__ldg" not in body.split("if (set < 0) {")[0]
    steps = text[text.index("void shrink_steps("):text.index("uint4 add_row(")]
    assert "__ldcg" in steps and "__ldg" not in steps
