"""The order of shared memory's single values (CPU: the source is read): none is
read and written between two barriers of the kernel, for a warp may be late to
its read when another one is at its write."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mamba_selective_state_gb300", "csrc")


def kernel_and_values(name):
    """The kernel's text without comments, and the names of the single values of
    its struct of shared memory."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    struct = re.search(r"struct Shared \{(.*?)\n\};", text, re.S).group(1)
    values = []
    for line in struct.split(";"):
        got = re.fullmatch(r"\s*(?:float|int|unsigned long long)\s+(\w+(?:\s*,\s*\w+)*)\s*", line)
        values += re.findall(r"\w+", got.group(1)) if got else []
    kernel = next(k for k in text.split("__global__")[1:] if "Shared<" in k)
    return kernel[:kernel.index("\n}\n")], values


def clashes(kernel, values):
    for part in re.split(r"__syncthreads\(\)|cluster\.sync\(\)", kernel):
        for v in values:
            written = re.search(rf"&sh\.{v}\b|\bsh\.{v}\s*=(?!=)", part)
            read = re.search(rf"(?<!&)\bsh\.{v}\b(?!\s*=(?!=))", part)
            if written and read:
                yield v


def test_the_check_itself():
    assert list(clashes("a = sh.n; f(sh.m); sh.n = 0; __syncthreads(); sh.m = 1;", ["n", "m"])) == ["n"]
    assert list(clashes("x[atomicAdd(&sh.n, 1)] = 2; if (sh.n == 3) f();", ["n"])) == ["n"]
    assert not list(clashes("sh.n = sh.m = 0; __syncthreads(); if (sh.n == sh.m) f();", ["n", "m"]))


@pytest.mark.parametrize("name", ["k_token_logprobs.cu"])
def test_no_value_is_read_and_written_between_two_barriers(name):
    kernel, values = kernel_and_values(name)
    assert {"bound", "owners", "count", "near"} <= set(values)
    assert not list(clashes(kernel, values))
