"""Kernels that are launched as dependents of one another (programmatic launches) are resident while the kernel before
them still writes.  What that kernel writes must be read by ordinary loads after the wait: __ldg and const __restrict__
allow non-coherent loads, which are for memory that nobody writes during the kernel and may be moved above the wait.
A race cannot be shown by running it, so the sources are read here."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "scale_only_quantization_gb300", "csrc")
WAIT = r"wait_for_previous\(\)|griddepcontrol\.wait"
# what an earlier kernel of a chain writes, by the names it goes by in the dependent kernels
CHAIN = {"head.cu": ("ref", "mul", "tval", "tcol", "target", "zt", "psum", "pmax", "u", "ur", "at", "p", "gate", "list", "asked"),
         "norm.cu": ("part", "status")}
OF_THE_CALLER = ("target", "g", "w", "h")  # parameters of plain kernels: inputs, read-only during the whole call


def kernels(text):
    """(signature, body) of every __global__ function."""
    for m in re.finditer(r"__global__", text):
        brace = text.index("{", m.start())
        depth, i = 0, brace
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        yield text[m.start():brace], text[brace:i]


@pytest.mark.parametrize("name", sorted(CHAIN))
def test_results_of_the_kernel_before_are_read_coherently(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    dependents = [(s, b) for s, b in kernels(text) if re.search(WAIT, b)]
    assert dependents
    for sig, body in dependents:
        for param in re.findall(r"__restrict__\s*(\w+)", sig):
            assert param in OF_THE_CALLER, (param, sig[:60])
        for arg in re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?([\w.]+)", body):
            assert arg.split(".")[-1] not in CHAIN[name] and not arg.startswith("p."), arg
    # device functions that take the chain's parameters as a struct
    for fn in re.findall(r"__ldg\(\s*(p\.\w+)", text) if name == "head.cu" else ():
        raise AssertionError("%s is written by an earlier kernel of the chain" % fn)


def test_every_dependent_kernel_is_listed():
    """A file that starts to launch dependents has to be looked at here."""
    found = {f for f in os.listdir(CSRC) if f.endswith(".cu") and re.search(WAIT, open(os.path.join(CSRC, f)).read())}
    assert found == set(CHAIN)
