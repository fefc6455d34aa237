"""Kernels that are launched to overlap their predecessor on the stream read what it may still be writing. They have to
wait for it first, and to read with ordinary loads: a non-coherent load (__ldg, ld.global.nc, or a load through a
const __restrict__ pointer, which the compiler may turn into one) is allowed only for memory that nobody writes
while the kernel is resident, and nothing keeps it behind the wait. Checked in the source; nothing is launched."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_gemm_moe_b200", "csrc")
NON_COHERENT = re.compile(r"__ldg\s*\(|\.nc\b|\bconst\s+\w+\s*\*\s*(?:const\s+)?__restrict__")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# every file whose kernels launch_dependent starts
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "launch_dependent(" in source(f))


def test_the_files_are_found():
    assert {"k_norm.cu", "k_mx4.cu", "k_mx4gemm.cu"} <= set(FILES)


@pytest.mark.parametrize("name", FILES)
def test_no_non_coherent_loads(name):
    src = source(name)
    found = [src[:m.start()].count("\n") + 1 for m in NON_COHERENT.finditer(src)]
    assert not found, f"{name}: non-coherent loads at lines {found}"


@pytest.mark.parametrize("name", FILES)
def test_every_kernel_waits_before_it_releases(name):
    """Each kernel waits for its predecessor, and none releases its successor before that."""
    kernels = re.split(r"\b__global__\b", source(name))[1:]
    assert kernels
    for k in kernels:
        wait, release = k.find("grid_dep_wait()"), k.find("grid_dep_launch()")
        assert wait >= 0 and (release < 0 or wait < release)


@pytest.mark.parametrize("text,bad", [
    ("x = __ldg(p);", True), ("x = *p;", False), ("void f(const float* __restrict__ s)", True), ("void f(float* __restrict__ s)", False),
    ('asm("ld.global.nc.v4.u32")', True), ("void f(const float* s, float* __restrict__ y)", False),
])
def test_the_pattern(text, bad):
    assert bool(NON_COHERENT.search(text)) == bad
