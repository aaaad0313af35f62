"""Kernels that may be set up while the one before them still runs (launch_early, programmaticStreamSerialization): in
every CTA they wait for that one before they end, whichever way they end. A kernel that ends without waiting lets
whatever follows, which is ordered behind it alone, run beside the kernel it was launched behind. (CPU: the sources.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_79_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def early_kernels(text):
    """Names of the __global__ functions that a file launches early, however they reach the launch."""
    if "launch_early(" not in text and "programmaticStreamSerializationAllowed" not in text:
        return []
    found = re.findall(r"__global__[^{;]*?\b(\w+)\s*\(const", text)
    return [k for k in found if re.search(r"(launch_early\([^;]*|cudaLaunchKernelEx\(&cfg, *)\b" + k + r"\b", text)]


def body(text, kernel):
    at = re.search(r"__global__[^;{]*\b" + kernel + r"\s*\([^{]*\{", text).end()
    depth, end = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end - 1]


def unwaited_exits(code):
    """Exits (returns and the end) that a path without wait_before() may reach. A block starts as its surroundings stand,
    and what it waited for counts behind it only if it stands outside any condition: pessimistic, so no exit is missed."""
    stack, waited, exits = [], False, []
    for m in re.finditer(r"[{}]|\bwait_before\(\);|\breturn\b(?=\s*;)", code):
        t = m.group()
        if t == "{":
            stack.append(waited)
        elif t == "}":
            waited = stack.pop()
        elif t.startswith("wait_before"):
            waited = True
        elif not waited:
            exits.append(code[:m.start()].count("\n"))
    return exits + ([] if waited else ["end"])


EARLY = [(f, k) for f in SOURCES for k in early_kernels(read(f))]


def test_the_early_kernels_are_found():
    assert {k for _, k in EARLY} == {"cache8_fwd_kernel", "cache8_finish_kernel", "cache8_append_kernel",
                                     "cache8_select_kernel", "cache8_gather_kernel"}


@pytest.mark.parametrize("file,kernel", EARLY)
def test_no_cta_ends_without_waiting(file, kernel):
    assert unwaited_exits(body(read(file), kernel)) == []


@pytest.mark.parametrize("file", sorted({f for f, _ in EARLY} | {"fa_cache8.cuh"}))
def test_no_loads_by_the_read_only_path(file):
    """ld.global.nc wants memory that nothing writes while the kernel lives, and an early kernel lives from its set-up on."""
    assert not re.search(r"__ldg|\.nc\b|__restrict__", read(file))


def test_the_reading_of_exits():
    assert unwaited_exits("wait_before(); if (a) return; b();") == []
    assert unwaited_exits("if (a) return; wait_before();") == [0]
    assert unwaited_exits("if (a) { wait_before(); return; }\nif (b) return;\nwait_before();") == [1]
    assert unwaited_exits("if (a) { wait_before(); }") == ["end"]
