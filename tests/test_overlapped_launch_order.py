"""Kernels whose launch overlaps the end of the kernel before them (griddepcontrol): the order
of their waits, allocations and signals, read from the sources. The orders refused here can
stop two kernels for good, so nothing runs them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_block_scaled_08_b200", "csrc")
WAIT, SIGNAL = "wait_for_previous_kernel(", "let_next_kernel_start("


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels():
    """(file:name, body) of every kernel that passes the wait."""
    found = []
    for name in sorted(n for n in os.listdir(CSRC) if n.endswith(".cu")):
        text = code(name)
        for m in re.finditer(r"__global__\b", text):
            open_ = text.index("{", text.index(") {", m.end()))
            depth, end = 1, open_ + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            head, body = text[m.end():open_], text[open_:end]
            if WAIT in body:
                found.append((name + ":" + re.findall(r"(\w+)\s*\(", head)[-1] if "(" in head else name, body))
    return found


KERNELS = kernels()


def test_the_overlapped_kernels_are_found():
    assert len(KERNELS) == 5, [k for k, _ in KERNELS]


@pytest.mark.parametrize("body", [b for _, b in KERNELS], ids=[k for k, _ in KERNELS])
def test_one_wait_and_one_signal(body):
    assert body.count(WAIT) == 1 and body.count(SIGNAL) == 1


@pytest.mark.parametrize("body", [b for _, b in KERNELS] + [code("fp8q_grouped.cuh")],
                         ids=[k for k, _ in KERNELS] + ["fp8q_grouped.cuh"])
def test_no_read_only_loads(body):
    """ld.global.nc is for memory that nobody writes while the kernel runs; these kernels may
    be resident while the one before them still writes. (Forms of a kernel that are not
    launched that way may keep it.)"""
    assert "ld.global.nc" not in body and "ld_nc" not in body
    for line in body.splitlines():
        assert "__ldg" not in line or "kGrouped ? ld_after_wait(" in line, line


@pytest.mark.parametrize("body", [b for _, b in KERNELS if "tmem_alloc" in b],
                         ids=[k for k, b in KERNELS if "tmem_alloc" in b])
def test_tensor_memory_is_allocated_after_the_wait_and_before_the_signal(body):
    """An allocation blocks until the columns are free. Before the wait a kernel could hold
    columns that its predecessor still needs; a kernel that signals first could find the
    columns held by a successor that waits for it."""
    alloc = [m.start() for m in re.finditer(r"tmem_alloc", body)]
    assert len(alloc) == 1
    assert body.index(WAIT) < alloc[0] < body.index(SIGNAL)
    # the whole CTA (pair) has its columns before any thread signals
    assert re.search(r"__syncthreads\(\)|cluster_sync\(\)", body[alloc[0]:body.index(SIGNAL)])
