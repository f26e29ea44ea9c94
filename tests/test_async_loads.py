"""Every kernel that starts asynchronous copies into its shared memory waits for
them (bounded) before it exits, whichever way it leaves its loop: a copy that
lands later would change the memory of the CTA that comes next. A wait that runs
out cannot be staged, so this reads the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_precision_b200", "csrc")
STARTS = re.compile(r"\b(tma_load_\dd\w*|tma_gather4|bulk_load)\(")


def past(text, i, open_, close):
    """The position behind the bracket that matches the one at i."""
    depth = 0
    while True:
        depth += {open_: 1, close: -1}.get(text[i], 0)
        i += 1
        if not depth:
            return i


def functions(text):
    """(name, whether a kernel, body) of every device function."""
    text = re.sub(r"//[^\n]*|__(?:launch_bounds|cluster_dims)__\([^()]*\)", "", text)
    for m in re.finditer(r"__(global|device)__", text):
        i = text.index("(", m.end())
        name, end = text[m.end():i].split()[-1], past(text, i, "(", ")")
        body = re.compile(r"\s*(?:const\s*)?(?=\{)").match(text, end)
        if body:
            yield name, m.group(1) == "global", text[body.end():past(text, body.end(), "{", "}")]


SOURCES = {os.path.basename(f): open(f).read() for f in glob.glob(os.path.join(CSRC, "*.cu*"))}
FUNCTIONS = [(f, *fn) for f, text in SOURCES.items() for fn in functions(text)]
# functions that start copies and wait for them themselves (a producer warp's)
PRODUCERS = {name for _, name, kernel, body in FUNCTIONS if not kernel and STARTS.search(body) and "drain_loads(" in body}
KERNELS = [(f, name, body) for f, name, kernel, body in FUNCTIONS
           if kernel and (STARTS.search(body) or any(p in body for p in PRODUCERS))]


def test_the_kernels_are_found():
    names = {n for _, n, _ in KERNELS}
    assert {"quant_row_kernel", "quant_col_kernel", "quant_col64_kernel", "amax_rowcol64_kernel", "gemm_grouped_kernel",
            "gemm_grouped_single_kernel", "rmsnorm_bwd_ring_kernel"} <= names
    assert sum(t.count("__global__ void") for t in SOURCES.values()) == sum(k for _, _, k, _ in FUNCTIONS)


@pytest.mark.parametrize("file,name", [k[:2] for k in KERNELS])
def test_copies_are_waited_for(file, name):
    body = next(b for f, n, b in KERNELS if (f, n) == (file, name))
    if STARTS.search(body):
        assert "drain_loads(" in body


def test_threads_of_a_cta_leave_at_the_same_row():
    """The ring's flag is set before the barrier of a row and read behind it. A thread that is a row ahead may set it
    while others still read, so rows take turns at two flags."""
    body = next(b for _, n, b in KERNELS if n == "rmsnorm_bwd_ring_kernel")
    uses = re.findall(r"ring\.dead(\[parity\])?", body)
    assert len(uses) == 2 and all(uses)
    assert body.index("ring.dead[parity] = 1") < body.index("__syncthreads()") < body.index("if (ring.dead[parity]) break")
