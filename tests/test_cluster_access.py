"""A block may touch the shared memory of another block of its cluster only once that block is known to run, which a
cluster barrier says: in every kernel the first such access has to stand behind the first wait on one. Read off the source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_tern_gemv_b200", "csrc")


def _functions(text):
    """{name: (whether a kernel, body without comments)} of a source's device functions."""
    text = re.sub(r"//[^\n]*", "", text)
    out = {}
    for m in re.finditer(r"__(device|global)__[^;{}()]*(?:\([^()]*\)[^;{}()]*)*?\b(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*(?:const\s*)?\{", text):
        depth, i = 1, m.end()
        while depth and i < len(text):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out[m.group(2)] = (m.group(1) == "global", text[m.end():i])
    return out


def _closure(functions, found):
    """Names of functions whose body `found` holds for, or that call one of them."""
    names = {n for n, (_, b) in functions.items() if found(b)}
    while True:
        more = {n for n, (kernel, b) in functions.items() if not kernel and n not in names
                and any(re.search(rf"\b{x}\s*[(<]", b) for x in names)}
        if not more:
            return names
        names |= more


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        functions = _functions(open(path).read())
        remote = _closure(functions, lambda b: "mapa.shared::cluster" in b)
        waits = _closure(functions, lambda b: "barrier.cluster.wait" in b)
        for name, (kernel, body) in functions.items():
            first = lambda names: min((m.start() for x in names for m in re.finditer(rf"\b{x}\s*\(", body)), default=None)  # noqa: E731
            if kernel and first(remote) is not None:
                yield os.path.basename(path), name, first(waits), first(remote)


KERNELS = list(_kernels())


def test_the_kernels_with_clusters_are_found():
    assert {k[1] for k in KERNELS} >= {"dz_kernel", "route_kernel", "layer_gemm_kernel"}


@pytest.mark.parametrize("source,kernel,wait,access", KERNELS, ids=[k[1] for k in KERNELS])
def test_other_blocks_are_known_to_run_before_their_memory_is_touched(source, kernel, wait, access):
    assert wait is not None and wait < access
