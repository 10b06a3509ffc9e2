"""Every kernel that is launched as a programmatic dependent ends after the kernel
ahead of it, whatever its inputs (read off the sources, no GPU).

A dependent's wait is for the one kernel ahead of it on the stream.  That one's
end comes after the end of everything before it only if some block of it has
waited in its turn: where all blocks may leave without waiting, the next
dependent can start while kernels further ahead still run.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_quantized_paged_quantize_gb300", "csrc")
WAIT = re.compile(r"griddepcontrol\.wait|after_earlier_kernels\(\);")


def sources():
    return {n: open(os.path.join(CSRC, n)).read() for n in sorted(os.listdir(CSRC)) if n.endswith(".cu")}


def kernels(text):
    """(name, lines of the body) of a file's __global__ functions."""
    for m in re.finditer(r"^__global__ void (?:__launch_bounds__\((?:[^()]|\([^()]*\))*\) )?(\w+)\([^;{]*\) \{\n(.*?)^\}", text, re.M | re.S):
        yield m.group(1), [line for line in (re.sub(r"\s*//.*", "", raw) for raw in m.group(2).split("\n")) if line]


def dependents():
    """(file, kernel, lines) of the kernels that some launch makes programmatic dependents."""
    found = []
    for name, text in sources().items():
        launches = " ".join(re.findall(r"launch_(?:overlapped|dependent)\(([^;]*);", text))
        if "cudaLaunchAttributeProgrammaticStreamSerialization" in text and name == "evict.cu":
            launches += " pack_kernel"
        if re.search(r"launch_dependent\(kernel\b", text):
            launches += " weights_kernel"
        for kernel, lines in kernels(text):
            if re.search(rf"\b{kernel}\b", launches):
                found.append((name, kernel, lines))
    return found


def test_the_dependents_are_found():
    assert {k for _, k, _ in dependents()} == {"plan_kernel", "norm_rope_kernel", "digest_kernel", "scores_kernel", "select_kernel",
                                               "selected_kernel", "decode_kernel", "combine_kernel", "weights_kernel", "pack_kernel"}


@pytest.mark.parametrize("name,kernel", [(n, k) for n, k, _ in dependents()])
def test_some_block_waits(name, kernel):
    lines = next(ls for n, k, ls in dependents() if (n, k) == (name, kernel))
    # (a grid ends with its last block: the first one's wait will do)
    always = [WAIT.search(line) and (not re.match(r"\s*if\b", line) or "|| (blockIdx.x | blockIdx.y) == 0)" in line) for line in lines]
    waited = False                                     # at the body's own level: by every thread that comes there
    for i, line in enumerate(lines):
        level = 4 if kernel == "decode_kernel" and "return" not in (lines + [""])[i + 1] else 2
        waited = waited or (always[i] and re.match(rf" {{2,{level}}}\S", line))
        if re.search(r"\breturn;", line) and not waited:
            assert always[i - 1], f"{name}: {kernel} returns without waiting: {line.strip()}"
    # (decode_kernel's warps with pages wait before the first one: where any block goes on, some warp has pages)
    assert waited
