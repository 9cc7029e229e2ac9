"""Rules that the device code keeps and no result shows while the compiler happens to be kind:
read from the sources."""
import os
import re

import pytest

from gradient_sync_zero_gb300 import build as dbuild

FILES = sorted(f for f in os.listdir(dbuild.CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    """A source without comments."""
    with open(os.path.join(dbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def asm_statements(text, instruction):
    """(what precedes it, the statement) of every asm statement that holds the instruction."""
    for m in re.finditer(r"\basm\b[^;]*?\((?:[^\"]|\"[^\"]*\")*?\);", text):
        if instruction in m.group():
            yield text[:m.start()].rstrip(), m.group()


@pytest.mark.parametrize("name", FILES)
def test_whole_warps_reach_cluster_barriers(name):
    """barrier.cluster's aligned form asks for all threads of a warp, which a branch before may have
    parted: each statement has one such barrier and follows __syncwarp()."""
    for before, asm in asm_statements(code(name), "barrier.cluster."):
        assert before.endswith("__syncwarp();"), (name, asm)
        assert asm.count("barrier.cluster.") == 1, (name, asm)


@pytest.mark.parametrize("name", FILES)
def test_whole_warps_load_tensor_memory_and_wait(name):
    """tcgen05.ld asks for the whole warp too, and its registers may be used behind tcgen05.wait::ld only:
    as a statement of its own that wait orders memory accesses, not arithmetic on registers."""
    for before, asm in asm_statements(code(name), "tcgen05.ld."):
        assert before.endswith("__syncwarp();"), (name, asm)
        assert "tcgen05.wait::ld" in asm, (name, asm)
