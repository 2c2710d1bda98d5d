"""The rules of chained launches (csrc/chain.cuh), checked on the sources: breaking one is a
hang or a stale read that no run is sure to show."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_self_b200", "csrc")


def kernels():
    """(file, name, body) of every __global__ function, comments taken out."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", text):
            at = text.index("{", text.index(")", m.end()))
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield os.path.basename(path), m.group(1), text[at:end]


KERNELS = list(kernels())


def test_the_kernels_are_found():
    names = {k[1] for k in KERNELS}
    assert {"bwd_dq_kernel", "bwd_dkv_kernel", "attn_pp_kernel", "row_stats_kernel", "list_bits_kernel",
            "dbias_kernel"} <= names


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[f"{f}-{n}" for f, n, _ in KERNELS])
def test_tensor_memory_is_held_before_the_next_kernel_is_released(file, name, body):
    """A CTA of the next kernel must not take tensor memory that this kernel still has to allocate."""
    if "grid_release()" not in body or "tmem_alloc(" not in body:
        return
    alloc, release = body.rindex("tmem_alloc("), body.index("grid_release()")
    assert alloc < release
    # the allocating warp is one of several: all threads have to know that it is done
    assert "__syncthreads()" in body[alloc:release]


# what the kernels of a chain hand to one another, by the names that the readers use
HANDED_ON = r"nlse|ndelta|slack|valid|km|kmean|off|offsets|bits|part|tab|bm|t_off|t_rows"


@pytest.mark.parametrize("file", ["attention_pp.cu", "backward.cu", "backward_dkv.cu", "backward_dq.cu",
                                  "relative_bias.cu", "relative_bias.cuh", "transpose_lists.cu"])
def test_what_the_chain_wrote_is_not_read_as_constant(file):
    """A read-only load may be moved across the wait for the kernel that writes the value."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    for m in re.finditer(r"__ldg\(([^;]*);", text):
        assert not re.search(r"\b(%s)\b" % HANDED_ON, m.group(1)), m.group(0)
    assert not re.search(r"const[^,()]*__restrict__ (%s)\b" % HANDED_ON, text)
    if file == "backward_dkv.cu":  # the transposed lists
        assert "__ldg(list" not in text


def test_the_dq_epilogue_waits_for_a_barrier_of_one_phase():
    """dq_done completes a phase per tile; a thread that has not followed every phase must not wait on its parity."""
    (body,) = (b for f, n, b in KERNELS if n == "bwd_dq_kernel")
    work = body[body.index("row_sum"):]     # the element-wise warps' part
    assert "mbar_wait(mma_done, 0" in work and "mbar_wait(dq_done" not in work
    assert body.count("umma_commit(mma_done)") == 1
