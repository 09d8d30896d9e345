"""What the attention kernels wait for, read from their source (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_sharded_linear_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels():
    """(file, body) of every kernel that is launched before the one ahead of it has ended."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")) or name == "heads_sm103.cuh":
            continue
        for part in code(name).split("__global__")[1:]:
            if "wait_for_previous_kernel();" in part:
                yield name, part


def test_tensor_memory_is_taken_after_the_kernel_before_has_ended():
    """A CTA that held tensor memory while waiting could keep a CTA of that kernel from its own: neither would end."""
    seen = 0
    for name, body in kernels():
        at = body.find("tcgen05.alloc")
        if at >= 0:
            seen += 1
            assert body.find("wait_for_previous_kernel();") < at, name
    assert seen == 1
