"""How the tree attention's launches share an SM (CPU: the source is read).

A kernel that is launched beside the one before takes tensor memory before it
waits for that one. A CTA that has none yet must not depend on columns that such
a kernel's CTAs hold, so the permission to start beside is given only once the
columns are held. (How many CTAs fit on an SM is asserted where the kernels are
launched, when they are compiled.)
"""
import os
import re

from prefill_decode_paged_pod_gb300 import _build


def test_the_next_kernel_starts_once_tensor_memory_is_held():
    with open(os.path.join(_build.CSRC, "pod_tree.cuh")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    body = src[src.index("pod_tree_kernel(const __grid_constant__"):]
    body = body[:body.index("cudaError_t launch_tree")]
    alloc = body.index("tmem_alloc(")
    held = body.index("__syncthreads()", alloc)      # every warp is past the allocation
    permits = [m.start() for m in re.finditer(r"griddepcontrol\.launch_dependents", body)]
    assert len(permits) == 1 and permits[0] > held
    assert body.index("griddepcontrol.wait") > held
