"""Which kernels a call launches: it is captured into a graph, not run, and the
graph's kernel nodes are asked for their names and grids."""
import collections
import ctypes as ct
import re

import torch

Launch = collections.namedtuple("Launch", "kernel args grid block")


class _Dim3(ct.Structure):
    _fields_ = [("x", ct.c_uint32), ("y", ct.c_uint32), ("z", ct.c_uint32)]


class _KernelParams(ct.Structure):  # hipKernelNodeParams
    _fields_ = [("block", _Dim3), ("extra", ct.c_void_p), ("func", ct.c_void_p), ("grid", _Dim3),
                ("args", ct.c_void_p), ("lds", ct.c_uint32)]


def _hip():
    with open("/proc/self/maps") as f:  # the runtime that torch has loaded
        path = next(line.split()[-1] for line in f if "libamdhip64" in line)
    hip = ct.CDLL(path)
    hip.hipKernelNameRefByPtr.restype = ct.c_char_p
    return hip


def launches(call):
    """The kernels of a call in order: name, integer template arguments, grid
    (x, y) and threads of a workgroup.  The call has to have run before."""
    hip = _hip()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        keep = call()
    raw, n = ct.c_void_p(graph.raw_cuda_graph()), ct.c_size_t(0)
    assert hip.hipGraphGetNodes(raw, None, ct.byref(n)) == 0
    nodes = (ct.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(raw, nodes, ct.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ct.c_int(-1), _KernelParams()
        assert hip.hipGraphNodeGetType(ct.c_void_p(node), ct.byref(kind)) == 0 and kind.value == 0
        assert hip.hipGraphKernelNodeGetParams(ct.c_void_p(node), ct.byref(p)) == 0
        name = hip.hipKernelNameRefByPtr(ct.c_void_p(p.func), None).decode()
        m = re.search(r"4fp4q\d+([a-z0-9_]+?_kernel)(?:I((?:Li\d+E)+)E)?", name)
        assert m, name
        args = tuple(int(a) for a in re.findall(r"Li(\d+)E", m.group(2) or ""))
        out.append(Launch(m.group(1), args, (p.grid.x, p.grid.y), p.block.x))
    del keep
    return out
