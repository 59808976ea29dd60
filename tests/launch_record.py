"""What the library launches for a call, on the host: a child process loads it
behind stand-ins for the HIP calls that launch kernels, which write down each
kernel's name, grid and workgroup and run nothing.  Pointers are never read."""
import json
import os
import re
import subprocess
import sys

import mxfp4_block_scaled_fp4q_amd as fq

SHIM = r"""
#include <stdint.h>
#include <stdio.h>
#include <string.h>
typedef struct { uint32_t x, y, z; } dim3;
static const void* stubs[4096];
static const char* names[4096];
static int count;
static struct { dim3 grid, block; size_t lds; void* stream; } now;
void** __hipRegisterFatBinary(const void* p) { return (void**)p; }
void __hipUnregisterFatBinary(void** m) {}
void __hipRegisterVar(void** m, void* v, char* h, char* d, int e, size_t s, int c, int g) {}
void __hipRegisterFunction(void** m, const void* f, char* d, const char* name, unsigned t, void* a,
                           void* b, void* c, void* e, int* w) {
    if (count < 4096) stubs[count] = f, names[count++] = name;
}
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void* stream) {
    now.grid = grid, now.block = block, now.lds = lds, now.stream = stream;
    return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, void** stream) {
    *grid = now.grid, *block = now.block, *lds = now.lds, *stream = now.stream;
    return 0;
}
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t lds, void* stream) {
    const char* name = "?";
    for (int i = 0; i < count; ++i)
        if (stubs[i] == f) name = names[i];
    printf("%s %u %u %u %u\n", name, g.x, g.y, g.z, b.x * b.y * b.z);
    return 0;
}
int hipGetLastError(void) { return 0; }
"""
CHILD = """
import ctypes, json, sys
shim = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
lib = ctypes.CDLL(sys.argv[2])
kinds = dict(p=ctypes.c_void_p, q=ctypes.c_int64, i=ctypes.c_int32, d=ctypes.c_double, z=ctypes.c_size_t)
for name, types, values in json.load(sys.stdin):
    f = getattr(lib, name)
    f.argtypes = [kinds[t] for t in types]
    status = f(*values)
    ctypes.CDLL(None).fflush(None)
    print("status", status, flush=True)
"""


def launches(folder, calls):
    """calls: [(function, a letter for each argument's type (p q i d z), values)].
    Returns for each (status, [(kernel, template arguments, grid, threads)])."""
    shim = os.path.join(str(folder), "launch_record.so")
    if not os.path.exists(shim):
        subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-x", "c", "-", "-o", shim], input=SHIM, text=True, check=True)
    lib = os.path.join(os.path.dirname(fq.__file__), "libfp4q.so")
    run = subprocess.run([sys.executable, "-c", CHILD, shim, lib], input=json.dumps(calls), text=True,
                         capture_output=True, timeout=100)
    assert run.returncode == 0, run.stderr[-2000:]
    out, seen = [], []
    for line in run.stdout.splitlines():
        if line.startswith("status"):
            out.append((int(line.split()[1]), seen))
            seen = []
            continue
        mangled, *numbers = line.split()
        x, y, z, threads = map(int, numbers)
        name = re.match(r"_ZN4fp4q(\d+)", mangled)
        at = name.end()
        kernel = mangled[at:at + int(name.group(1))]
        values = re.match(r"I((?:Li-?\w+?E)+)", mangled[at + len(kernel):])
        values = [int(v) for v in re.findall(r"Li(\w+?)E", values.group(1))] if values else []
        seen.append((kernel, values, (x, y, z), threads))
    return out
