"""What the library would launch, without a GPU: its calls into the HIP runtime answered by a recorder that says there
is one gfx950 device of 256 compute units and writes each launch's grid and block down.  Nothing runs, so pointers
are only looked at for their alignment."""
import os
import subprocess
import sys

SOURCE = r"""
#include <hip/hip_runtime_api.h>
#include <cstdio>
#include <cstring>
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipGetDeviceCount(int* n) { *n = 1; return hipSuccess; }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_t* p, int) {
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950");
  p->multiProcessorCount = 256;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 g, dim3 b, void**, size_t, hipStream_t) {
  std::printf("launch %u %u %u %u %u %u\n", g.x, g.y, g.z, b.x, b.y, b.z);
  std::fflush(stdout);
  return hipSuccess;
}
}
"""

RUN = r"""
import ctypes, sys
ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
i64, f32, u32, vp = ctypes.c_int64, ctypes.c_float, ctypes.c_uint32, ctypes.c_void_p
import activation_sparse_gemm_token_amd as rtl
for line in sys.stdin:
    name, args = eval(line)
    fn = getattr(ctypes.CDLL(rtl.library_path), name)
    fn.restype = ctypes.c_int
    print("status", fn(*(eval(a) if isinstance(a, str) else i64(a) for a in args)), flush=True)
"""


def recorder(folder):
    """Builds the recorder into `folder`; returns its path."""
    src, lib = os.path.join(folder, "recorder.cpp"), os.path.join(folder, "recorder.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include", src, "-o", lib], check=True)
    return lib


def record(lib, calls):
    """[(status, [(grid, block)])] of each (entry point, arguments): an int is 64 bits wide, a text as `f32(0.5)`
    an argument of another type."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", RUN, lib, root], input="".join(f"{c!r}\n" for c in calls), text=True,
                         stdout=subprocess.PIPE, check=True).stdout
    got, launches = [], []
    for line in out.splitlines():
        word, *n = line.split()
        n = [int(i) for i in n]
        if word == "launch":
            launches.append((tuple(n[:3]), tuple(n[3:])))
        else:
            got.append((n[0], launches))
            launches = []
    return got


def launchable(grid, block):
    """The limits of a launch: threads of a dimension, blocks of y and z, threads of a block."""
    return all(0 < g and 0 < b and g * b < 1 << 32 for g, b in zip(grid, block)) and max(grid[1:]) < 1 << 16 and \
        block[0] * block[1] * block[2] <= 1024
