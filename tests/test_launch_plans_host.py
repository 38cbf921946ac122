"""What the host code launches, without a GPU: a stand-in for the CUDA runtime's calls is loaded in front of it, which says
it has one or two devices and notes every launch (kernel, grid, cluster, shared memory and the first argument's first
bytes) instead of making it. The calls are made in a process of their own, on addresses that are no memory."""
import json
import os
import subprocess
import sys
import textwrap

import pytest

from w4a16_moe_expert_router_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The calls that the library makes on its way to a launch. Clusters of a size that fit a device: `room` CTAs over it.
STAND_IN = r"""
#include <cuda_runtime_api.h>
#include <string.h>
typedef struct { const void *kernel; unsigned grid, block, smem, cluster; unsigned char arg[64]; } launch_t;
launch_t fake_launches[64];
int fake_count = 0, fake_device = 0, fake_room[2] = {152, 152};
cudaError_t cudaGetDevice(int *d) { *d = fake_device; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int d) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *f, enum cudaFuncAttribute a, int v) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes *a, const void *f) {
  memset(a, 0, sizeof *a);
  a->numRegs = 168;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) *n = fake_room[fake_device] / c->attrs[i].val.clusterDim.x;
  return cudaSuccess;
}
struct { const void *kernel; const char *name; } fake_kernels[1024];  /* what the library registers when it is loaded */
int fake_registered = 0;
void __cudaRegisterFunction(void **h, const char *kernel, char *d, const char *name, int limit, void *t, void *b, void *bd,
                            void *gd, int *w) {
  fake_kernels[fake_registered].kernel = kernel;
  fake_kernels[fake_registered++].name = name;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **args) {
  launch_t *l = &fake_launches[fake_count++ % 64];
  l->kernel = f;
  l->grid = c->gridDim.x;
  l->block = c->blockDim.x;
  l->smem = c->dynamicSmemBytes;
  l->cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) l->cluster = c->attrs[i].val.clusterDim.x;
  memcpy(l->arg, args[0], sizeof l->arg);
  return cudaSuccess;
}
"""

PROGRAM = """
import ctypes, json, sys
from w4a16_moe_expert_router_gb300 import binding as B
fake, lib, P = ctypes.CDLL(sys.argv[1]), B.lib(), 4096
class Launch(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("grid", "block", "smem", "cluster")] + [
        ("arg", ctypes.c_uint64 * 8)]
ring = (Launch * 64).in_dll(fake, "fake_launches")
count, device = ctypes.c_int.in_dll(fake, "fake_count"), ctypes.c_int.in_dll(fake, "fake_device")
room = (ctypes.c_int * 2).in_dll(fake, "fake_room")

def launches(call):
    count.value = 0
    assert call() == B.OK
    return [ring[i] for i in range(count.value)]

def few(*shape):
    shape, w = B.make_shape(*shape), B.Weights(P, P)
    return [(l.grid, l.block, l.smem, l.cluster) for l in launches(lambda: lib.moe_w4a16_few(
        ctypes.byref(shape), 0, P, P, ctypes.byref(w), None, None, None, P, P, 1 << 40, None))]

def norm(R, d, typ, gate_rows, x, y, post, gate, pre, out, u):
    cfg = B.make_norm(R, d, typ, gate_rows)
    return launches(lambda: lib.moe_w4a16_norm(ctypes.byref(cfg), x, y, post, gate, pre, out, u, None))

def kernels(part):  # of one of the library's files, by the name that the compiler gave them
    class Kernel(ctypes.Structure):
        _fields_ = [("kernel", ctypes.c_void_p), ("name", ctypes.c_char_p)]
    n = ctypes.c_int.in_dll(fake, "fake_registered").value
    return {k.kernel: k.name.decode() for k in (Kernel * 1024).in_dll(fake, "fake_kernels")[:n] if part in k.name.decode()}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """Runs a program behind PROGRAM and returns what it prints last, as JSON."""
    libbuild.build()
    folder = tmp_path_factory.mktemp("stand_in")
    src, lib = folder / "stand_in.c", folder / "stand_in.so"
    src.write_text(STAND_IN)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(libbuild._nvcc()))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-I", include, str(src), "-o", str(lib)], check=True)

    def go(program):
        env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT)
        done = subprocess.run([sys.executable, "-c", PROGRAM + textwrap.dedent(program), str(lib)], env=env, cwd=ROOT,
                              capture_output=True, text=True, timeout=300)
        assert done.returncode == 0, done.stderr[-2000:]
        return json.loads(done.stdout.splitlines()[-1])

    return go


def test_a_kernel_reads_what_its_launch_has(run):
    """Every form of the norms' forward call, in every size class and type: a kernel that one call launches with an
    output u (and its weight) or with y is launched by no call that has none, so none follows a null pointer."""
    forms = run("""
        seen = {}
        for R in (1, 5000):
            for d in (8, 264, 1000, 2048, 4104, 8192):
                for typ in (0, 1, 2):
                    for gate_rows in (1, 7, R):
                        for x, y, post, gate, pre, out in ((i & 1, i & 2, i & 4, i & 8, i & 16, i & 32) for i in range(64)):
                            if (y or x and not post and not gate) and (out or pre):
                                a = [P if v else None for v in (x, y, post, gate, pre, out, pre)]
                                for l in norm(R, d, typ, gate_rows, *a):
                                    seen.setdefault(l.kernel, set()).add((bool(y), bool(pre), bool(l.arg[4]), bool(l.arg[6])))
        print(json.dumps([sorted(v) for v in seen.values()]))
    """)
    assert len(forms) > 20
    for kinds in forms:
        assert len(kinds) == 1 and kinds[0][1] == kinds[0][2] == kinds[0][3], kinds


def test_a_devices_plan_is_its_own(run):
    """The plan for a few tokens (how many CTAs share a sum, and so its order) does not change when another device,
    on which fewer clusters fit, is used for the first time."""
    seen = run("""
        shapes = [(1, 2048, 704, 128, 8, 64, 64), (16, 2048, 704, 128, 8, 64, 64), (22, 512, 256, 200, 8, 64, 64),
                  (10, 2048, 1408, 64, 4, 64, 64)]
        room[0], room[1] = 152, 24
        first = [few(*s) for s in shapes]
        device.value = 1
        other = [few(*s) for s in shapes]
        device.value = 0
        print(json.dumps([first, other, [few(*s) for s in shapes]]))
    """)
    first, other, again = seen
    assert first != other and again == first


def test_every_kernel_of_the_norms_is_reached(run):
    """What norm.cu builds and what some call of its two operators launches is the same."""
    built, left = run("""
        reached = set()
        for R in (1, 700, 5000):
            for d in (8, 264, 520, 1000, 1344, 2048, 2056, 4104, 8192):
                for typ in (0, 1, 2):
                    for gate_rows in (1, 7, R):
                        cfg = B.make_norm(R, d, typ, gate_rows)
                        for post, gate, pre, out, y, x in ((i & 1, i & 2, i & 4, i & 8, i & 16, i & 32) for i in range(64)):
                            w = lambda v: P if v else None
                            if (y or x and not post and not gate) and (out or pre):
                                reached |= {l.kernel for l in norm(R, d, typ, gate_rows, w(x), w(y), w(post), w(gate), w(pre),
                                                                   w(out), w(pre))}
                            if y or not post and not gate:
                                reached |= {l.kernel for l in launches(lambda: lib.moe_w4a16_norm_backward(
                                    ctypes.byref(cfg), w(y), w(post), w(gate), P, w(pre), P, w(pre), w(x or not pre), w(y), w(post),
                                    w(gate), w(pre), P, 1 << 40, None))}
        built = kernels("norm_cu")
        print(json.dumps([len(built), sorted(name for k, name in built.items() if k not in reached)]))
    """)
    assert built > 100 and left == []
