"""Memory of another device is refused argument by argument, on the CPU: the calls'
compiled objects are linked with a stand-in for the query of where an address lies,
which says of one argument at a time that it is another device's. They run in a
process that sees no GPU, so that nothing is launched whatever they answer."""

import json
import os
import subprocess
import sys

import pytest

STAND_IN = """
#include <cuda_runtime_api.h>
struct tf_segments;
static const void* elsewhere = nullptr;
extern "C" void put_elsewhere(const void* p) { elsewhere = p; }
namespace tf {
bool on_this_device(const void* p) { return p != elsewhere; }
bool on_this_device(const tf_segments*) { return true; }
int sm_count() { return 152; }
int cuda_fail(cudaError_t) { return -100; }
}
"""

CALLS = """
import ctypes, json, sys
lib = ctypes.CDLL(sys.argv[1])
vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
lib.tf_norm_rows.argtypes = [vp, i64, vp, i64, vp, f32, i32, i32, vp, i64, vp, vp, vp]
lib.tf_linear_rows.argtypes = [vp, i64, vp, i32, i32, vp, vp, vp, i32, vp, i64, vp]
lib.put_elsewhere.argtypes = [vp]
at = lambda i: 0x7F0000000000 + (i << 36)
NORM = dict(x=at(0), res=at(1), w=at(2), sum=at(3), codes=at(4), scales=at(5))
LINEAR = dict(x=at(0), x_scales=at(1), w=at(2), w_scales=at(3), s=at(4), y=at(5))
def norm(res=True):
    a = dict(NORM) if res else dict(NORM, res=None, sum=None)
    return lib.tf_norm_rows(a["x"], 64, a["res"], 64, a["w"], 1e-5, 4, 64, a["sum"], 64, a["codes"], a["scales"], None)
def linear(x_scales=True):
    a = dict(LINEAR) if x_scales else dict(LINEAR, x_scales=None)
    return lib.tf_linear_rows(a["x"], 64, a["x_scales"], 4, 64, a["w"], a["w_scales"], a["s"], 40, a["y"], 40, None)
def status(call, address, *args):
    lib.put_elsewhere(address)
    return call(*args)
print(json.dumps({
    "norm": {n: status(norm, p) for n, p in NORM.items()},
    "norm alone": {n: status(norm, p, False) for n, p in NORM.items() if n not in ("res", "sum")},
    "linear": {n: status(linear, p) for n, p in LINEAR.items()},
    "linear of bf16": {n: status(linear, p, False) for n, p in LINEAR.items() if n != "x_scales"},
    "here": [status(norm, at(9)), status(norm, at(9), False), status(linear, at(9)), status(linear, at(9), False)]}))
"""


@pytest.fixture(scope="module")
def statuses(tmp_path_factory):
    import __graft_entry__
    __graft_entry__.build()
    from stream_speculative_decode_gb300 import build as b
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(b.nvcc_path())))
    d = tmp_path_factory.mktemp("elsewhere")
    src, lib = d / "stand_in.cpp", d / "libcalls.so"
    src.write_text(STAND_IN)
    objs = [os.path.join(b.OUT_DIR, o) for o in ("norm.o", "linear.o")]
    subprocess.run([b.nvcc_path(), "-shared", "-cudart", "shared", "-Xcompiler", "-fPIC", "-o", str(lib), str(src)] + objs +
                   ["-Xlinker", "-rpath," + os.path.join(cuda, "lib64")], check=True)
    r = subprocess.run([sys.executable, "-c", CALLS, str(lib)], env={**os.environ, "CUDA_VISIBLE_DEVICES": ""},
                       stdout=subprocess.PIPE, check=True, timeout=120)
    return json.loads(r.stdout)


@pytest.mark.parametrize("call", ["norm", "norm alone", "linear", "linear of bf16"])
def test_every_argument_is_looked_at(statuses, call):
    from stream_speculative_decode_gb300 import tf
    assert statuses[call] == dict.fromkeys(statuses[call], tf.TF_EINVAL)


def test_memory_of_this_device_is_not_refused(statuses):
    """What answers these calls is the launch, in a process without a GPU."""
    from stream_speculative_decode_gb300 import tf
    assert tf.TF_EINVAL not in statuses["here"] and tf.TF_OK not in statuses["here"]
