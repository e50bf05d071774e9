"""What the library asks of the HIP runtime around its launches, without a GPU: a stand-in for the runtime, loaded
before the library, writes down the calls and fails those that it is told to."""

import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_linear_layers_absmean_amd", "libsbl.so")
OK, LAUNCH = 0, 5

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="fake addresses: only where no GPU is")

RUNTIME = r"""
#include <cstdio>
#include <cstring>
#include <map>
#include <string>
struct dim3 { unsigned x, y, z; };
static std::map<const void*, std::string> names;
static std::string text;
static int device = 0, fail_attribute = 0, fail_launch = 0, launches = 0, last = 0;
static dim3 g, b;
static size_t lds;
static void* stream;
static std::string name(const void* f) { auto i = names.find(f); return i == names.end() ? "?" : i->second; }
extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* p; return &p; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* n, unsigned, void*, void*, void*, void*, int*) { names[f] = n; }
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(dim3 gg, dim3 bb, size_t l, void* s) { g = gg; b = bb; lds = l; stream = s; return 0; }
int __hipPopCallConfiguration(dim3* gg, dim3* bb, size_t* l, void** s) { *gg = g; *bb = b; *l = lds; *s = stream; return 0; }
int hipGetDevice(int* d) { *d = device; return 0; }
int hipGetLastError() { const int e = last; last = 0; return e; }
int hipDeviceGetAttribute(int* v, int, int) { *v = 256; return 0; }
int hipFuncSetAttribute(const void* f, int, int bytes) {
  text += "limit " + std::to_string(device) + " " + std::to_string(bytes) + " " + name(f) + "\n";
  return fail_attribute ? last = 1 : 0;
}
int hipLaunchKernel(const void* f, dim3, dim3, void**, size_t bytes, void*) {
  text += "launch " + std::to_string(device) + " " + std::to_string(bytes) + " " + name(f) + "\n";
  return ++launches == fail_launch ? last = 719 : 0;
}
void use(int d, int attribute, int launch) { device = d; fail_attribute = attribute; fail_launch = launch; launches = 0; text.clear(); }
const char* seen() { return text.c_str(); }
}
"""

CALLS = r"""
import ctypes, json, sys
runtime = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
runtime.seen.restype = ctypes.c_char_p
lib = ctypes.CDLL(sys.argv[2])
GB = 1 << 30
p = [ctypes.c_void_p(GB * 64 * i) for i in range(1, 9)]
i64, i32, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
none = ctypes.c_void_p(None)
def embed():
    return lib.sbl_embed_backward(p[0], p[1], i32(0), i64(5000), i64(262144), i64(256), f32(1.0), p[2], i32(0), i32(0), p[3],
                                  i64(1 << 35), none)
def linear():
    return lib.sbl_linear(p[0], none, i32(0), i32(6), i32(8), p[1], p[2], p[3], i64(8), i64(28672), i64(8192), p[4], none, none)
out = []
for call, device, attribute, launch in json.loads(sys.argv[3]):
    runtime.use(device, attribute, launch)
    status = dict(embed=embed, linear=linear)[call]()
    out.append([status, runtime.seen().decode().splitlines()])
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    if not os.path.exists(LIB):
        pytest.fail("libsbl.so is not built (run __graft_entry__.build())")
    at = tmp_path_factory.mktemp("runtime")
    source, lib = at / "runtime.cpp", at / "runtime.so"
    source.write_text(RUNTIME)
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    subprocess.run([compiler, "-shared", "-fPIC", "-O1", str(source), "-o", str(lib)], check=True)

    def run(*asked):
        r = subprocess.run([sys.executable, "-c", CALLS, str(lib), LIB, json.dumps(asked)], capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout.splitlines()[-1])

    return run


@pytest.mark.parametrize("call,kernel", [("embed", "sort_kernel"), ("linear", "gemv_kernel")])
def test_lds_limit_is_raised_on_every_gpu(calls, call, kernel):
    """Once on each device, before the first launch there, whichever device was first."""
    seen = calls(*[(call, d, 0, 0) for d in (1, 1, 0, 0, 1, 3)])
    for i, (status, lines) in enumerate(seen):
        assert status == OK
        raised = [x for x in lines if x.startswith("limit")]
        own = [x for x in lines if x.startswith("launch") and kernel in x]
        assert len(own) == 1 and int(own[0].split()[2]) >= 64 * 1024
        if i in (0, 2, 5):
            limit = [x for x in raised if x.split()[3] == own[0].split()[3]]
            assert len(limit) == 1 and limit[0].split()[1] == own[0].split()[1] and int(limit[0].split()[2]) >= int(own[0].split()[2])
            assert lines.index(limit[0]) < lines.index(own[0])
        else:
            assert not raised


@pytest.mark.parametrize("call", ["embed", "linear"])
def test_a_limit_that_cannot_be_raised_is_an_error(calls, call):
    """Nothing is launched; the next call tries again."""
    (status, lines), (status2, lines2) = calls((call, 0, 1, 0), (call, 0, 0, 0))
    assert status == LAUNCH and not [x for x in lines if x.startswith("launch")]
    assert status2 == OK and [x for x in lines2 if x.startswith("limit")] and [x for x in lines2 if x.startswith("launch")]


def test_sums_do_not_follow_a_sort_that_did_not_start(calls):
    """The sums take places in memory from the order that the sort writes: without it nothing more is launched."""
    for failing in (1, 2, 3):
        status, lines = calls(("embed", 0, 0, failing))[0]
        kernels = [x.split()[3] for x in lines if x.startswith("launch")]
        assert status == LAUNCH and len(kernels) == failing
        assert ["sort_kernel", "sum_kernel", "join_kernel"][failing - 1] in kernels[-1]
