"""The batched attention on more than one device, on the CPU: a stand-in for the few
runtime calls of a launch (loaded ahead of the real runtime, in a process of its own)
keeps the attributes of each device apart, as the runtime does."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <cuda_runtime_api.h>
#include <string.h>
static int dev, fail_next, n_set;
static struct { const void* f; int dev; long bytes; } set[64];
static const int sms[2] = {152, 100};
unsigned last_grid;
int launches;

void fake_device(int d) { dev = d; }
void fake_failure(void) { fail_next = 1; }
int fake_set_calls(void) { return n_set; }
unsigned fake_last_grid(void) { return last_grid; }
int fake_launches(void) { return launches; }

cudaError_t cudaGetDevice(int* d) { *d = dev; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  if (a != cudaDevAttrMultiProcessorCount) return cudaErrorInvalidValue;
  *v = sms[d];
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  if (fail_next) { fail_next = 0; return cudaErrorMemoryAllocation; }
  set[n_set].f = f; set[n_set].dev = dev; set[n_set].bytes = v;
  ++n_set;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  long most = 48 << 10;
  for (int i = 0; i < n_set; ++i)
    if (set[i].f == f && set[i].dev == dev) most = set[i].bytes;
  if ((long)c->dynamicSmemBytes > most) return cudaErrorInvalidValue;
  last_grid = c->gridDim.x;
  ++launches;
  return cudaSuccess;
}
static int encode(void* map) { memset(map, 0, 128); return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned v,
                                             unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult* q) {
  *fn = (void*)encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
"""

RUN = r"""
import ctypes as C, sys
fake = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)
lib = C.CDLL(sys.argv[2])
class KV(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k", "v", "t")] + [(n, C.c_int32) for n in "lhdpn"] + \
               [("cap", C.c_int64)]
class KV8(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k", "v", "ks", "vs", "t")] + \
               [(n, C.c_int32) for n in "lhdpn"] + [("cap", C.c_int64)]
class Batch(C.Structure):
    _fields_ = [("start", C.c_void_p), ("pos", C.c_void_p), ("n", C.c_int32), ("rows", C.c_int32),
                ("keys", C.c_int64)]
P = C.c_void_p(1 << 20)
lib.sub_last_error.restype = C.c_char_p

def attn(d, codes, rows):
    b = Batch(1 << 20, 1 << 20, 1, rows, 0)
    at = [1 << 20] * (5 if codes else 3)
    kv = (KV8 if codes else KV)(*at, 1, 2, d, 64, 64, 4096)
    need = C.c_int64()
    assert lib.sub_chunk_attn_workspace(2, 2, d, 1, rows, C.byref(need)) == 0
    fn = lib.sub_chunk_attn8 if codes else lib.sub_chunk_attn
    return fn(P, C.c_int64(2 * d), 2, C.byref(kv), 0, C.byref(b), C.c_float(0.1),
              C.c_void_p(1 << 21), C.c_void_p(1 << 22), need, None), need.value

cases = [(d, codes, rows) for d in (64, 128) for codes in (0, 1) for rows in (1, 12, 300)]
fake.fake_device(0)
fake.fake_failure()
assert attn(*cases[0])[0] != 0                       # the attribute could not be set ..
need = {}
for dev, sms in ((0, 152), (1, 100), (0, 152)):
    fake.fake_device(dev)
    before = fake.fake_set_calls()
    for c in cases:
        code, n = attn(*c)                           # .. which is no answer for later calls
        assert code == 0, (dev, c, lib.sub_last_error())
        assert fake.fake_last_grid() == sms, (dev, c)
        assert need.setdefault((sms, c), n) == n
    assert fake.fake_set_calls() - before == (0 if (dev, before) == (0, 2 * len(cases)) else len(cases))
assert all(need[152, c] > need[100, c] for c in cases)
assert fake.fake_launches() == 3 * 2 * len(cases)
print("ok")
"""


def test_attention_is_set_up_on_each_device(tmp_path):
    gcc, nvcc = shutil.which("gcc"), shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if gcc is None or not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("no C compiler or no CUDA headers")
    (tmp_path / "fake.c").write_text(FAKE)
    (tmp_path / "run.py").write_text(RUN)
    so = str(tmp_path / "fake.so")
    subprocess.run([gcc, "-shared", "-fPIC", "-I", include, str(tmp_path / "fake.c"), "-o", so], check=True)
    lib = os.path.join(ROOT, "substitute_speculative_decoding_gb300", "libsubspec.so")
    r = subprocess.run([sys.executable, str(tmp_path / "run.py"), so, lib], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
