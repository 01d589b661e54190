"""The library over a stand-in for the HIP runtime (hip_stub.cpp): launches
are recorded, nothing runs, no GPU is needed. `run` executes a snippet in a
child process where the stand-in is in place, with

  S          the binding           ctypes   the module
  launches() [(kernel, grid, block)] since the last call of it
  first(i)   the address of the first argument's bytes of launch i (before launches())
  refuse(s)  kernels with s in their name refuse their attributes
  P          an aligned address that nothing reads

and returns what the snippet assigned to `result` (JSON)."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STUB = os.path.join(ROOT, "_build", "libhip_stub.so")

_PRELUDE = """
import ctypes, json, sys
stub = ctypes.CDLL({stub!r}, ctypes.RTLD_GLOBAL)   # before the library: its symbols come first
sys.path.insert(0, {root!r})
import bit_svdquant_diffusion_amd as S
stub.stub_kernel.restype = ctypes.c_char_p
stub.stub_first_argument.restype = ctypes.c_void_p
P = 0x7f0000000000
def first(i):
    return stub.stub_first_argument(i)
def launches():
    out = []
    for i in range(stub.stub_launches()):
        v = (ctypes.c_uint32 * 6)()
        stub.stub_shape(i, v)
        out.append((stub.stub_kernel(i).decode(), list(v[:3]), list(v[3:])))
    stub.stub_clear()
    return out
def refuse(part):
    stub.stub_refuse_attributes_of(part.encode())
result = None
"""


def build() -> str:
    src = os.path.join(ROOT, "tests", "hip_stub.cpp")
    if not os.path.exists(STUB) or os.path.getmtime(STUB) < os.path.getmtime(src):
        os.makedirs(os.path.dirname(STUB), exist_ok=True)
        tmp = f"{STUB}.tmp{os.getpid()}"
        subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I/opt/rocm/include", src, "-o", tmp], check=True)
        os.replace(tmp, STUB)
    return STUB


def run(snippet: str):
    code = _PRELUDE.format(stub=build(), root=ROOT) + snippet + "\nprint('RESULT ' + json.dumps(result))\n"
    r = subprocess.run([sys.executable, "-c", code], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-3000:])
    return json.loads([line for line in r.stdout.splitlines() if line.startswith("RESULT ")][-1][7:])
