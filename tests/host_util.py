"""Runs host code of the library without a GPU: a child process in which the HIP calls are hip_stub.c's."""
import os
import subprocess
import sys
import textwrap

HERE = os.path.dirname(os.path.abspath(__file__))

PRELUDE = """
import ctypes, sys, threading

class Dim(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]

class Launch(ctypes.Structure):
    _fields_ = [("thread", ctypes.c_uint64), ("kernel", ctypes.c_void_p), ("grid", Dim), ("block", Dim)]

hip = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
hip.stub_launches.restype = ctypes.POINTER(Launch)
hip.stub_thread.restype = ctypes.c_uint64
import tensor_core_mixed_amd as T

def launches():
    return [hip.stub_launches()[i] for i in range(hip.stub_count())]

def at(i):  # an address of its own, 2^40 bytes from the next; nothing reads it
    return (i + 1) << 40
"""


def run(tmp_path, body):
    """`body` in a child process, after PRELUDE; its output."""
    stub = os.path.join(str(tmp_path), "libhipstub.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", os.path.join(HERE, "hip_stub.c"), "-o", stub, "-lpthread"],
                   check=True)
    r = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(body), stub], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout
