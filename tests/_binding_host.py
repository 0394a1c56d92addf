"""The native binding (csrc/binding.cpp) driven without a GPU: tensors over
host memory that claim a CUDA device, C entries replaced by functions that note
the call, and a runtime whose current device is 0.  Runs as a child process
(the stand-ins for what it asks the runtime are preloaded): reads a list of calls as JSON,
prints what became of each: "called" or the refusal."""
from __future__ import annotations

import ctypes
import json
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ENTRIES = 4


def build(directory: str) -> None:
    import torch
    base = os.path.dirname(torch.__file__)
    subprocess.run(
        ["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
         "-D_GLIBCXX_USE_CXX11_ABI=1", "-I" + os.path.join(base, "include"),
         "-I" + sysconfig.get_paths()["include"], os.path.join(HERE, "host_tensors.cpp"),
         "-o", os.path.join(directory, "host_tensors.so"), "-L" + os.path.join(base, "lib"),
         "-ltorch_python", "-ltorch_cpu", "-lc10"], check=True, capture_output=True)
    source = os.path.join(directory, "device.c")
    with open(source, "w") as f:
        f.write("int cudaGetDevice(int *d) { *d = 0; return 0; }\n"
                "int cudaGetDeviceCount(int *n) { *n = 2; return 0; }\n"
                "int cudaDeviceGetStreamPriorityRange(int *a, int *b) { *a = *b = 0; return 0; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", source, "-o", os.path.join(directory, "device.so")],
                   check=True, capture_output=True)


def outcomes(directory: str, calls: list) -> list:
    """What becomes of each call: a dict of a name and keyword arguments, where
    a tensor is [shape, type, device]."""
    env = dict(os.environ, LD_PRELOAD=os.path.join(directory, "device.so"))
    r = subprocess.run([sys.executable, os.path.abspath(__file__), directory], env=env,
                       input=json.dumps(calls), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


def main(directory: str) -> None:
    sys.path[:0] = [directory, ROOT]
    import torch  # noqa: F401

    import host_tensors
    import quantized_gguf_dequant_gb300 as q

    room = (ctypes.c_char * (1 << 20))()
    address = (ctypes.addressof(room) + 255) // 256 * 256
    seen = []
    kind = ctypes.CFUNCTYPE(ctypes.c_int)

    def entry():
        seen.append(1)
        return 0

    fakes = [kind(entry) for _ in range(ENTRIES)]
    last = ctypes.cast(q.lib().qmm_last_error, ctypes.c_void_p).value
    n = q.native()
    n.init(q.QmmError, *(ctypes.cast(f, ctypes.c_void_p).value for f in fakes), last)
    cache = n.cache(1, 0, 2, 64)  # of device 0, two heads of 64

    def value(v):
        if isinstance(v, list):
            return host_tensors.cuda_tensor(address, tuple(v[0]), v[1], v[2])
        if isinstance(v, dict):  # a Rope, made past its own checks
            rope = q.Rope.__new__(q.Rope)
            for name, x in v.items():
                setattr(rope, name, x)
            pairs = v["pairs"]
            rope.inv_freq = host_tensors.cuda_tensor(address, (sum(pairs),), "f32", v["device"])
            rope.desc = q.RopeDesc(2 * sum(pairs), 0, len(pairs), (ctypes.c_int32 * 4)(*pairs),
                                   address)
            rope.address = ctypes.addressof(rope.desc)
            return rope
        return v

    out = []
    for call in json.loads(sys.stdin.read()):
        a = {k: value(v) for k, v in call["args"].items()}
        a["stream"] = 0
        del seen[:]
        try:
            if call["name"] == "logits_adjust":
                q.logits_adjust(a.pop("logits"), **a)
            else:
                c = q.KVCache.__new__(q.KVCache)
                c.h, c._native, c._cache = None, n, cache
                getattr(c, call["name"])(**a)
            out.append("called" if seen else "not called")
        except (ValueError, RuntimeError) as e:
            out.append(f"{type(e).__name__}: {e}" + (" (after the call)" if seen else ""))
    print(json.dumps(out))


if __name__ == "__main__":
    main(sys.argv[1])
