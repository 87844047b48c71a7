"""What a call of the library launches, without a GPU: ``Recorder`` runs the
library in a child process on the stand-in runtime of ``recording_runtime.cpp``
and gives back each call's status and launches. Addresses are never
dereferenced there, so calls of any size can be asked for."""
from __future__ import annotations

import ctypes
import json
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
GRID, BLOCK = ("gx", "gy", "gz"), ("bx", "by", "bz")


def build(folder) -> str:
    out = os.path.join(str(folder), "librecording.so")
    subprocess.run(["/opt/rocm/bin/hipcc", "-O1", "-std=c++17", "-fPIC", "-shared", "-x", "c++",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", os.path.join(HERE, "recording_runtime.cpp"),
                    "-o", out], check=True)
    return out


class Recorder:
    def __init__(self, folder):
        self.p = subprocess.Popen([sys.executable, os.path.abspath(__file__), build(folder)], stdin=subprocess.PIPE,
                                  stdout=subprocess.PIPE, text=True)

    def ask(self, **request):
        self.p.stdin.write(json.dumps(request) + "\n")
        self.p.stdin.flush()
        return json.loads(self.p.stdout.readline())

    def kernels(self) -> list:
        """Every kernel the library holds."""
        return self.ask()

    def close(self):
        self.p.stdin.close()
        self.p.stdout.close()
        self.p.wait(30)


def _answer(rt, H, q):
    """q: the configuration's class and values, the entry point's name and
    arguments, the handle's device, the caller's current device, the stream."""
    cfg = getattr(H, q["config"])(**q["values"])
    kind = {"Config": "hcgr", "BlockConfig": "hcgr_block", "LinearConfig": "hcgr_linear"}[q["config"]]
    rt.hipSetDevice(0)
    handle = getattr(H, kind + "_create")(cfg, q.get("device", 0))
    try:
        rt.hipSetDevice(q.get("current", 0))
        rt.forget_launches()
        status = getattr(H, q["call"])(handle, *q["args"], stream=q.get("stream", 0), check=False)
        now = ctypes.c_int()
        rt.hipGetDevice(ctypes.byref(now))
        launches = []
        for line in rt.recorded_launches().decode().splitlines():
            *n, name = line.split(" ", 9)
            launches.append({**dict(zip((*GRID, *BLOCK, "lds", "stream", "device"), map(int, n))), "kernel": name})
        return {"status": status, "error": H.last_error(), "current": now.value, "launches": launches}
    finally:
        getattr(H, kind + "_destroy")(handle)


def main():
    rt = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # before the library, which then binds to it
    rt.recorded_launches.restype = rt.registered_kernels.restype = ctypes.c_char_p
    sys.path.insert(0, ROOT)
    import skinny_gemm_hcgr_amd as H
    H.load_library()
    for line in sys.stdin:
        q = json.loads(line)
        got = _answer(rt, H, q) if q else rt.registered_kernels().decode().splitlines()
        print(json.dumps(got), flush=True)


if __name__ == "__main__":
    main()
