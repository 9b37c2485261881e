"""The library's own host code linked against tests/launch_recorder.cpp in
place of the HIP runtime: what a C entry launches, on 256 compute units, is
written down and nothing runs."""
import concurrent.futures as cf
import ctypes as ct
import os
import re
import shutil
import subprocess

from mlp_matmul_amd import _capi, build

TESTS = os.path.dirname(os.path.abspath(__file__))


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, (cmd, r.stderr[-3000:])
    return r.stdout


class Recorder:
    """`lib` has the entries of include/unweight.h; `launches(call)` says what
    a call launches: [(kernel, grid, block, first argument's bytes)]."""

    def __init__(self, folder):
        folder = str(folder)
        hipcc, objs = build._hipcc(), []
        flags = [f"--offload-arch={build.ARCH}", "--offload-host-only", "-O0", "-std=c++17", "-fPIC", f"-I{build.INCLUDE}",
                 f"-I{build.CSRC}"]
        jobs = []
        for src in build.HIP_SOURCES + build.HOST_SOURCES:
            objs.append(os.path.join(folder, src + ".o"))
            jobs.append([hipcc, *flags, "-x", "hip", "-c", os.path.join(build.CSRC, src), "-o", objs[-1]])
        objs.append(os.path.join(folder, "recorder.o"))
        jobs.append(["g++", "-std=c++17", "-O1", "-fPIC", "-c", os.path.join(TESTS, "launch_recorder.cpp"), "-o", objs[-1]])
        with cf.ThreadPoolExecutor(8) as ex:
            list(ex.map(_run, jobs))
        # the device code that the host code would register
        names = sorted(set(re.findall(r"\b__hip_fatbin_\w+", _run(["nm", *objs]))))
        with open(os.path.join(folder, "fatbins.c"), "w") as f:
            f.writelines(f"char {n}[16];\n" for n in names)
        so = os.path.join(folder, "librecorded.so")
        _run(["g++", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-pthread", *objs, "-x", "c", os.path.join(folder, "fatbins.c"),
              "-o", so])
        self.lib = ct.CDLL(so, mode=os.RTLD_LAZY | os.RTLD_LOCAL)
        for name, (res, args) in _capi.SIGNATURES.items():
            f = getattr(self.lib, name)
            f.restype, f.argtypes = res, args
        self.lib.recorded_kernel.restype = self.lib.recorded_launch.restype = ct.c_char_p
        self.lib.record_start.argtypes = [ct.c_uint64]
        every = [self.lib.recorded_kernel(i).decode() for i in range(self.lib.recorded_kernels())]
        plain = _run([shutil.which("c++filt") or "c++filt", *every]).splitlines()
        short = [re.sub(r"^void |uwk::|\(anonymous namespace\)::|\((?!anonymous).*$", "", p) for p in plain]
        self._name = dict(zip(every, short))

    def kernels(self):
        """Every kernel that the library holds."""
        return sorted(self._name.values())

    def launches(self, call, arg_bytes=0):
        self.lib.record_start(arg_bytes)
        call()
        out = []
        for i in range(self.lib.recorded_launches()):
            dims, lds, args = (ct.c_uint32 * 6)(), ct.c_uint64(), (ct.c_uint8 * max(arg_bytes, 1))()
            name = self.lib.recorded_launch(i, dims, ct.byref(lds), args)
            out.append((self._name[name.decode()], tuple(dims[:3]), tuple(dims[3:]), bytes(args)[:arg_bytes]))
        return out
