"""The host code behind logra_policy.h under AddressSanitizer and
UndefinedBehaviorSanitizer, built and run as that of logra.h is
(test_host_sanitizers.py): sizes and strides of every magnitude, and the table
of an AdamW step in buffers of exactly its size."""
import concurrent.futures
import os
import subprocess

from test_host_sanitizers import CSRC, INCLUDE, ROCM, SAN, _run, _tools

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host_sanitize",
                      "policy_host_checks.c")
SOURCES = ["abi.cpp", "regen.hip", "sketch.hip", "merge.hip", "kl.hip", "kl_sweep.hip",
           "optim.hip", "noalloc.hip", "policy/abi_policy.cpp", "policy/logprob.hip",
           "policy/adamw.hip", "policy/adapter.hip"]


def test_policy_host_code_under_asan_and_ubsan(tmp_path):
    hipcc, clang = _tools()
    out = str(tmp_path)

    def compile_one(src):
        obj = os.path.join(out, os.path.splitext(os.path.basename(src))[0] + ".o")
        _run([hipcc, "--offload-arch=gfx950", "-O2", "-std=c++17", "-fPIC", "-Xclang",
              "-target-feature", "-Xclang", "-packed-fp32-ops", "-Xarch_host", "-g",
              f"-I{INCLUDE}", f"-I{CSRC}", *SAN, "-c", os.path.join(CSRC, src), "-o", obj], out)
        return obj

    with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    exe = os.path.join(out, "policy_host_checks")
    _run([clang, "-x", "c", "-std=c11", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", f"-I{INCLUDE}",
          f"-I{ROCM}/include", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-c",
          DRIVER, "-o", exe + ".o"], out)
    _run([hipcc, "--offload-arch=gfx950", *SAN, exe + ".o", *objs, f"-L{ROCM}/lib",
          f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64", "-o", exe], out)
    for obj in objs:
        syms = _run(["nm", obj], out).stdout
        assert "__asan_" in syms, obj
        if os.path.basename(obj) in ("abi_policy.o", "adamw.o", "adapter.o"):
            assert "__ubsan_handle" in syms, obj
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    env.pop("LD_PRELOAD", None)
    res = subprocess.run([exe], cwd=out, capture_output=True, text=True, env=env, timeout=120)
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-8000:]
    assert "0 failed" in res.stdout
