"""What accepted calls of the library launch, followed on the CPU: a child process opens
tests/host_launch/fake_hip.c in place of the HIP runtime and then liblogra.so, makes
the calls with stand-in addresses, and reports each one's status and launches.  Nothing is run
on a GPU: the child makes no call unless the library's kernels have been registered with
the stand-in.
"""
import ctypes
import importlib.util
import json
import os
import subprocess
import sys
from collections import namedtuple

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = os.path.join(HERE, "host_launch", "fake_hip.c")
LOADER = os.path.join(os.path.dirname(HERE), "rank_gradient_sketching_amd", "_lib.py")

Launch = namedtuple("Launch", "name grid block")


def follow(calls, folder):
    """[(status, [Launch, ...]), ...] of calls [(entry point, [arguments]), ...]; folder:
    where the stand-in is built.  An argument {"grads": [[entries, type], ...]} is the table
    that logra_grad_table makes of such tensors."""
    fake = os.path.join(str(folder), "fake_hip.so")
    if not os.path.exists(fake):
        subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC",
                        FAKE, "-o", fake], check=True)
    res = subprocess.run([sys.executable, os.path.abspath(__file__), fake], input=json.dumps(calls),
                         capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    return [(st, [Launch(n, tuple(g), tuple(b)) for n, g, b in ls]) for st, ls in
            json.loads(res.stdout)]


def _table(loader, lib, grads):
    items = (loader.GradItem * len(grads))()
    for q, (n, kind) in zip(items, grads):
        q.g, q.n, q.g_type = 1 << 40, n, kind
    size = lib.logra_grad_table_bytes(len(grads))
    table = (ctypes.c_uint64 * (size // 8))()
    if lib.logra_grad_table(len(grads), items, table, size) != 0:
        sys.exit("the table was refused")
    return table


def _child(fake):
    class Record(ctypes.Structure):
        _fields_ = [("name", ctypes.c_char_p), ("grid", ctypes.c_uint32 * 3),
                    ("block", ctypes.c_uint32 * 3)]

    stand_in = ctypes.CDLL(fake, mode=ctypes.RTLD_GLOBAL)
    stand_in.fake_hip_launch.restype = ctypes.POINTER(Record)
    spec = importlib.util.spec_from_file_location("_lib", LOADER)
    loader = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(loader)
    lib = loader.lib()
    if stand_in.fake_hip_kernels() < 50:
        sys.exit("the library's kernels are not registered with the stand-in")
    out = []
    for name, args in json.load(sys.stdin):
        tables = [_table(loader, lib, x["grads"]) if isinstance(x, dict) else None for x in args]
        args = [x if t is None else ctypes.addressof(t) for x, t in zip(args, tables)]
        stand_in.fake_hip_clear()
        status = getattr(lib, name)(*args)
        n = stand_in.fake_hip_launches()
        recs = [stand_in.fake_hip_launch(i).contents for i in range(n)]
        out.append((status, [(r.name.decode(), list(r.grid), list(r.block)) for r in recs]))
    json.dump(out, sys.stdout)


if __name__ == "__main__":
    _child(sys.argv[1])
