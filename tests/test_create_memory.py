"""fkv_create where the host has no memory for the context: a status, no C++
exception across the C boundary (which would end the process)."""

import os
import subprocess
import sys

import cross_layer_kv_gb300 as fkv
from cross_layer_kv_gb300 import fusedkv as B

CHILD = """
import ctypes, resource, sys

class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("num_layers", "batch", "max_seq", "num_q_heads", "num_kv_heads",
                                            "head_dim", "dtype", "store_upper")]
    _fields_ += [("softmax_scale", ctypes.c_float), ("decode_ctas", ctypes.c_int)]

lib = ctypes.CDLL(sys.argv[1])
pages = int(open("/proc/self/statm").read().split()[0])
room = pages * resource.getpagesize() + (1 << 30)
resource.setrlimit(resource.RLIMIT_AS, (room, room))
out = ctypes.c_void_p(1234)
cfg = Config(1 << 30, 1, 256, 4, 2, 64, 1, 0, 0.0, 0)
print(lib.fkv_create(ctypes.byref(cfg), ctypes.byref(out)), out.value)
"""


def test_no_memory_for_the_layers_is_a_status():
    fkv.load()
    # the child's structure is the binding's
    assert [n for n, _ in B.fkv_config._fields_] == [
        "num_layers", "batch", "max_seq", "num_q_heads", "num_kv_heads", "head_dim", "dtype",
        "store_upper", "softmax_scale", "decode_ctas"]
    r = subprocess.run([sys.executable, "-c", CHILD, B.library_path()], capture_output=True, text=True,
                       timeout=120, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.split() == [str(B.FKV_ERR_INVALID_ARG), "None"]
