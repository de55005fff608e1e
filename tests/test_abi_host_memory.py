"""moe_grad_clip where the host's memory does not suffice to check a long list: an error, and the process
goes on. On the CPU, in a process of its own with a limit on its memory."""
import subprocess
import sys

from test_abi_residual import lib  # noqa: F401  (fixture)

CODE = r"""
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
class Grad(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32)]
n = 1 << 20
one = bytes(Grad(1 << 40, 1 << 40, 8, 0))
grads = ctypes.create_string_buffer(one * n, len(one) * n)   # the same tensor again and again: refused
lib.moe_last_error.restype = ctypes.c_char_p
lib.moe_grad_clip.argtypes = [ctypes.c_int32] + [ctypes.c_void_p] * 2 + [ctypes.c_float] * 2 + [ctypes.c_void_p]
call = lambda: lib.moe_grad_clip(n, grads, 1 << 41, 1.0, 1e-6, None)
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (8 << 20),) * 2)
print(call(), lib.moe_last_error().decode())
print("went on")
"""


def test_no_memory_to_check_a_long_list(lib):  # noqa: F811
    import mixture_experts_lora_amd as mel
    p = subprocess.run([sys.executable, "-c", CODE, mel.library_path()], capture_output=True, text=True,
                       timeout=120)
    assert p.returncode == 0, (p.returncode, p.stdout, p.stderr)
    assert p.stdout.splitlines() == ["4 moe_grad_clip: out of memory", "went on"]
