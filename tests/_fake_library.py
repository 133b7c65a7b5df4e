"""A library with the entry points that csrc/binding.cpp calls: it computes nothing, waits as long and returns the status
that a test tells it, and counts its calls."""
import ctypes
import subprocess

SOURCE = """
#include <unistd.h>
int calls, status, wait_us;
static int call(void) { ++calls; if (wait_us) usleep(wait_us); return status; }
int striped_kv4_store(void) { return call(); }
int striped_kv4_load(void) { return call(); }
int striped_attn_decode_kv4(void) { return call(); }
unsigned long striped_attn_decode_kv4_workspace_size(void) { return 256; }
int striped_attn_key_weight(void) { return call(); }
unsigned long striped_attn_key_weight_workspace_size(void) { return 256; }
int striped_kv_evict(void) { return call(); }
"""


class Fake:
    def __init__(self, folder):
        src = folder / "fake.c"
        src.write_text(SOURCE)
        self.path = str(folder / "libfake.so")
        subprocess.run(["gcc", "-shared", "-fPIC", "-o", self.path, str(src)], check=True)
        self._lib = ctypes.CDLL(self.path)

    def __getitem__(self, name):
        return ctypes.c_int.in_dll(self._lib, name).value

    def __setitem__(self, name, value):
        ctypes.c_int.in_dll(self._lib, name).value = value
