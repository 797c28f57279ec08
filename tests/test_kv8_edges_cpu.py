"""Host side of the 8-bit attention at its edges, without a GPU. Calls that once
ended the process run in a process of their own."""

import subprocess
import sys


def alone(code):
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path[:0] = ['.', 'tests']\n" + code], capture_output=True,
                       text=True, timeout=300)
    return r.returncode, r.stdout.split()


def test_a_batch_of_no_queries_with_any_group():
    """No query token at all, as in an empty step: nothing to do, whatever the
    query heads of a KV head (17 and more once divided by zero)."""
    code = """
import ctypes
from test_kv_append_cpu import attend, batch, pool8, lib
for group in (1, 16, 17, 32, 100, 128):
    for b in (batch(B=0, q=(0, 0), docs=(0, 0)), batch(q=(0, 0)), batch(q=(0, 0), docs=(3000, 2000))):
        n = lib().rag_kv8_workspace_size(ctypes.byref(pool8()), ctypes.byref(b), 8 * group)
        print(attend(pool8(), b, hq=8 * group, q=None, o=None) if n >= 256 else n)
"""
    assert alone(code) == (0, ["0"] * 18)
