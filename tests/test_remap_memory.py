"""A radix tree's remap where the host has no memory for it: an error code, not
the end of the process, and the tree as it was."""
import subprocess
import sys

SCRIPT = """
import resource
import numpy as np
import paged_hybrid_sliding_gb300 as phs

n = 300_000                      # nodes: 4 MB for the list of them
alloc = phs.PageAllocator(n)
tree = phs.RadixTree(alloc, 1)
pages = alloc.alloc(n).astype(np.int32)
lib, h = phs.lib(), tree._h
token = np.zeros(1, np.int32)
for i in range(n):
    token[0] = i
    assert lib.phs_radix_insert(h, token.ctypes.data, 1, pages[i:].ctypes.data, None) == 0
page_map = np.arange(n, dtype=np.int32)[::-1].copy()
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
soft, hard = resource.getrlimit(resource.RLIMIT_AS)
resource.setrlimit(resource.RLIMIT_AS, (used + 65536, hard))
code = lib.phs_radix_remap(h, page_map.ctypes.data, n)
resource.setrlimit(resource.RLIMIT_AS, (soft, hard))
assert code in (0, -5), code
first = tree.match([0]).tolist()
assert first == [int(pages[0] if code else page_map[pages[0]])]
tree.remap(page_map if code else np.arange(n, dtype=np.int32))
print("code", code)
"""


def test_remap_without_memory_is_an_error_code():
    r = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.strip() == "code -5"
