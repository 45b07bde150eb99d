"""Host-side sizes of the layer operators at the ends of their ranges (no GPU): no tokens, one token.  Each
query runs in a process of its own, so that one that dies is a failure of its test alone."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# records as in include/gdn_layers.h; fake offsets are an address that is never read
QUERY = """
import ctypes, struct, sys
L = ctypes.CDLL(sys.argv[1])
for n in ("dn_conv_workspace_size", "dn_scan_workspace_size"):
    f = getattr(L, n); f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_int], ctypes.c_size_t
for n in ("dn_scan_saved_size", "dn_norm_workspace_size"):
    f = getattr(L, n); f.argtypes, f.restype = [ctypes.c_char_p], ctypes.c_size_t
T, packed = int(sys.argv[2]), int(sys.argv[3])
B, n, cu = (1, 3, 1 << 20) if packed else (2, 0, 0)
for dtype in (0, 1):
    conv = struct.pack("8iq", B, 3, T, 16, 4, dtype, 1, n, cu)
    print(L.dn_conv_workspace_size(conv, 0), L.dn_conv_workspace_size(conv, 1))
    for N in (1, 16, 32, 64, 128):
        scan = struct.pack("8iq", B, T, 32, N, 1, dtype, 1, n, cu)
        print(L.dn_scan_workspace_size(scan, 0), L.dn_scan_workspace_size(scan, 1), L.dn_scan_saved_size(scan))
    print(L.dn_norm_workspace_size(struct.pack("6ifi", B, 3, T, 16, dtype, 0, 1e-6, 0)))
"""


@pytest.fixture(scope="module")
def library():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_delta_rule_02_gb300 import binding
    return binding.library_path()


@pytest.mark.parametrize("packed", [0, 1])
@pytest.mark.parametrize("T", [0, 1])
def test_sizes_without_tokens_and_with_one(library, T, packed):
    r = subprocess.run([sys.executable, "-c", QUERY, library, str(T), str(packed)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr)
    sizes = [int(v) for v in r.stdout.split()]
    assert len(sizes) == 2 * (2 + 3 * 5 + 1) and all(v > 0 for v in sizes)
