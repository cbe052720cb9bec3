"""The library in a process whose device context is reset between calls (the
process's own context; nothing else on the GPU is touched)."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes
from ctypes import byref, c_int, c_size_t, c_uint64, c_void_p
from muon_polar_orthogonalized_b200 import _native as N

cu = ctypes.CDLL("libcuda.so.1")

def ok(r):
    assert r == 0, r

ok(cu.cuInit(0))
dev = c_int()
ok(cu.cuDeviceGet(byref(dev), 0))
L = N.lib()
n, vocab, dim = 20000, 1000, 8          # a sort of 16 blocks
ids = (ctypes.c_int32 * n)(*[(i * 7) % vocab for i in range(n)])
ones = (ctypes.c_float * (n * dim))(*([1.0] * (n * dim)))
for turn in range(3):
    ctx = c_void_p()
    ok(cu.cuDevicePrimaryCtxRetain(byref(ctx), dev))
    ok(cu.cuCtxSetCurrent(ctx))

    def alloc(nbytes, host=None):
        p = c_uint64()
        ok(cu.cuMemAlloc_v2(byref(p), c_size_t(nbytes)))
        if host is not None:
            ok(cu.cuMemcpyHtoD_v2(p, host, c_size_t(nbytes)))
        return p

    need = L.muon_embedding_grad_workspace_size(vocab, dim, n)
    d_ids, d_out, d_grad, d_ws = alloc(4 * n, ids), alloc(4 * n * dim, ones), alloc(4 * vocab * dim), alloc(need)
    st = L.muon_embedding_grad(d_out.value, N.MUON_F32, dim, d_ids.value, 32, n, vocab, dim, 1.0, d_grad.value,
                               N.MUON_F32, 0, d_ws.value, need, None)
    assert st == N.MUON_OK, (turn, N.last_error())
    assert L.muon_query_status(d_ws.value, None) == N.MUON_OK
    got = (ctypes.c_float * (vocab * dim))()
    ok(cu.cuMemcpyDtoH_v2(got, d_grad, c_size_t(4 * vocab * dim)))
    assert all(v == n / vocab for v in got)
    ok(cu.cuDevicePrimaryCtxReset_v2(dev))
print("three contexts")
"""


def test_large_sort_after_a_reset_of_the_context():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "three contexts" in r.stdout, r.stdout + r.stderr
