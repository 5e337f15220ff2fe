"""A caller with a CUDA context of its own: it stays the current one, and the
call's work is done in it. In a process of its own, without torch's context."""
import os
import subprocess
import sys

import pytest
import torch

import exact_attention_134_b200 as attn

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes
import sys

sys.path.insert(0, sys.argv[1])
import exact_attention_134_b200 as attn

lib = attn.lib()
cu = ctypes.CDLL("libcuda.so.1")
vp, sz = ctypes.c_void_p, ctypes.c_size_t


def ok(r):
    assert r == 0, r


def current():
    c = vp()
    ok(cu.cuCtxGetCurrent(ctypes.byref(c)))
    return c.value


ok(cu.cuInit(0))
ctx, base = vp(), vp()
ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))
assert current() == ctx.value
page = lib.attn_kv4_page_bytes(1, 64, 16)
ok(cu.cuMemAlloc_v2(ctypes.byref(base), sz(4 * page + 512)))
src, dst = base.value + 4 * page, base.value + 4 * page + 256
data = bytes((7 * i + i // page) % 251 for i in range(4 * page))
for at, b in ((base.value, data), (src, (ctypes.c_int * 2)(0, 4)), (dst, (ctypes.c_int * 2)(2, 1))):
    ok(cu.cuMemcpyHtoD_v2(vp(at), bytes(b), sz(len(bytes(b)))))
# page 0 to page 2; there is no page 4, which the status word says
assert lib.attn_kv4_copy_pages(base, 1, 4, page, vp(src), vp(dst), 2, None) == 0
assert current() == ctx.value
where = ctypes.c_int()
assert lib.attn_get_status_ex(None, ctypes.byref(where)) == 1 and where.value == 0x530
assert lib.attn_get_status_ex(None, ctypes.byref(where)) == 0
assert current() == ctx.value
back = ctypes.create_string_buffer(4 * page)
ok(cu.cuMemcpyDtoH_v2(back, base, sz(4 * page)))
assert back.raw == data[:2 * page] + data[:page] + data[3 * page:]
ok(cu.cuMemFree_v2(base))
ok(cu.cuCtxDestroy_v2(ctx))
print("done")
"""


def test_the_callers_context_stays_current():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    root = os.path.dirname(os.path.dirname(os.path.abspath(attn.__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, root], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]
