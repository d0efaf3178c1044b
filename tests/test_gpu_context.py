"""Calls that encode tensor maps, from host threads with a context of their own (driver API), with none, and with one
that was taken off again: a context that the caller made current is used and stays current. Each in a process of its
own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = """
import ctypes, threading
import numpy as np
import torch
import routed_expert_ffn_moe_gb300 as moe
from mx_helpers import quantised

torch.zeros(1, device="cuda")  # the primary context
moe.load()
cu = ctypes.CDLL("libcuda.so.1")
vp, u64 = ctypes.c_void_p, ctypes.c_uint64


def ok(code):
    assert code == 0, code


def current():
    c = vp()
    ok(cu.cuCtxGetCurrent(ctypes.byref(c)))
    return c.value


T, N, K = 1, 128, 1024  # one launch: the call's first use of the driver is a tensor map
r = np.random.default_rng(1)
w = (r.standard_normal((N, K))).astype(np.float32)
x = torch.from_numpy(r.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16)
rows, shape = moe.mx_rows(N, K, "f32", True), moe.mx_shape(T, N, K)
n_ws, n_s = moe.moe_mx_linear_workspace_size(shape), moe.moe_mx_scale_bytes(rows)
ref = quantised(x.double().numpy())[0] @ quantised(w)[0].T
xb = x.view(torch.int16).numpy()


def near(y):
    y = torch.from_numpy(y).view(torch.bfloat16).double().numpy()
    mag = np.abs(quantised(x.double().numpy())[0]) @ np.abs(quantised(w)[0]).T
    acc = (K + 2) * 2.0 ** -23 * mag  # K products summed in fp32, then half a step of bf16
    assert (np.abs(y - ref) <= acc + 2.0 ** -8 * (np.abs(ref) + acc)).all()


def in_thread(f):
    errors = []

    def run():
        try:
            f()
        except BaseException as e:
            errors.append(e)

    th = threading.Thread(target=run)
    th.start()
    th.join()
    if errors:
        raise errors[0]
"""

OWN = COMMON + """
def work():
    dev, own = ctypes.c_int(), vp()
    ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
    ok(cu.cuCtxCreate_v2(ctypes.byref(own), 0, dev))
    assert current() == own.value

    def alloc(n):  # memory of this context, zeros
        p = u64()
        ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(n)))
        ok(cu.cuMemsetD8_v2(p, 0, ctypes.c_size_t(n)))
        return p.value

    def put(a):
        p = alloc(a.nbytes)
        ok(cu.cuMemcpyHtoD_v2(u64(p), a.ctypes.data_as(vp), ctypes.c_size_t(a.nbytes)))
        return p

    y = np.zeros((T, N), np.int16)
    dw, dx, dc, ds, dy, ws = put(w), put(xb), alloc(N * K // 2), alloc(n_s), alloc(y.nbytes), alloc(n_ws)
    moe.moe_mx_quantize(rows, dw, dc, ds, stream=0)
    for _ in range(2):
        moe.moe_mx_linear(shape, dx, None, dc, ds, None, None, dy, ws, stream=0, ws_bytes=n_ws)
        assert current() == own.value, "another context is current"
    ok(cu.cuCtxSynchronize())
    moe.moe_check_device_status(ws, stream=0)
    ok(cu.cuMemcpyDtoH_v2(y.ctypes.data_as(vp), u64(dy), ctypes.c_size_t(y.nbytes)))
    near(y)
    assert current() == own.value
    ok(cu.cuCtxDestroy_v2(own))


in_thread(work)
print("done")
"""

NONE = COMMON + """
dev = [torch.from_numpy(w).cuda(), x.cuda(), torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"),
       torch.empty(n_s, dtype=torch.uint8, device="cuda"), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda"),
       torch.zeros(n_ws, dtype=torch.uint8, device="cuda")]
moe.moe_mx_quantize(rows, dev[0], dev[2], dev[3])
torch.cuda.synchronize()
primary = current()
dw, dx, dc, ds, dy, ws = (t.data_ptr() for t in dev)


def work():
    for _ in range(2):  # none yet; then taken off again
        assert current() is None
        moe.moe_mx_linear(shape, dx, None, dc, ds, None, None, dy, ws, stream=0, ws_bytes=n_ws)
        assert current() == primary
        ok(cu.cuCtxSynchronize())
        near(dev[4].view(torch.int16).cpu().numpy())
        dev[4].zero_()
        ok(cu.cuCtxSynchronize())
        ok(cu.cuCtxSetCurrent(None))


in_thread(work)
print("done")
"""


@pytest.mark.parametrize("script", [NONE, OWN], ids=["none", "own"])
def test_the_caller_s_context(script):
    from routed_expert_ffn_moe_gb300 import build
    build.build()
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    out = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, env=env, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "done", out.stderr[-2000:]
