"""Host-side fault injection (PROJ_FAULT, read once per process) at the decode-step operators' entry
points: each failure becomes its status, nothing leaks, and the context stays usable.  The failure is
made on the host, before anything reaches the device."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, torch
import dense_linear_projection_gb300 as dlp
bf16, dev = torch.bfloat16, "cuda"


def status(f):
    try:
        f()
        return 0
    except dlp.ProjError as e:
        return e.status


def scenario():
    out = {}
    X = torch.zeros((4, 256), dtype=bf16, device=dev)
    codes = torch.zeros((64, 128), dtype=torch.uint8, device=dev)
    scales = torch.zeros((64, 4), dtype=bf16, device=dev)
    proj = dlp.Q4Projection(4, 64, 256, 64)
    packed = torch.zeros(dlp.proj_q4_packed_bytes(64, 256, 64), dtype=torch.uint8, device=dev)
    out["pack"] = status(lambda: proj.pack(codes, scales))
    out["run"] = status(lambda: proj(X, packed))
    proj.close()
    k, v = (torch.zeros((4, 16, 2, 64), dtype=bf16, device=dev) for _ in "kv")
    kv = []
    out["create"] = status(lambda: kv.append(dlp.PagedKV(k, v, 4, 2)))
    if kv:
        rows = torch.zeros((2, 8, 64), dtype=bf16, device=dev)
        ints = torch.zeros(2, dtype=torch.int32, device=dev)
        table = torch.arange(4, dtype=torch.int32, device=dev).view(2, 2)
        out["append"] = status(lambda: kv[0].append(rows[:, :4], rows[:, 4:6], rows[:, 6:], ints, table))
        out["attend"] = status(lambda: kv[0].attend(rows[:, :4], table, ints + 1))
        out["status"] = kv[0].status()
        kv[0].close()
    torch.cuda.synchronize()
    return out


first = scenario()
torch.cuda.synchronize()
torch.cuda.empty_cache()
free = torch.cuda.mem_get_info()[0]
for _ in range(3):
    assert scenario() == first
torch.cuda.empty_cache()
first["leak"] = max(0, free - torch.cuda.mem_get_info()[0])
first["alive"] = (torch.ones(10, device=dev) * 2).sum().item() == 20.0
print("RESULT " + json.dumps(first))
"""


@pytest.mark.parametrize("fault", ["", "alloc", "launch"])
def test_faults(fault):
    import dense_linear_projection_gb300 as dlp
    dlp.build()
    env = {k: v for k, v in os.environ.items() if k != "PROJ_FAULT"}
    if fault:
        env["PROJ_FAULT"] = fault
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    lines = [x for x in r.stdout.splitlines() if x.startswith("RESULT ")]
    assert r.returncode == 0 and lines, r.stdout + r.stderr
    got = json.loads(lines[-1][7:])
    assert got.pop("alive") and got.pop("leak") == 0
    ok, cuda = dlp.PROJ_OK, dlp.PROJ_ERR_CUDA
    launched = cuda if fault == "launch" else ok
    want = {"pack": launched, "run": launched, "create": ok, "append": launched, "attend": launched, "status": ok}
    if fault == "alloc":
        want = {"pack": ok, "run": ok, "create": dlp.PROJ_ERR_OUT_OF_MEMORY}
    assert got == want


def test_handles_of_another_device():
    # Every handle is taken for another device's: each call is refused before anything is launched.
    # (The host's check alone: no launch with addresses of the wrong device is made.)
    import dense_linear_projection_gb300 as dlp
    dlp.build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, PROJ_FAULT="device"), capture_output=True,
                       text=True, timeout=300)
    lines = [x for x in r.stdout.splitlines() if x.startswith("RESULT ")]
    assert r.returncode == 0 and lines, r.stdout + r.stderr
    got = json.loads(lines[-1][7:])
    assert got.pop("alive") and got.pop("leak") == 0 and got.pop("create") == dlp.PROJ_OK
    assert set(got) == {"pack", "run", "append", "attend", "status"} and set(got.values()) == {dlp.PROJ_ERR_INVALID_ARG}
