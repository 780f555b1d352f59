"""A call that throws between giving the interpreter's lock away and taking it
back: a tensor without memory throws where its pointer is read, with the lock
away.  In a process of its own, since one that goes on without the lock ends."""

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))

CODE = """
import sys, threading
sys.path[:0] = [{here!r}, {root!r}]
import torch
import fp8_fine_grained_quant_amd as fq
from fake_device import NO_MEMORY, current_device, hollow

i32, u8 = torch.int32, torch.uint8
x, rows, ids, w = hollow(6, 32), hollow(24, 32), hollow(6, 4, dt=i32), hollow(6, 4)
calls = [lambda: fq.fp8q_moe_route(x, ids, w),
         lambda: fq.fp8q_moe_route_bwd(w, x, ids, hollow(6, 32)),
         lambda: fq.fp8q_moe_sort(ids, 8, hollow(9, dt=i32), ids, hollow(24, dt=i32)),
         lambda: fq.fp8q_moe_dispatch(x, ids, rows, hollow(24, 32, dt=u8), hollow(24, 1)),
         lambda: fq.fp8q_moe_dispatch_bwd(rows, ids, x),
         lambda: fq.fp8q_moe_combine(rows, ids, w, x),
         lambda: fq.fp8q_moe_combine_bwd(x, rows, ids, w, w, rows),
         lambda: fq.fp8q_grad_clip([], [], 1.0, hollow(), hollow(8, dt=u8))]
with current_device(0):
    for i, call in enumerate(calls):
        try:
            call()
        except RuntimeError as e:
            assert NO_MEMORY in str(e), (i, e)
        else:
            raise SystemExit(f"call {{i}} did not throw")
        # another thread runs, and this one after it
        seen = []
        t = threading.Thread(target=lambda: seen.append(i))
        t.start()
        t.join()
        assert seen == [i]
print("ended well")
"""


def test_lock_comes_back():
    code = CODE.format(here=HERE, root=os.path.dirname(HERE))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split("\n")[-2] == "ended well", (r.returncode, r.stdout, r.stderr)
