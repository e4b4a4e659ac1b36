"""The bounded waits of the drafted tokens' attention, driven to run out.

A test-only build of the library (build.build_starve: waits give up after 2 ms)
runs in a subprocess.  There one warp of thread block 0 does not tell of its part of
the first queries.  The call must report MSA_ERR_TIMEOUT within a second, its thread
blocks must end, and the same call without that must then give the bits that it gave
before.

No wait here is unbounded: a starved wait gives up after 2 ms, every role leaves its
loop on the thread block's abort flag, and copies and products under way are waited
for with a limit before the block ends.
"""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys, time, ctypes
sys.path.insert(0, ROOT)
import torch
from block_sparse_gqa_msa_gb300 import api, build
api.LIB_PATH = build.build_starve()
lib = api.lib()
lib.msa_test_starve.argtypes = [ctypes.c_int32]
lib.msa_test_starve.restype = ctypes.c_int32
dev = "cuda:0"
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)

def run(dtype, dim, kv, share, S, lens, trees, sparse):
    gen = torch.Generator(device=dev).manual_seed(3)
    rows = len(lens)
    need = [-(-(n + m) // S) for n, m in zip(lens, trees)]
    pool, width = sum(need), max(need)
    order, table, at = torch.randperm(pool, generator=gen, device=dev).tolist(), [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (width - n))
        at += n
    offs = [0]
    for m in trees:
        offs.append(offs[-1] + m)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev).to(dtype)
    cache = api.PagedCache(rnd(pool, S, kv, dim), rnd(pool, S, kv, dim))
    q2k = None
    if sparse:
        q2k = torch.full((kv, offs[-1], 16), -1, dtype=torch.int32, device=dev)
        for r, n in enumerate(lens):
            blocks = min(16, -(-n // 128))
            q2k[:, offs[r]:offs[r + 1], :blocks] = torch.arange(blocks, device=dev, dtype=torch.int32)
    args = (cache, rnd(offs[-1], kv * share, dim), i32(table), i32(offs), i32(lens), 0.1)
    call = lambda: api.msa_paged_tree(*args, q2k=q2k)
    status = lambda: api.msa_paged_read_status(cache, clear=True)
    assert lib.msa_test_starve(0) == 0
    o, lse = call()
    assert status() == 0
    assert lib.msa_test_starve(4) == 0
    torch.cuda.synchronize()
    t0 = time.time()
    call()
    st = status()
    seconds = time.time() - t0
    assert lib.msa_test_starve(0) == 0
    o1, lse1 = call()
    return {"status": st, "seconds": seconds, "after": status(),
            "same": bool(torch.equal(o, o1) and torch.equal(lse, lse1))}

bf, fp = torch.bfloat16, torch.float16
out = {
    # a tile a thread block: the copying warps are done before the wait runs out
    "short": run(bf, 128, 4, 16, 64, [100], [8], False),
    # both slots, and more tiles than the rings hold
    "long": run(bf, 128, 4, 16, 64, [20000] * 6, [64] * 6, False),
    # slots that share a tile, heads of 64 channels
    "split": run(fp, 64, 8, 3, 16, [9000] * 20, [5] * 20, False),
    # pages too small for tensor copies
    "pages": run(fp, 64, 2, 3, 4, [3000, 500], [5, 64], False),
    "blocks": run(bf, 128, 4, 16, 128, [5000] * 9, [16] * 9, True),
}
out["matmul"] = float((torch.ones(256, 256, device=dev) @ torch.ones(256, 256, device=dev))[0, 0])
print("RESULT " + json.dumps(out))
"""


def test_starved_waits_report_timeout_and_leave_nothing_behind():
    r = subprocess.run([sys.executable, "-c", CHILD.replace("ROOT", repr(ROOT))],
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    line = [x for x in r.stdout.splitlines() if x.startswith("RESULT ")][-1]
    res = json.loads(line[len("RESULT "):])
    assert res.pop("matmul") == 256.0
    assert len(res) == 5
    for name, got in res.items():
        assert got["status"] == 8, (name, got)   # MSA_ERR_TIMEOUT
        assert got["seconds"] < 1.0, (name, got)
        assert got["after"] == 0 and got["same"], (name, got)
