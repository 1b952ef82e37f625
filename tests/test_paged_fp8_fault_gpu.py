"""Failure detection of the paged attention kernels over a cache in E4M3 without
faulting the GPU: one key tile is left unloaded (fa_test_set_stall), the waits on
it run out, the call reports FA_ERR_TIMEOUT and the next call is right."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import json, sys, time
sys.path.insert(0, {root!r})
import torch
import exact_tiled_attention_18_gb300 as fa
from tests.test_paged_fp8_gpu import make_batch
B, Hq, Hkv, Nq, d, page, lens, prefix, unit = {case!r}
q, c = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=1)
n = prefix // page
for b in range(B):
    c.table[b, :n] = c.table[0, :n]
k, v, ks, vs, table = c.cuda()
q = q.cuda()
lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
stream = torch.cuda.current_stream().cuda_stream

def run():
    if prefix:
        return fa.forward_shared_prefix_fp8(q, k, v, ks, vs, table[0, :n].contiguous(), prefix, table, lk)
    return fa.forward_paged_fp8(q, k, v, ks, vs, table, lk)

good = run()
assert fa.fa_sync_status(stream) == 0
out = dict()
fa.fa_test_set_stall(unit)
t0 = time.time()
run()
out["stalled_status"] = fa.fa_sync_status(stream)
out["seconds"] = time.time() - t0
out["failure"] = fa.fa_last_failure()
fa.fa_test_set_stall(-1)
again = run()
out["after_status"] = fa.fa_sync_status(stream)
out["same"] = bool(torch.equal(good[0], again[0]) and torch.equal(good[1], again[1]))
print("RESULT " + json.dumps(out))
"""

STEPS, TILES = (82, 83), (75, 76, 77, 78, 79, 80, 84)


@pytest.mark.parametrize("what,case,sites", [
    ("steps", (3, 4, 2, 2, 128, 64, [700, 650, 1500], 0, 0), STEPS),
    ("steps, a later CTA", (3, 4, 2, 2, 128, 64, [700, 650, 1500], 0, 3), STEPS),
    ("steps of 24 rows", (3, 8, 2, 6, 64, 16, [700, 650, 1500], 0, 1), STEPS),
    ("tiles", (3, 4, 2, 300, 128, 64, [700, 650, 1500], 0, 0), TILES),
    ("tiles, d = 64", (3, 4, 2, 300, 64, 16, [700, 650, 1500], 0, 0), TILES),
    ("tiles, two row tiles on the same rows", (3, 4, 2, 32, 128, 64, [700, 650, 1500], 0, 0), TILES),
    ("tiles, drawn", (38, 20, 20, 257, 64, 64, [700] * 38, 0, 2), TILES),
    ("prefix", (3, 4, 2, 3, 128, 64, [700, 650, 1500], 256, 0), STEPS + TILES),
], ids=lambda x: x.replace(" ", "-") if isinstance(x, str) else "")
def test_stalled_wait_reports_timeout_and_recovers(what, case, sites):
    env = dict(os.environ, FA_WAIT_LIMIT_MS="300")
    env.pop("FA_TEST_STALL_UNIT", None)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, case=case)], env=env, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    res = json.loads(next(line for line in r.stdout.splitlines() if line.startswith("RESULT "))[7:])
    assert res["stalled_status"] == 5, res          # FA_ERR_TIMEOUT
    assert res["failure"][0] == 5 and res["failure"][1] in sites, res
    assert res["failure"][2] == (case[-1] if sites == STEPS else 0), res  # the CTA whose tile was left out
    assert res["seconds"] < 30, res
    assert res["after_status"] == 0 and res["same"], res
