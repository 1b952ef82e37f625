"""Failure detection of the paged attention kernels without faulting the GPU:
one key tile is left unloaded (fa_test_set_stall), the waits on it run out, the
call reports FA_ERR_TIMEOUT and the next call is right.  Covers the step
kernel, the tile kernel on a sequence's own rows (line and drawn units) and on
a shared prefix."""

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
from tests.test_paged_gpu import make_batch
which, unit = {which!r}, {unit}
Nq = dict(steps=2, tiles=300, prefix=3)[which]
lens = [700, 650, 1500]
q, kp, vp, table = make_batch(3, 4, 2, Nq, 128, 64, lens, seed=1)
for b in range(3):
    table[b, :4] = table[0, :4]
dev = [t.cuda() for t in (q, kp, vp, table)]
lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
stream = torch.cuda.current_stream().cuda_stream

def run():
    if which == "prefix":
        return fa.forward_shared_prefix(dev[0], dev[1], dev[2], dev[3][0, :4].contiguous(), 256, dev[3], lk)
    return fa.forward_paged(*dev, lk)

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


@pytest.mark.parametrize("which,unit,sites", [
    ("steps", 0, (73, 74)),
    ("steps", 3, (73, 74)),
    ("tiles", 0, (75, 76, 77, 78, 79, 80)),
    ("prefix", 0, (73, 74, 75, 76, 77, 78, 79, 80)),
])
def test_stalled_wait_reports_timeout_and_recovers(which, unit, sites):
    env = dict(os.environ, FA_WAIT_LIMIT_MS="300")
    env.pop("FA_TEST_STALL_UNIT", None)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, which=which, unit=unit)], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    res = json.loads(next(l for l in r.stdout.splitlines() if l.startswith("RESULT "))[7:])
    assert res["stalled_status"] == 5, res          # FA_ERR_TIMEOUT
    assert res["failure"][0] == 5 and res["failure"][1] in sites, res
    assert res["failure"][2] == (unit if which == "steps" else 0), res  # the CTA whose tile was left out
    assert res["seconds"] < 30, res
    assert res["after_status"] == 0 and res["same"], res


UNITS_SCRIPT = r"""
import json, sys, time
sys.path.insert(0, {root!r})
import torch
import exact_tiled_attention_18_gb300 as fa
from tests.test_paged_gpu import make_batch
B, Hq, Hkv, Nq, d, page, lens, unit = {case!r}
q, kp, vp, table = make_batch(B, Hq, Hkv, Nq, d, page, lens, seed=1)
dev = [t.cuda() for t in (q, kp, vp, table)]
lk = torch.tensor(lens, dtype=torch.int32, device="cuda")
stream = torch.cuda.current_stream().cuda_stream
good = fa.forward_paged(*dev, lk)
assert fa.fa_sync_status(stream) == 0
out = dict()
fa.fa_test_set_stall(unit)
t0 = time.time()
fa.forward_paged(*dev, lk)
out["stalled_status"] = fa.fa_sync_status(stream)
out["seconds"] = time.time() - t0
out["failure"] = fa.fa_last_failure()
fa.fa_test_set_stall(-1)
again = fa.forward_paged(*dev, lk)
out["after_status"] = fa.fa_sync_status(stream)
out["same"] = bool(torch.equal(good[0], again[0]) and torch.equal(good[1], again[1]))
print("RESULT " + json.dumps(out))
"""


@pytest.mark.parametrize("what,case", [
    # five units for every CTA of 152, all of one length: CTA 0 has one or two pieces of the line, the third is drawn
    ("behind the line", (38, 20, 20, 257, 64, 64, [700] * 38, 2)),
    ("all drawn, the first", (1, 20, 20, 4096, 64, 64, [4096], 0)),
    ("all drawn, the second", (1, 20, 20, 4096, 64, 64, [4096], 1)),
    ("two row tiles on the same rows", (3, 4, 2, 32, 128, 64, [700, 650, 1500], 0)),
])
def test_stalled_unit_reports_timeout_and_recovers(what, case):
    """The tile kernel's other ways to a unit: drawn from the counter, and two
    row tiles on the same rows."""
    env = dict(os.environ, FA_WAIT_LIMIT_MS="300")
    env.pop("FA_TEST_STALL_UNIT", None)
    r = subprocess.run([sys.executable, "-c", UNITS_SCRIPT.format(root=ROOT, case=case)], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    res = json.loads(next(l for l in r.stdout.splitlines() if l.startswith("RESULT "))[7:])
    assert res["stalled_status"] == 5, res          # FA_ERR_TIMEOUT
    assert res["failure"][0] == 5 and res["failure"][1] in (75, 76, 77, 78, 79, 80), res
    assert res["failure"][2] == 0, res              # the CTA whose tile was left out
    assert res["seconds"] < 30, res
    assert res["after_status"] == 0 and res["same"], res
