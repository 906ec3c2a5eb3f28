"""What a failed call of the low-bit operators leaves behind: nothing."""
import os
import subprocess
import sys

import pytest

from codebook_decode_gb300 import qtts

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Calls that wait for the device are refused by the runtime while a stream is captured, and end the capture. In a
# process of its own: torch's capture fails with it.
IN_CAPTURE = """
import numpy as np, torch
from codebook_decode_gb300 import qtts

c = qtts.qtts_kv8_create(qtts.Kv8Config(1, 2, 2, 64, 1e6, 16, 2, 64, 8))
w = qtts.qtts_w4_create(64, 64, 64)
ones = np.full((64, 64), 0x3f80, np.uint16)
qtts.qtts_w4_quantize(w, ones)
q, s = np.zeros((64, 64), np.int8), np.zeros((64, 1), np.uint16)
x = torch.zeros(4, device="cuda")

def call(what):
    try:
        return what()
    except qtts.QttsError as e:
        return e.code

calls = {"status": lambda: qtts.qtts_kv8_status(c, raise_on_error=False)[0],
         "quantize": lambda: call(lambda: qtts.qtts_w4_quantize(w, ones)),
         "export": lambda: call(lambda: qtts.qtts_w4_export(w, q, s)),
         "create": lambda: call(lambda: qtts.qtts_w4_create(64, 64, 64) and 0),
         "create_kv8": lambda: call(lambda: qtts.qtts_kv8_create(qtts.Kv8Config(1, 2, 2, 64, 1e6, 16, 2, 64, 8)) and 0)}
rc = []
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        x.add_(1)
        rc.append(calls["%s"]())
except RuntimeError:
    pass
print(rc[0])
for what in calls.values():
    print(what())
qtts.qtts_w4_export(w, q, s)
print(int((q == 7).all()))
"""


@pytest.mark.parametrize("name", ["status", "quantize", "export", "create", "create_kv8"])
def test_a_call_refused_during_a_capture_leaves_no_error_for_the_next(name):
    r = subprocess.run([sys.executable, "-c", IN_CAPTURE % name], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-800:]
    # an error of the runtime, not one of memory; then every call as if nothing had been
    assert r.stdout.split() == [str(qtts.QTTS_E_CUDA), "0", "0", "0", "0", "0", "1"]
