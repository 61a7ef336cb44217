"""GPU test of calls after one whose launch CUDA refused: an error is reported once, by the
call that met it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

# A wait inside a capture invalidates it (an error on the host, documented for cudaStreamSynchronize),
# and launches into an invalidated capture are refused.  In a process of its own: the capture is lost.
PROGRAM = """
import torch
from w4a16_int4_weight_sigmoid_gb300 import chord
x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
codes = torch.empty((4, 32), dtype=torch.uint8, device="cuda")
scales = torch.empty((4, 2), dtype=torch.uint8, device="cuda")
packed = torch.zeros(chord.chord_mxfp4_prepack_bytes(1, 8, 64), dtype=torch.uint8, device="cuda")
w = [torch.zeros((1, 8, n), dtype=torch.uint8, device="cuda") for n in (32, 2)]
chord.chord_mxfp4_quantize(x, codes, scales)
torch.cuda.synchronize()
graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(s):
    graph.capture_begin()
    try:
        s.synchronize()
    except RuntimeError:
        pass
    try:
        chord.chord_mxfp4_quantize(x, codes, scales)
        raise SystemExit("the launch was not refused")
    except chord.ChordError as e:
        assert e.code == chord.CHORD_ERR_CUDA, e
    try:
        graph.capture_end()
    except RuntimeError:
        pass
chord.chord_mxfp4_prepack(*w, False, packed)
torch.cuda.synchronize()
assert packed[:4].view(torch.int32).item() == 0x4D344843
print("FINE")
"""


def test_a_refused_launch_is_not_the_next_call_s_error():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "FINE" in r.stdout, r.stdout + r.stderr
