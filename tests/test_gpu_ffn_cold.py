"""A process whose first calls of the feed-forward and 4-bit operators are captured into a graph, or come
from several threads at once: what a first call asks of the GPU and sets up does not disturb either."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = """
import sys, threading
import torch
import dense_fp32_gemm_05_gb300 as sg
gen = torch.Generator(device="cuda").manual_seed(0)
rand = lambda *s: torch.randn(s, device="cuda", generator=gen)
BF = torch.bfloat16
D, F = 256, 1024
gate, up, down = (rand(F, D) / 16).to(BF), (rand(F, D) / 16).to(BF), (rand(D, F) / 32).to(BF)
few, many, dy = rand(5, D).to(BF), rand(300, D).to(BF), rand(300, D).to(BF)
w = rand(600, D)

def calls():
    out = [sg.ffn(few, gate, up, down)[0], sg.ffn(many, gate, up, down)[0]]
    for keep in (BF, torch.float8_e4m3fn):
        y, kept = sg.ffn(many, gate, up, down, keep=keep)
        out += [y, *sg.ffn_backward(dy, many, gate, up, down, kept)]
    for group in (32, 64, 128):
        for symmetric in (True, False):
            q, s, z = sg.q4_quantize(w, group, symmetric)
            out += [sg.q4_gemm(x, q, s, Z=z, group=group) for x in (few, few.float(), many[:30], many[:70])]
    return out

def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
"""

CAPTURED = COMMON + """
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert same(got, calls()), "captured first"
"""

THREADS = COMMON + """
torch.cuda.synchronize()
got, start = {}, threading.Barrier(4)
def run(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        got[i] = [calls() for _ in range(3)]
        torch.cuda.current_stream().synchronize()
threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
for t in threads: t.start()
for t in threads: t.join()
want = calls()
assert len(got) == 4 and all(same(out, want) for outs in got.values() for out in outs), "threads"
assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
"""


@pytest.mark.parametrize("program", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(program):
    env = dict(os.environ, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
