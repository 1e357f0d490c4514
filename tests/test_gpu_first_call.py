"""The library's calls as the first GPU work of a process: torch not yet initialised, a kernel's
first launch inside a capture, two host threads at once (each case in a process of its own)."""
import os
import subprocess
import sys

import pytest

from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import threading, torch
import pose_retrieved_kv_b200 as P
pg = P.make_paged(n_seqs=2, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=90,
                  max_pages=45)
def call():
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    a = dict(q=bf(2, 4, 64), k=bf(2, 2, 64), v=bf(2, 2, 64), kp=bf(90, 2, 16, 64),
             vp=bf(90, 2, 16, 64), qr=bf(2, 4, 64), out=bf(2, 4, 64),
             table=torch.arange(90, device="cuda").int().reshape(2, 45),
             lens=torch.tensor([700, 33], device="cuda").int(), scratch=torch.empty(
                 P.prsink_paged_attention_scratch_bytes(pg), dtype=torch.uint8, device="cuda"))
    def run():
        P.prsink_paged_append(pg, a["k"], a["v"], a["kp"], a["vp"], a["table"], a["lens"],
                              q=a["q"], q_rot=a["qr"])
        P.prsink_paged_attention(pg, a["qr"], a["kp"], a["vp"], a["table"], a["lens"], a["out"],
                                 a["scratch"])
    return a, run
"""

CASES = {
    "status of a process without a context": """
assert not torch.cuda.is_initialized()
assert P.prsink_sync_status() == P.PRSINK_OK
assert torch.cuda.is_initialized()
""",
    "first launch inside a capture": """
a, run = call()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
assert P.prsink_sync_status() == P.PRSINK_OK
b, run = call()
run()
torch.cuda.synchronize()
assert torch.isfinite(b["out"].float()).all()
assert all(torch.equal(a[x], b[x]) for x in ("kp", "vp", "qr", "out"))
""",
    "two host threads": """
calls = [call() for _ in range(2)]
torch.cuda.synchronize()
errors = []
def work(run):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                run()
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=work, args=(run,)) for _, run in calls]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors and P.prsink_sync_status() == P.PRSINK_OK
assert all(torch.equal(calls[0][0][x], calls[1][0][x]) for x in ("kp", "vp", "qr", "out"))
""",
}


@pytest.mark.parametrize("name", CASES)
def test_first_calls(name):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", SETUP + CASES[name]], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
