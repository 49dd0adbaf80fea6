"""Tree, compaction and reordering calls made in ways of their own: the first
ones of a process inside a stream capture, and from two host threads at once."""

import os
import subprocess
import sys
import threading

import pytest
import torch

from cross_layer_kv_gb300 import fusedkv as B
from tree_parity import TreeSetup

pytestmark = pytest.mark.gpu

CHILD = """
import os, sys
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, os.path.join(sys.argv[1], "tests"))
import torch
from cross_layer_kv_gb300 import fusedkv as B
from tree_parity import TreeSetup

s = TreeSetup(fmt=sys.argv[2], T=12, lens=(100, 700, 1200), S=1400)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
idx, counts = i32([[3, 1], [0, 2], [1, 1]]), i32([2, 2, 2])
src, lens = i32([1, 2, 0]), i32([1400, 300, 0])
before = {l: (s.k[l].clone(), s.v[l].clone()) for l in (1, 2)}
side = torch.cuda.Stream()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
    s.run(stream=side)
    s.ctx.fkv_compact_rows(s.seq, idx, counts, stream=side)
    s.ctx.fkv_reorder_seqs(src, lens, stream=side)
assert (s.out == -77).all()
g.replay()
torch.cuda.synchronize()
assert s.ctx.fkv_get_device_status() == B.FKV_OK
after = {l: (s.k[l].clone(), s.v[l].clone()) for l in (1, 2)}
for l in (1, 2):
    s.k[l].copy_(before[l][0])
    s.v[l].copy_(before[l][1])
s.check("captured")
got = s.out.clone()
assert torch.equal(s.run(), got)
s.ctx.fkv_compact_rows(s.seq, idx, counts)
s.ctx.fkv_reorder_seqs(src, lens)
torch.cuda.synchronize()
for l in (1, 2):
    assert torch.equal(s.k[l].view(torch.uint8), after[l][0].view(torch.uint8))
    assert torch.equal(s.v[l].view(torch.uint8), after[l][1].view(torch.uint8))
print("captured first")
"""


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "f32", "q4"])
def test_the_first_calls_of_a_process_are_captured(fmt):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, root, fmt], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout[-500:] + r.stderr[-1500:]


def test_two_host_threads_on_one_context():
    s = TreeSetup(T=12, lens=(100, 700, 1200), S=1400)
    want = {m: s.ctx.fkv_tree_attn(s.q, 3, m, s.seq, s.mask, torch.empty_like(s.q), s.ws).clone()
            for m in ("lite", "fused")}
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(mode):
        try:
            st = torch.cuda.Stream()
            out, ws = torch.empty_like(s.q), s.ctx.tree_workspace(s.T)
            st.wait_stream(torch.cuda.default_stream())
            for _ in range(300):
                s.ctx.fkv_tree_attn(s.q, 3, mode, s.seq, s.mask, out, ws, stream=st)
            st.synchronize()
            got[mode] = out
        except Exception as e:      # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(m,)) for m in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert s.ctx.fkv_get_device_status() == B.FKV_OK
    for m in want:
        assert torch.equal(got[m], want[m])
