"""GPU: serving calls captured into CUDA graphs: behind nodes of every kind, and
as the first calls of a process."""
import os
import subprocess
import sys

import pytest
import torch

import block_sparse_masked_tile_b200 as bsmt
from tests.serving_helpers import Both, ints, queries

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "kernel", "join", "itself", "wait"])
def test_attention_behind_nodes_of_every_kind(before):
    b = Both(400, 2, 64, 2, 200, 64, 1, "e4m3")
    b.add([0, 1], [9000, 300])
    source, q, seqs = queries(2, 8, 64).cuda(), torch.zeros((2, 8, 64), dtype=torch.bfloat16, device="cuda"), ints([1, 0])
    out, lse = torch.empty_like(q), torch.empty((8, 2), device="cuda")
    junk = torch.empty(1 << 20, device="cuda")
    side = torch.cuda.Stream()
    attend = lambda x: bsmt.paged_attention(x, b.dev, seqs, mask_mod=bsmt.causal(), enable_gqa=True, out=out, lse=lse)  # noqa: E731
    want = [t.clone() for t in attend(source)]
    other = torch.randn_like(source)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        now = torch.cuda.current_stream()
        if before == "nothing":
            x = source
        elif before == "copy":
            x = q.copy_(source)
        elif before == "fill":
            junk.zero_()
            x = source
        elif before == "kernel":
            x = torch.add(source, 0.0, out=q)
        elif before == "join":  # two nodes in front, of two streams
            side.wait_stream(now)
            with torch.cuda.stream(side):
                junk.mul_(2.0)
                torch.add(source, 0.0, out=q)
            junk[:100].add_(1.0)
            now.wait_stream(side)
            x = q
        elif before == "itself":
            attend(other)
            x = source
        else:  # another stream alone
            side.wait_stream(now)
            with torch.cuda.stream(side):
                q.copy_(source)
            now.wait_stream(side)
            x = q
        attend(x)
    for _ in range(5):
        q.zero_()
        out.fill_(3.0)
        lse.fill_(3.0)
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    bsmt.check_device_status()


FIRST = """
import torch, block_sparse_masked_tile_b200 as bsmt
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
c = bsmt.create_paged_cache(20, 2, 64, 4, 4, 16)
x = torch.randn((8, 8, 64), device="cuda").bfloat16()
seqs, counts, cu, pos = i(0, 2), i(5, 3), i(0, 5, 8), torch.arange(8, dtype=torch.int32, device="cuda")
src, dst, gone = i(0), i(1), i(2)
spec, mask = bsmt.rotary_spec(64), bsmt.causal()
call = {
    "rotary": lambda: bsmt.rotary(x[:, :4], x[:, 4:6], pos, spec),
    "extend": lambda: bsmt.cache_extend(c, seqs, counts),
    "write": lambda: bsmt.cache_write(c, seqs, i0, x[:, 4:6], x[:, 6:], cu),
    "attend": lambda: bsmt.paged_attention(x[:, :4].contiguous(), c, seqs, cu, mask, enable_gqa=True),
    "gather": lambda: bsmt.cache_gather(c, seqs, None, 8, cu),
    "fork": lambda: bsmt.cache_fork(c, src, dst),
    "free": lambda: bsmt.cache_free(c, gone),
    "compact": lambda: bsmt.cache_compact(c),
}[WHAT]
i0 = i(0, 0)
if WHAT in ("write", "attend", "gather", "fork", "free"):
    c.page_table[0, 0], c.page_table[2, 0] = 3, 4
    c.seq_lens[0], c.seq_lens[2] = 5, 3
    c.ref_counts[3:5] = 1
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
bsmt.check_device_status()
print("ran")
"""


@pytest.mark.parametrize("what", ["rotary", "extend", "write", "attend", "gather", "fork", "free", "compact"])
def test_the_first_call_of_a_process_is_captured(what):
    got = subprocess.run([sys.executable, "-c", f"WHAT = {what!r}\n" + FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip().endswith("ran"), got.stderr[-2000:]


REFUSED = """
import torch, block_sparse_masked_tile_b200 as bsmt
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
c = bsmt.create_paged_cache(20, 2, 64, 4, 4, 16)
q, seqs = torch.randn((2, 4, 64), device="cuda").bfloat16(), i(0, 2)
out, lse = torch.empty_like(q), torch.empty((4, 2), device="cuda")
ws = torch.empty(bsmt.paged_attention_workspace_bytes(64), dtype=torch.uint8, device="cuda")
call = lambda: bsmt.paged_attention(q, c, seqs, enable_gqa=True, out=out, lse=lse, workspace=ws)
call()
bsmt.cache_free(c, seqs)
torch.cuda.synchronize()
side, other, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()

def fails(f):
    try:
        f()
    except Exception as e:
        return str(e)
    raise SystemExit("no error")

with torch.cuda.stream(side):
    g.capture_begin()
    fails(torch.cuda.synchronize)  # not allowed during a capture: it ends there
    assert "CUDA_ERROR" in fails(call)
    with torch.cuda.stream(other):
        bsmt.cache_free(c, seqs)  # outside the capture: as ever
    fails(g.capture_end)
torch.cuda.synchronize()
bsmt.check_device_status()
print("ran")
"""


def test_a_refused_launch_leaves_no_error_behind():
    got = subprocess.run([sys.executable, "-c", REFUSED], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip().endswith("ran"), got.stdout[-500:] + got.stderr[-2000:]
