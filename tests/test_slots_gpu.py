"""fa_paged_slots against the loop reference: every output exact, untouched table entries intact."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tiled_attention_10_gb300 as fa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _case(seed, n, ps, cols, past_hi, new_hi, total_q, n_free, odd=False):
    g = np.random.default_rng(seed)
    past = g.integers(0, past_hi + 1, n).astype(np.int32)
    new = g.integers(0, new_hi + 1, n).astype(np.int32)
    if odd:                       # lengths no request has: they clamp
        past[:: 5] = -3
        new[1:: 7] = -9
        past[2:: 11] = cols * ps + 100
    ids = g.permutation(n * cols + n_free + 5).astype(np.int32)
    table = ids[: n * cols].reshape(n, cols).copy()
    free = ids[n * cols: n * cols + n_free].copy()
    return past, new, free, table, ps, total_q


CASES = [
    # n, page, cols, past up to, new up to, total_q (None: the sum), free pages (None: enough)
    (1, 16, 1, 0, 1, None, None), (1, 64, 4, 200, 0, None, None), (3, 16, 4, 40, 20, None, None),
    (128, 64, 64, 4000, 1, 128, None), (33, 32, 300, 0, 8192, None, None), (7, 1, 90, 40, 40, None, None),
    (5, 48, 20, 500, 400, None, None), (600, 128, 3, 300, 80, None, None),
    (40, 16, 8, 100, 60, "short", None),        # more tokens than rows
    (40, 16, 8, 100, 60, "padded", None),       # rows of no request
    (40, 16, 20, 100, 100, None, 30),           # the free list runs out
    (40, 16, 8, 100, 100, None, 0),
    (16384, 16, 2, 16, 2, None, None), (513, 16, 4, 30, 30, None, None),
]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_slots(cuda_lib, c, odd):
    n, ps, cols, past_hi, new_hi, total, n_free = c
    past, new, free, table, ps, _ = _case(n + ps, n, ps, cols, past_hi, new_hi, 0, n * cols if n_free is None else n_free, odd)
    rows = int(np.maximum(new, 0).sum())
    total_q = {None: rows, "short": rows // 2, "padded": rows + 77}.get(total, total)
    want = ref.slots(past, new, free, table, ps, total_q)
    d = {k: torch.from_numpy(v).cuda() for k, v in dict(past=past, new=new, free=free, table=table).items()}
    got = fa.paged_slots(d["past"], d["new"], d["free"], d["table"], page_size=ps, total_q=total_q)
    for w, t in zip(want[:2] + want[3:5], (got.cu_seqlens_q, got.seqused_k, got.positions, got.slot_map)):
        assert np.array_equal(w, t.cpu().numpy())
    assert np.array_equal(want[2], d["table"].cpu().numpy())
    assert int(got.pages_taken) == want[5]
    # the same call once more finds the same (the table it wrote is the table it reads)
    again = fa.paged_slots(d["past"], d["new"], d["free"], d["table"], page_size=ps, total_q=total_q)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_slots_no_rows(cuda_lib):
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    past = torch.tensor([0, 5, 16, 17], dtype=torch.int32, device="cuda")
    table = torch.full((4, 2), 9, dtype=torch.int32, device="cuda")
    got = fa.paged_slots(past, z, z[:0], table, page_size=16, total_q=0)
    assert got.cu_seqlens_q.tolist() == [0] * 5 and got.seqused_k.tolist() == [0, 5, 16, 17]
    assert int(got.pages_taken) == 0 and (table == 9).all()


def test_slots_graph_replays_with_new_lengths(cuda_lib):
    past, new, free, table, ps, _ = _case(9, 20, 16, 6, 60, 3, 0, 200)
    d = {k: torch.from_numpy(v).cuda() for k, v in dict(past=past, new=new, free=free, table=table).items()}
    fa.paged_slots(d["past"], d["new"], d["free"], d["table"].clone(), page_size=ps, total_q=64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.paged_slots(d["past"], d["new"], d["free"], d["table"], page_size=ps, total_q=64)
    past2 = np.roll(past, 3)
    d["past"].copy_(torch.from_numpy(past2))
    graph.replay()
    want = ref.slots(past2, new, free, table, ps, 64)
    assert np.array_equal(want[4], got.slot_map.cpu().numpy()) and np.array_equal(want[2], d["table"].cpu().numpy())


def run_alone(code):
    """Python code in a process of its own: no larger launch before it has asked for shared memory."""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


@pytest.mark.parametrize("n", [6111, 6112, 6128, 6143, 6144])
def test_slots_around_48_kb_of_sums(cuda_lib, n):
    run_alone(f"""
import numpy as np, torch, tiled_attention_10_gb300 as fa
from tests import paged_reference as ref
past, new = np.arange({n}, dtype=np.int32) % 40, np.arange({n}, dtype=np.int32) % 3
table, free = np.full(({n}, 3), -1, np.int32), np.arange(2 * {n}, dtype=np.int32)
want = ref.slots(past, new, free, table, 16, int(new.sum()))
d = [torch.from_numpy(a.copy()).cuda() for a in (past, new, free, table)]
got = fa.paged_slots(*d, page_size=16, total_q=int(new.sum()))
for w, t in zip((*want[:5], want[5]), (got.cu_seqlens_q, got.seqused_k, d[3], got.positions, got.slot_map, got.pages_taken)):
    assert np.array_equal(np.asarray(w).reshape(-1), t.cpu().numpy().reshape(-1))
""")
