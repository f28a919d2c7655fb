"""The pages' entry points on the GPU at the ends of their ranges, against plain loops over
the definitions."""
import os
import random
import subprocess
import sys

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4
from test_gpu_pages import dev, lengths, plain_resize, pool, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


def resize_rows(cols, rows):
    """One call for each number of rows; (table, counts, copies) as they have to be."""
    for B in rows:
        table, counts = pool(B, B, cols, extra=0, share=0, kept=0)
        used = len(counts)
        counts += [0] * min(B, 16384 - used if cols == 1 else B)
        seq = lengths(B, table, 16)
        t, c, st = dev(table), dev(counts), status()
        copies, ws = torch.empty((B, 2), dtype=torch.int32, device="cuda"), vae4.alloc_pages_workspace(len(counts))
        vae4.verify_attn_e4m3_resize_pages(t, dev(seq), c, copies, ws, page_tokens=16, status=st)
        want, wc, wcp, wst = plain_resize(table, counts, seq, 16)
        assert t.tolist() == want and c.tolist() == wc and copies.tolist() == wcp and int(st) == wst, B


@pytest.mark.parametrize("cols,rows", [(1, (6080, 6104, 6105, 6144, 6145, 16384)), (6, (6080, 6081, 6144, 6145, 16384))],
                         ids=["cluster", "grid"])
def test_resize_of_many_rows(cols, rows):
    """Eight bytes a row, and what the kernels hold beside them, pass the 48 KB that a launch
    may have without asking between 6080 and 6145 rows: a call past it asks, in a process
    where none has before."""
    for ask in [rows[2:3], rows]:
        here = os.path.dirname(os.path.abspath(__file__))
        code = (f"import sys; sys.path[:0] = [{os.path.dirname(here)!r}, {here!r}]\n"
                f"import test_gpu_pages_limits as t; t.resize_rows({cols}, {ask})")
        r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]

def full_compact(table, counts, m):
    """The definition: what moves, and the status of all entries whether or not one does."""
    st = 0
    n = sum(c != 0 for c in counts)
    holes = [x for x in range(n) if counts[x] == 0]
    moves = list(zip([x for x in reversed(range(n, len(counts))) if counts[x] > 0], holes))[:m]
    to = dict(moves)
    for row in table:
        for j, e in enumerate(row):
            if e < -1 or e >= len(counts):
                st = vae4.STATUS_BAD_BLOCK
            row[j] = to.get(e, e)
    for a, b in moves:
        counts[b], counts[a] = counts[a], 0
    return table, counts, [list(x) for x in moves] + [[-1, -1]] * (m - len(moves)), st


@pytest.mark.parametrize("B,cols", [(1, 1), (3, 7), (8, 64), (40, 1000), (2, 40000)])
@pytest.mark.parametrize("m", [0, 1, 9])
@pytest.mark.parametrize("moves", [False, True])
@pytest.mark.parametrize("bad", [-2, -2 ** 31, 0, 2 ** 31 - 1, None])
def test_compact_reports_entries_whether_or_not_pages_move(B, cols, m, moves, bad):
    """On one cluster and on the whole GPU; with room in the list or none."""
    r = random.Random(B + m)
    n_pages = B * cols + 30
    ids = r.sample(range(n_pages), B * cols) if moves else list(range(B * cols))
    table = [ids[b * cols:(b + 1) * cols] for b in range(B)]
    counts = [0] * n_pages
    for e in ids:
        counts[e] = 1
    if bad is not None:
        e = table[B - 1][cols - 1]
        table[B - 1][cols - 1] = bad if bad else n_pages
        counts[e] = -1  # kept: the pool is as full as before
    t, c, st = dev(table), dev(counts), status()
    out = torch.full((m, 2), 55, dtype=torch.int32, device="cuda")
    vae4.verify_attn_e4m3_compact_pages(t, c, out, status=st)
    want, wc, wm, wst = full_compact(table, counts, m)
    assert t.tolist() == want and c.tolist() == wc and out.tolist() == wm and int(st) == wst
    assert (wst != 0) == (bad is not None)
