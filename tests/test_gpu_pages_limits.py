"""The pages' entry points on the GPU at the ends of their ranges, against plain loops over
the definitions."""
import os
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
