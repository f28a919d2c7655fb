"""Sizes at which a launch's static and dynamic shared memory together first pass the 48 KB
that it may have without asking, each in a process where no call has asked for more."""
import os
import subprocess
import sys

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


def alone(call):
    here = os.path.dirname(os.path.abspath(__file__))
    code = (f"import sys; sys.path[:0] = [{os.path.dirname(here)!r}, {here!r}]\n"
            f"import test_gpu_shared_memory as t; t.{call}")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def pages(cols, D=64):
    """Keys of zeros; the row's entries are pages of values 1, 2 and 4 in turn."""
    k = torch.zeros(3, 16, 1, D, dtype=torch.uint8, device="cuda")
    v = (0x38 + 8 * torch.arange(3, device="cuda")).to(torch.uint8).view(3, 1, 1, 1).expand(3, 16, 1, D).contiguous()
    bt = (torch.arange(cols, device="cuda") % 3).int()[None].contiguous()
    seq = torch.tensor([[16 * cols, 1]], dtype=torch.int32, device="cuda")
    q = torch.ones(1, 1, 1, D, dtype=torch.float16, device="cuda")
    return q, k, v, bt, seq


def sparse(blocks):
    q, k, v, bt, seq = pages(blocks)
    ids = torch.tensor([[[[3, 4, blocks - 1 - (blocks - 1) % 3 - 1]]]], dtype=torch.int32, device="cuda")  # 1, 2, 4
    out = torch.zeros_like(q)
    ws = vae4.alloc_sparse_workspace(1, 1, 1, 1, 64, 16 * blocks, 16, 3)
    vae4.verify_attn_e4m3_sparse(q, k, v, bt, seq, torch.ones(3, 2, 1, 1, device="cuda"), ids, out, ws)
    assert vae4.read_status(ws) == 0
    assert bool(((out.double() - 7 / 3).abs() <= 7 / 3 * 2.0 ** -10).all())  # weights are exact


@pytest.mark.parametrize("blocks", [24512, 24544, 24576, 24584])
def test_visit_lists(blocks):
    alone(f"sparse({blocks})")


def partitions(n):
    q, k, v, bt, seq = pages(n)
    out = torch.zeros_like(q)
    ws = vae4.alloc_workspace(1, 1, 1, 1, 64, 16 * n, 16)
    vae4.verify_attn_e4m3_kv(q, k, v, bt, seq, torch.ones(1, 2, device="cuda"), out, ws, partition_tokens=16)
    assert vae4.read_status(ws) == 0
    assert bool(((out.double() - 7 / 3).abs() <= 7 / 3 * 2.0 ** -10).all())  # n is a multiple of 3


@pytest.mark.parametrize("n", [5625, 5631, 6000, 6144, 6147, 8190])
def test_partitions_of_one_sequence(n):
    alone(f"partitions({n})")
