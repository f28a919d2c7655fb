"""The binding of the block-scaled cache's calls on the host: what it has to
refuse, and what it must not.  No compute call is made here."""
import glob
import os

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4


def arguments(kind):
    x = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    c = torch.zeros(2, 16, 1, 64, dtype=torch.uint8).view(kind)
    return dict(x=x, c=c, bt=torch.zeros(1, 1, dtype=torch.int32),
                seq=torch.ones(1, 2, dtype=torch.int32), sc=torch.ones(2, 2, 1, 1),
                ids=torch.zeros(1, 1, 1, 1, dtype=torch.int32),
                bd=torch.zeros(2, 1, 1, 2, 64, dtype=torch.uint8).view(kind),
                scores=torch.zeros(1, 1, 1, 1), ws=torch.zeros(1024, dtype=torch.uint8))


CALLS = {
    "append": lambda a, **kw: vae4.verify_attn_e4m3_append(
        a["x"], a["x"], a["c"], a["c"], a["bt"], a["seq"], a["sc"], k_bounds=a["bd"], **kw),
    "attend": lambda a, **kw: vae4.verify_attn_e4m3_block_scaled(
        a["x"], a["c"], a["c"], a["bt"], a["seq"], a["sc"], a["x"], a["ws"], **kw),
    "sparse": lambda a, **kw: vae4.verify_attn_e4m3_sparse(
        a["x"], a["c"], a["c"], a["bt"], a["seq"], a["sc"], a["ids"], a["x"], a["ws"], **kw),
    "scores": lambda a, **kw: vae4.verify_attn_e4m3_block_scores(
        a["x"], a["bd"], a["bt"], a["seq"], a["sc"], a["scores"], block_tokens=16, **kw),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_fp8_types_have_to_agree_with_the_flags(name):
    """An E5M2 tensor without the flag, or an E4M3 one with it, would be read
    (or written) in the other format.  The right ones and uint8 get as far as
    the check of the device."""
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    for kind, flags in ((e5, 0), (e4, vae4.FLAG_KV_E5M2)):
        with pytest.raises(TypeError, match="other FP8 format"):
            CALLS[name](arguments(kind), flags=flags)
    for kind, flags in ((e4, 0), (e5, vae4.FLAG_KV_E5M2), (torch.uint8, 0),
                        (torch.uint8, vae4.FLAG_KV_E5M2)):
        with pytest.raises(ValueError, match="device"):
            CALLS[name](arguments(kind), flags=flags)


class OnDevice:
    """What the binding asks of a CUDA tensor, on a device that need not exist."""

    def __init__(self, t, device):
        self.t, self.device = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device

    @property
    def is_cuda(self):
        return self.device >= 0

    def data_ptr(self):
        return 0x100000


@pytest.mark.parametrize("name", ["append", "scores", "select"])
def test_status_has_to_be_on_the_current_device(name, monkeypatch):
    """Device 0 is current: a status word on device 1 or on the host is refused
    before the library is called; one on device 0 reaches it."""
    a = {k: OnDevice(t, 0) for k, t in arguments(torch.uint8).items()}
    calls = dict(CALLS, select=lambda a, **kw: vae4.verify_attn_e4m3_select_blocks(
        a["scores"], a["seq"], a["ids"], block_tokens=16, **kw))
    reached = []

    class Library:
        def __getattr__(self, fn):
            return lambda *args: reached.append(fn) or 0

    with pytest.raises(ValueError):  # (looks up what it needs of torch)
        vae4.verify_attn_e4m3_select_blocks(*[arguments(torch.uint8)[k] for k in ("scores", "seq", "ids")],
                                            block_tokens=16)
    monkeypatch.setattr(vae4, "_lib", Library())
    monkeypatch.setattr(vae4, "_device", lambda: 0)
    monkeypatch.setattr(vae4, "_raw_stream", lambda dev: 0)
    word = torch.zeros(1, dtype=torch.int32)
    for wrong in (OnDevice(word, 1), word, OnDevice(word.float(), 0), OnDevice(word[:0], 0)):
        with pytest.raises(ValueError, match="status"):
            calls[name](a, status=wrong)
    assert not reached
    for right in (None, OnDevice(word, 0)):
        calls[name](a, status=right)
    assert len(reached) == 2


@pytest.mark.parametrize("shape,both", [
    ((1024, 8, 8, 1, 128, 1 << 23), False),
    ((8192, 64, 8, 1, 128, 1 << 20), False),
    ((65535, 8, 8, 1, 128, 1 << 17), False),
    ((2, 12, 2, 8, 128, 4096), True),
])
def test_a_workspace_for_every_batch_of_the_head_scaled_calls(shape, both, monkeypatch):
    """Batches past the block-scaled plan's line of 2^30 places get the
    head-scaled calls' workspace; others one that serves both."""
    head, blocked = vae4.workspace_bytes, vae4.block_scaled_workspace_bytes
    monkeypatch.setattr(vae4, "workspace_bytes", lambda *a: head(*a, num_sms=152))
    monkeypatch.setattr(vae4, "block_scaled_workspace_bytes", lambda *a: blocked(*a, num_sms=152))
    monkeypatch.setattr(torch, "zeros", lambda n, **kw: n)
    n = vae4.alloc_workspace(*shape, device="cpu")
    if both:
        assert n == max(head(*shape, num_sms=152), blocked(*shape, num_sms=152))
    else:
        with pytest.raises(vae4.Vae4Error):
            blocked(*shape, num_sms=152)
        assert n == head(*shape, num_sms=152)
    with pytest.raises(vae4.Vae4Error):  # what no call takes
        vae4.alloc_workspace(1, 7, 2, 1, 128, 4096, device="cpu")


def test_dependent_kernels_read_their_inputs_coherently():
    """A kernel launched as a programmatic dependent is there while the kernels
    before it write its inputs: the read-only path, which is not coherent with
    such writes, is not for it."""
    csrc = os.path.join(os.path.dirname(vae4.__file__), "csrc")
    files = [f for name in ("append.cu", "block_*.cu", "select_blocks.cu", "seg_*.cu*")
             for f in glob.glob(os.path.join(csrc, name))]
    assert len(files) >= 9
    for f in files:
        text = open(f).read()
        assert "__ldg(" not in text and "ld.global.nc" not in text, f


def test_workspace_sizes_refuse_rows_past_32_bits():
    """2^32 + 16 rows are not 16."""
    for fn in (lambda *a: vae4.block_scaled_workspace_bytes(*a, 152),
               lambda *a: vae4.sparse_workspace_bytes(*a, 16, 4, 152)):
        with pytest.raises(vae4.Vae4Error, match="UNSUPPORTED"):
            fn(1, (1 << 28) + 1, 1, 16, 64, 1000)
        assert fn(1, 1, 1, 16, 64, 1000) > 0


def test_profiled_sources_hold_the_head_scaled_kernels_alone():
    """bench.py reports the head-scaled kernel's DRAM traffic while the sources
    that were profiled are unchanged: what only the block-scaled kernels use
    stays out of them, or a change there would void the record."""
    import bench
    for rel in bench.SPLIT_SOURCES:
        text = open(os.path.join(bench.ROOT, rel)).read()
        for name in ("SegParams", "AppendParams", "ScoreParams", "SelectParams", "ListParams",
                     "launch_dependent(", "elect_one", "mbar_wait_brief"):
            assert name not in text, (rel, name)
