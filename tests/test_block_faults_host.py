"""The binding of the block-scaled cache's calls on the host: what it has to
refuse, and what it must not.  No compute call is made here."""
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
