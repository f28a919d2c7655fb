"""Chunk attention on the GPU at the ends of its number ranges, against its definition in
64 bits; caches, definition and the derivation of the bound are those of test_gpu_chunk."""
import math

import pytest
import torch

import fp8_paged_attention_e4m3_gb300 as vae4
from test_gpu_blocks import Cache
from test_gpu_chunk import KIND, attend, check, queries, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    vae4.load()


# lens of which rows lie in masked tiles, whole and alone, in one unit and in several
LENS = [(300, 300), (900, 40), (17, 1)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("power,scale_k", [(-100, -40), (-120, -40), (-120, -30), (-133, -40), (-93, -40), (-110, 40)])
def test_small_queries_and_small_scales(D, power, scale_k):
    """BF16 queries of 2^power beside K scales of 2^scale_k: what a score is multiplied with
    may be too small for 32 bits.  All scores are next to zero, hidden keys stay hidden."""
    c = Cache(LENS, 2, D, 32, 16, seed=D)
    c.scales[:, 0] = torch.where(c.scales[:, 0].isnan(), c.scales[:, 0], 2.0 ** scale_k)
    q = (queries(c, 300, 2, "f16").double() * 2.0 ** power).bfloat16()  # (NaN in the padding still)
    q[0, 5] = 0
    got, status = attend(c, q)
    assert status == 0
    check(got, *reference(c, q))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-36, 1e-38, 1e-44])
def test_small_softmax_scales(D, kind, scale):
    c = Cache(LENS, 2, D, 32, 16, seed=D)
    q = queries(c, 300, 2, kind)
    got, status = attend(c, q, softmax_scale=scale)
    assert status == 0
    check(got, *reference(c, q, scale))


FACTORS = [("bf16", 100, 0.0), ("bf16", 120, 0.0), ("f16", 3, 1e30), ("bf16", 60, 1e25)]  # queries, softmax_scale


def past_32_bits(D, lens, signs, kind, power, scale):
    """Queries of one large value; keys of zeros, every other one of the sequence's sign,
    so that a score is 0 or past 2^128."""
    c = Cache(lens, 1, D, 32, 16, seed=D)
    for b, sign in enumerate(signs):
        pg = c.table[b, :-(-lens[b][0] // 32)].long()
        k = c.codes[0][pg]
        k[:, 0::2] = 0
        k[:, 1::2] = (k[:, 1::2] & 0x7F).clamp(0x38, 0x70) | sign
        c.codes[0][pg] = k
    c.scales[:, 0] = torch.where(c.scales[:, 0].isnan(), c.scales[:, 0], 2.0 ** 40)
    q = torch.full((len(lens), 300, 2, D), 2.0 ** power).to(KIND[kind][0])
    for b, (_, n) in enumerate(lens):
        q[b, n:] = float("nan")
    assert math.log2(D) + power + 40 + math.log2(scale or D ** -0.5) > 129  # of a key of ones
    return c, q


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind,power,scale", FACTORS)
def test_factors_past_32_bits(D, kind, power, scale):
    """Scores of 0, although what they are multiplied with is infinite in 32 bits, beside
    others of -infinity."""
    c, q = past_32_bits(D, [(300, 300), (200, 40)], (0x80, 0x80), kind, power, scale)
    got, status = attend(c, q, softmax_scale=scale)
    assert status == 0
    check(got, *reference(c, q, scale))
