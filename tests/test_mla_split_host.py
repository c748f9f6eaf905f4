"""bf16 queries as the sum of two 8-bit floats (e4m3), as the scores over 4-bit latents take them: what
include/kda_mla_cache.h says of their precision, over all bf16 numbers and all blocks. No GPU needed;
tests/test_gpu_mla_cache_more.py holds the kernels to the same numbers."""
import os
import re

import torch

import gated_delta_rule_chunk_amd as kda

HEADER = os.path.join(os.path.dirname(kda.HEADER_PATH), "kda_mla_cache.h")


def stated():
    """The numbers of the header: channels from `exact` of their block's largest on are exact, smaller ones lose at
    most `loss` of it; where it is below `tiny`, any loses at most `least`."""
    text = re.sub(r"\s+\*?\s*", " ", open(HEADER).read())
    m = re.search(r"except for channels below 2\^-(\d+) of the largest of their 32, which are off by at most "
                  r"2\^-(\d+) of that; where the largest is below 2\^-(\d+), any of them by at most 2\^-(\d+)", text)
    assert m, "the header states the precision of the queries"
    return tuple(2.0 ** -int(x) for x in m.groups())


def test_the_split_of_all_queries():
    exact, loss, tiny, least = stated()
    q = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    q = q[q.isfinite()].float()                                  # all magnitudes
    for top in range(0, 255):                                    # the exponent of the block's largest
        low = 2.0 ** (top - 127) if top else 2.0 ** -133         # it is this at least, and below 2^(top - 126)
        x = q[q < 2.0 ** (max(top, 1) - 126)].double()
        s = top - 7 if top >= 16 else 9                          # the scale byte
        y = x * 2.0 ** (127 - s)
        hi = y.float().to(torch.float8_e4m3fn).double()
        lo = ((y - hi) * 16).float().to(torch.float8_e4m3fn).double()
        off = ((hi + lo / 16) * 2.0 ** (s - 127) - x).abs()
        # (x is a channel of blocks whose largest is x or more)
        largest = torch.clamp(x, min=low)
        assert bool((off <= torch.where(largest < tiny, least, loss * largest)).all()), top
        if low >= tiny:
            assert not off[x >= exact * low].any(), top
