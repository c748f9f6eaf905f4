"""What include/kda_mla_cache.h says of the rounding to 4 bits, over all largest magnitudes of a block. No GPU needed;
tests/test_gpu_mla_cache.py holds the kernels to the same rounding bit by bit."""
import os
import re

import torch

import gated_delta_rule_chunk_amd as kda
from tests import mla_cache_ref as ref

HEADER = os.path.join(os.path.dirname(kda.HEADER_PATH), "kda_mla_cache.h")


def test_no_rounding_is_off_by_more_than_stated():
    text = re.sub(r"\n \* *", " ", open(HEADER).read())
    m = re.search(r"no rounding is off by more than 2\^e, or in blocks of more than 7 \* 2\^125 by (\d) \* 2\^e", text)
    assert m, "the header states how far a rounding is off"
    top = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    top = top[top.isfinite() & (top >= 2.0 ** -100)]
    g = torch.Generator().manual_seed(2)
    x = top[:, None].double() * (2 * torch.rand((len(top), 32), generator=g, dtype=torch.float64) - 1)
    x[:, 7] = top.double()
    x = x.float()
    codes, scales = ref.encode(x)
    two = ref.power(scales.long() - 127)
    off = (ref.values(codes, scales) - x.double()).abs().amax(1, keepdim=True) / two
    past = (top.double() > 7 * 2.0 ** 125)[:, None]
    assert bool((off[~past] <= 1).all()) and bool((off[past] <= int(m.group(1))).all())
    assert past.any() and bool((off[past] > 1).all())            # (the statement is no weaker than it has to be)
