"""The serving operators at the edges of their numbers and arguments: infinities and the largest
values in a cache, row scales over the whole range of fp32, non-finite frequencies."""
import math

import numpy as np
import pytest
import torch

from gpu_common import fa_module
from oracle import serving as ref
from test_gpu_serving import (TYPES, _clean_status, check_decode, check_rotary, gather64, i32, make_cache,  # noqa: F401
                              np64, rand, random_cache, raw)

pytestmark = pytest.mark.gpu

# Lengths whose tables map few tokens (a CTA takes a head alone) and many (the keys are split).
NARROW, WIDE = [1, 17, 40, 300], [1, 17, 40, 3000]
# Split keys again, several steps to a warp.
MANY = [3000 - 7 * b for b in range(90)]


def rows64(cache, table, lens):
    """The cached K and V of each sequence, (H, n, D) float64."""
    return [[gather64(cache, table, b, n, w) for b, n in enumerate(lens)] for w in (0, 1)]


def put(cache, table, b, key, head, dim, value):
    cache.v[table[b, key // cache.page_size].item(), head, key % cache.page_size, dim] = value


# ---------------------------------------------------------------- workspaces

def test_decode_refuses_a_workspace_that_is_not_contiguous():
    # A broadcast or strided tensor's size in bytes is more than the memory behind it.
    fa = fa_module()
    cache, table, _, _ = random_cache("s8", [20, 20], 16, 2, 64)
    q, n = rand((2, 4, 1, 64)), i32(20, 20)
    need = fa.decode_workspace_bytes(2, 4, 2, 64)
    one = torch.empty(16, dtype=torch.uint8, device="cuda")
    strided = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (one[:1].expand(need), one[None].expand(need // 16 + 1, 16), strided[::2], strided.view(2, need).t()):
        with pytest.raises(ValueError, match="workspace"):
            fa.decode_attention(q, cache, table, n, workspace=ws)
    fa.decode_attention(q, cache, table, n, workspace=strided)
    torch.cuda.synchronize()


