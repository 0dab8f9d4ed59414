"""The tensor-core attention kernel's bounded waits: none runs out, and the word that says so is read."""
import ctypes

import pytest
import torch

from test_gpu_paged import Case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def word(kda):
    flags = ctypes.c_uint(0)
    assert kda.load().kda_device_watchdog(ctypes.byref(flags), 1) == 0
    return flags.value


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (128, 8), (64, 256)])
def test_no_wait_runs_out(kda, d, page):
    # more than 32 rows to a head of the cache: whole items, parts of items, rows without keys, values that are not finite
    word(kda)
    for new, lens in (([300, 1, 40], [700, 2000, 41]), ([1500], [1500]), ([70] * 40, [100] * 40), ([200, 100], [0, 50])):
        c = Case(new, lens, 8, 2, d, page, BF)
        c.check(kda)
        if lens[0] > 200:
            p, s = c.at(0, lens[0] - 2)
            c.vc[p, 0, s, 3] = float("inf")
            c.check(kda)
            c.check(kda, causal=False)
    assert word(kda) == 0
