"""Layouts of the scan over the GPU that other tests' shapes do not reach: the
elementwise form in blocks of 32 and of 8 channels, on one CTA and on
clusters, and blocks of 64 channels with both write rules."""
import numpy as np
import pytest
import torch

import test_gpu_scan as scan
from _block_ref import np64

pytestmark = pytest.mark.gpu
LAYOUTS = {
    # rows off 16 bytes, blocks of 32 channels: more of them than SMs take; on clusters of 4 and of 2 CTAs; partly filled
    "elementwise_many": ([60, 1, 17, 0, 33] * 4, 3, 5, 65),
    "elementwise_cluster4": ([900, 700, 300, 1000, 600], 0, 5, 65),
    "elementwise_cluster2": ([300] * 9, 7, 5, 65),
    "elementwise_short_rounds": ([129] * 45, 0, 1, 33),
    # blocks of 8 channels on clusters of 8 CTAs of 16 warps
    "elementwise_long": ([9000], 0, 1, 33),
    # blocks of 64 channels
    "wide": ([300, 129, 128, 15], 5, 48, 64),
}


def with_lost_powers(a, want):
    """d_decay's bound with what an alpha below 2^-126, which is 0 in fp32 without subnormals, may take away: less
    than 2^-126 |D_t| (|h_{t-1}| + |x_t|), and D_t = dx_t, as w = 1 - alpha is 1 there."""
    rows = scan.live_rows(a)
    prev = np.concatenate([np64(a["initial_state"])[:1], want["out"][0][:-1]])
    for n, first in enumerate(a["cu"][:-1]):
        if first < a["cu"][n + 1]:
            prev[first] = np64(a["initial_state"])[n]
    v, e = want["d_decay"]
    lost = 2.0 ** -126 * np.abs(want["dx"][0]) * (np.abs(prev) + np.abs(np64(a["x"])))
    lost[rows:] = 0.0
    return v, e + lost


@pytest.mark.parametrize("write", ["one", "complement"])
@pytest.mark.parametrize("dtype,gate", scan.KINDS)
@pytest.mark.parametrize("shape", list(LAYOUTS))
def test_layout(kda, shape, dtype, gate, write):
    a = scan.make(LAYOUTS[shape], dtype, gate, seed=50)
    rows, mark = scan.live_rows(a), 7.0
    want = scan.definition(a, write, bwd=True)
    out = torch.full_like(a["x"], mark)
    o, fs, states = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], scan.G_MIN, a["initial_state"], a["cu_seqlens"], out,
                                     write=write, want_states=True)
    scan.check(o, want["out"], a["x"].dtype, rows, "out")
    scan.check(fs, want["final_state"], torch.float32, None, "final_state")
    for st in (states, None):
        gr = dict(dx=torch.full_like(a["x"], mark), d_decay=torch.full_like(a["decay"], mark),
                  dA_log=None if a["A_log"] is None else torch.empty_like(a["A_log"]), d_initial_state=torch.empty_like(fs))
        kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], scan.G_MIN, a["initial_state"], a["dST"],
                         a["cu_seqlens"], st, write=write, grads=gr)
        scan.check(gr["dx"], want["dx"], a["x"].dtype, rows, "dx")
        scan.check(gr["d_decay"], with_lost_powers(a, want), a["decay"].dtype, rows, "d_decay")
        scan.check(gr["d_initial_state"], want["d_initial_state"], torch.float32, None, "d_initial_state")
        if a["A_log"] is not None:
            scan.check(gr["dA_log"], want["dA_log"], torch.float32, None, "dA_log")
        for t in (gr["dx"], gr["d_decay"], out):
            assert (t[rows:] == mark).all()


def test_side_stream_keeps_a_dropped_input(kda):
    """An input dropped right after a call on another stream is not reused before that call is done with it."""
    a = scan.make(([5000, 3000], 0, 8, 64), "bf16", "fp32", seed=12)
    o0, fs0 = kda.kda_scan_fwd(a["x"], a["decay"], None, scan.G_MIN, a["initial_state"], a["cu_seqlens"])
    side = torch.cuda.Stream()
    wait = torch.randn(4096, 4096, device="cuda:0")
    for _ in range(3):
        x = a["x"].clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):  # keeps the side stream busy for a while
                wait.mm(wait)
        o, fs = kda.kda_scan_fwd(x, a["decay"], None, scan.G_MIN, a["initial_state"], a["cu_seqlens"], stream=side)
        del x
        over = [torch.full_like(a["x"], float("nan")) for _ in range(4)]  # on the current stream, into freed memory if any
        side.synchronize()
        assert torch.equal(o, o0) and torch.equal(fs, fs0)
        del over
