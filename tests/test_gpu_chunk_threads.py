"""Two threads that run the CUDA-core prefill and the backward of the delta
rule with other head sizes, that is with other amounts of shared memory:
neither call is refused."""
import ctypes
import threading

import pytest
import torch

from test_gpu_scan_threads import compiled_loops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_two_head_sizes_from_two_threads(kda, tmp_path):
    lib, P = kda.load(), ctypes.c_void_p
    loop = compiled_loops(tmp_path).hammer_chunk
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    sets, results, start = [], {}, threading.Barrier(2)
    T, H = 64, 1
    for dk, dv, chunk in ((128, 128, 64), (16, 16, 16)):
        q, k, v = n(T, H, dk), torch.nn.functional.normalize(n(T, H, dk), dim=-1), n(T, H, dv)
        ins = (q, k, v, -torch.rand(T, H, dk, generator=gen, device=DEV), torch.rand(T, H, generator=gen, device=DEV), n(T, H, dv))
        o, _ = kda.kda_chunk_fwd(*ins[:5], chunk=chunk, kernel="simt")
        gr = kda.kda_chunk_bwd(*ins, chunk=chunk, want_d_initial_state=False)
        want = (o, *(gr[name] for name in ("dq", "dk", "dv", "dlog_alpha", "dbeta")))
        desc = kda.chunk_desc(q, v, chunk=chunk, out_dtype=o.dtype, gate_dtype=0, kernel="simt")
        ws = torch.empty(kda.kda_chunk_bwd_workspace_size(desc), dtype=torch.uint8, device=DEV)
        sets.append((desc, ins, [torch.zeros_like(t) for t in want], want, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(i):
        desc, ins, outs, _, ws, stream = sets[i]
        start.wait()
        results[i] = loop(ctypes.cast(lib.kda_chunk_fwd, P), ctypes.cast(lib.kda_chunk_bwd, P), ctypes.byref(desc),
                          *(P(t.data_ptr()) for t in (*ins, *outs)), P(ws.data_ptr()), ctypes.c_size_t(ws.numel()),
                          P(stream.cuda_stream), 2000)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert results == {0: 0, 1: 0}
    for _, _, outs, want, _, _ in sets:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
