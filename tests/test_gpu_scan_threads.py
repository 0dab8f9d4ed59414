"""Two threads that launch the same kernels with different amounts of shared
memory: neither call is refused."""
import ctypes
import os
import subprocess
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HERE = os.path.dirname(os.path.abspath(__file__))


def compiled_loops(folder):
    so = str(folder / "hammer.so")
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-I", os.path.join(os.path.dirname(HERE), "include"),
                    os.path.join(HERE, "_hammer.c"), "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("d", [64, 33])
def test_two_layouts_of_one_kernel_from_two_threads(kda, tmp_path, d):
    """bf16 logits: 300 tokens run on 8 warps, 5000 on a cluster of CTAs of 16."""
    lib, hammer = kda.load(), compiled_loops(tmp_path).hammer
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    P, A, results, sets = ctypes.c_void_p, torch.zeros(1, device=DEV), {}, []
    for T in (300, 5000):
        x, z, do = (torch.randn(T, 1, d, generator=gen, device=DEV).bfloat16() for _ in range(3))
        o, _, st = kda.kda_scan_fwd(x, z, A, want_states=True)
        g = kda.kda_scan_bwd(x, z, do, A, states=st)
        bufs = [torch.zeros_like(t) for t in (o, st, g["dx"], g["d_decay"], g["dA_log"])]
        sets.append((kda.KdaScanDesc(1, T, 1, d, 0, 1, 1, 0, 0), (x, z, A, do), bufs, (o, st, g["dx"], g["d_decay"], g["dA_log"]),
                     torch.empty(1 << 22, dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(i):
        desc, ins, bufs, _, ws, stream = sets[i]
        start.wait()
        results[i] = hammer(ctypes.cast(lib.kda_scan_fwd, P), ctypes.cast(lib.kda_scan_bwd, P), ctypes.byref(desc),
                            *(P(t.data_ptr()) for t in (*ins, *bufs)), P(ws.data_ptr()), ctypes.c_size_t(ws.numel()),
                            P(stream.cuda_stream), 3000)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert results == {0: 0, 1: 0}
    for _, _, bufs, want, _, _ in sets:
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))
