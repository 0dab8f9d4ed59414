"""The decay gate at the ends of its range."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def inputs(T, H, d, dtype, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    return n(T, H, d).to(dtype), n(T, H, d).to(dtype), n(T, H, d).to(dtype), 0.3 * n(H), n(1, H, d)


@pytest.mark.parametrize("d", [16, 33])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("write", ["one", "complement"])
def test_nan_scale_reaches_its_own_head(kda, write, dtype, d):
    """Without validate mode a NaN in A_log shows in that head's results, and in no other's."""
    x, z, do, A, s0 = inputs(70, 3, d, DT[dtype], 2)
    bad = A.clone()
    bad[1] = float("nan")
    res = []
    for a in (A, bad):
        o, fs, st = kda.kda_scan_fwd(x, z, a, initial_state=s0, write=write, want_states=True)
        gr = kda.kda_scan_bwd(x, z, do, a, initial_state=s0, states=st, write=write)
        o1, s1 = kda.kda_scan_step(x[:1], z[:1], s0, a, state_out=torch.empty_like(s0), write=write)
        res.append([("out", o, 1), ("final_state", fs, 1), ("d_decay", gr["d_decay"], 1), ("dA_log", gr["dA_log"], 0),
                    ("d_initial_state", gr["d_initial_state"], 1), ("step", o1, 1), ("step's state", s1, 1)])
    for (name, p, dim), (_, q, _) in zip(*res):
        others = torch.tensor([0, 2], device=DEV)
        assert torch.equal(p.index_select(dim, others), q.index_select(dim, others)), name
        assert q.select(dim, 1).isnan().all(), name


@pytest.mark.parametrize("d", [16, 33])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("write", ["one", "complement"])
def test_infinite_logits_have_no_gradient(kda, write, dtype, d):
    """Exactly none, however large the gradient of the outputs is."""
    x, z, do, A, s0 = inputs(70, 2, d, DT[dtype], 1)
    low, high = torch.finfo(DT[dtype]).min, torch.finfo(DT[dtype]).max
    z[5:9], z[30], z[31], z[50:52] = -float("inf"), float("inf"), high, low
    gr = kda.kda_scan_bwd(x, z, (1e30 * do.float()).to(DT[dtype]), A, initial_state=s0, write=write)
    at = [5, 6, 7, 8, 30, 31, 50, 51]
    assert torch.equal(gr["d_decay"][at], torch.zeros_like(gr["d_decay"][at]))
    rest = [t for t in range(70) if t not in at]
    assert (gr["d_decay"][rest] != 0).all() and gr["dA_log"].isfinite().all()
