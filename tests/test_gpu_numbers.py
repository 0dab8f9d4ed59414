"""Numbers of a call that are held in tensors: each call has their value at that time."""
import pytest
import torch

from test_gpu_paged import Case, DEV, freqs, rand

pytestmark = pytest.mark.gpu


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


@pytest.mark.parametrize("where", ["cpu", DEV])
def test_numbers_that_change_in_place(kda, where):
    c = Case([3, 1], [40, 9], 4, 2, 64, 16, torch.float32)
    k, v = rand(c.gen, 4, 2, 64), rand(c.gen, 4, 2, 64)
    f, pos = freqs(64), torch.arange(4, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)

    def rope(**how):
        return kda.kda_qk_rope_fwd(c.q, k, pos, f, **how)

    def turned_back(**how):
        return tuple(kda.kda_qk_rope_bwd(c.q, k, c.q, k, pos, f, **how).values())

    def append(**how):
        return (kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, c.cu, q=c.q, inv_freq=f, norm=True, **how),)

    def attend(**how):
        return c.attend(kda, **how)

    def norm(**how):
        return kda.kda_block_norm_fwd(c.q.view(16, 64), post_weight=w, **how)

    for call, name in ((rope, "rot_scale"), (rope, "eps"), (turned_back, "rot_scale"), (turned_back, "eps"),
                       (append, "rot_scale"), (append, "eps"), (attend, "scale"), (norm, "post_eps")):
        x = torch.tensor(0.5, device=where)
        first = call(**{name: x})
        x.fill_(2.0)
        second = call(**{name: x})
        assert same(first, call(**{name: 0.5})), name
        assert same(second, call(**{name: 2.0})) and not same(first, second), name
