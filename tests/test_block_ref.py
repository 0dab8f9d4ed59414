"""The fp64 definitions behind the recurrence's and the norms' GPU tests, pinned
to closed forms and to central differences (CPU)."""
import numpy as np
import pytest

import _block_ref as ref


def rng(seed=0):
    return np.random.default_rng(seed)


def test_scan_closed_forms():
    r = rng()
    x = r.standard_normal((6, 2, 3))
    s0 = r.standard_normal((1, 2, 3))
    # alpha = 1 with w = 1 is a running sum; alpha = 0 forgets everything
    o = ref.scan(x, np.zeros_like(x), s0=s0, cu=[0, 6])["out"][0]
    np.testing.assert_allclose(o, s0 + np.cumsum(x, 0), rtol=1e-13)
    o = ref.scan(x, np.full_like(x, -np.inf), s0=s0, cu=[0, 6])["out"][0]
    np.testing.assert_array_equal(o, x)
    # a constant decay: geometric sum
    g = np.full_like(x, np.log(0.5))
    o = ref.scan(np.ones_like(x), g, cu=[0, 6])["out"][0]
    np.testing.assert_allclose(o[:, 0, 0], 2 - 2.0 ** -np.arange(6), rtol=1e-13)
    # complement: a running mean keeps a constant input fixed
    o = ref.scan(np.full_like(x, 3.0), g, s0=np.full((1, 2, 3), 3.0), cu=[0, 6], write="complement")["out"][0]
    np.testing.assert_allclose(o, 3.0, rtol=1e-13)


def test_gate_closed_forms():
    g, s = ref.gate(np.array([[[0.0], [np.log(3.0)]]]), np.array([0.0, 0.0]), -4.0)
    np.testing.assert_allclose(g[0, :, 0], [-2.0, -3.0], rtol=1e-13)
    np.testing.assert_allclose(s[0, :, 0], [-1.0, -0.75], rtol=1e-13)
    g, _ = ref.gate(np.array([[[1.0], [1.0]]]), np.array([0.0, np.log(2.0)]), -1.0)
    np.testing.assert_allclose(g[0, :, 0], [-1 / (1 + np.exp(-1)), -1 / (1 + np.exp(-2))], rtol=1e-13)


@pytest.mark.parametrize("write", ["one", "complement"])
@pytest.mark.parametrize("logits", [False, True])
def test_scan_gradients_are_differences(write, logits):
    r = rng(1)
    cu = [0, 4, 4, 9]
    x, dec = r.standard_normal((9, 2, 2)), r.standard_normal((9, 2, 2))
    A = r.standard_normal(2) * 0.3 if logits else None
    dec = dec if logits else -np.abs(dec)
    s0, dO, dS = r.standard_normal((3, 2, 2)), r.standard_normal((9, 2, 2)), r.standard_normal((3, 2, 2))

    def loss(x, dec, A, s0):
        o = ref.scan(x, dec, A, s0=s0, cu=cu, write=write)
        return np.sum(o["out"][0] * dO) + np.sum(o["final_state"][0] * dS)

    got = ref.scan(x, dec, A, s0=s0, cu=cu, write=write, d_out=dO, dST=dS)
    args = dict(x=x, dec=dec, A=A, s0=s0)
    for name, gname in (("x", "dx"), ("dec", "d_decay"), ("A", "dA_log"), ("s0", "d_initial_state")):
        if args[name] is None:
            continue
        v = r.standard_normal(args[name].shape)
        e = 1e-5
        plus, minus = ({**args, name: args[name] + sgn * e * v} for sgn in (1, -1))
        diff = (loss(**plus) - loss(**minus)) / (2 * e)
        assert abs(diff - np.sum(got[gname][0] * v)) <= 1e-7 * (1 + abs(diff)), gname


def test_norm_closed_forms():
    y = np.array([[3.0, 4.0]])
    o = ref.block_norm(y, e1=0.0, normed=False)["out"][0]
    np.testing.assert_allclose(o, y / np.sqrt(12.5), rtol=1e-13)
    o = ref.block_norm(y, gate=np.array([[0.0, np.log(3.0)]]), post=False, scale=np.array([2.0, 4.0]),
                       residual=np.array([[1.0, -1.0]]), normed=False)["out"][0]
    np.testing.assert_allclose(o, [[4.0, 11.0]], rtol=1e-13)
    n = ref.block_norm(y, post=False, w2=np.array([1.0, 2.0]), e2=12.5)["normed"][0]
    np.testing.assert_allclose(n, [[0.6, 1.6]], rtol=1e-13)


@pytest.mark.parametrize("post,gated,res", [(True, True, True), (True, False, False), (False, True, True)])
def test_norm_gradients_are_differences(post, gated, res):
    r = rng(2)
    R, W = 3, 5
    a = dict(y=r.standard_normal((R, W)), residual=r.standard_normal((R, W)) if res else None,
             gate=r.standard_normal((R, W)) if gated else None, w1=r.standard_normal(W) if post else None,
             scale=r.standard_normal(W), w2=r.standard_normal(W))
    do, dn = r.standard_normal((R, W)), r.standard_normal((R, W))

    def loss(**kw):
        o = ref.block_norm(post=post, e1=0.1, e2=0.2, **kw)
        return np.sum(o["out"][0] * do) + np.sum(o["normed"][0] * dn)

    got = ref.block_norm(post=post, e1=0.1, e2=0.2, d_out=do, d_normed=dn, **a)
    names = dict(y="d_y", residual="d_residual", gate="d_gate", w1="d_post_weight", scale="d_scale",
                 w2="d_pre_weight")
    for name, gname in names.items():
        if a[name] is None:
            continue
        v = r.standard_normal(a[name].shape)
        e = 1e-5
        diff = (loss(**{**a, name: a[name] + e * v}) - loss(**{**a, name: a[name] - e * v})) / (2 * e)
        assert abs(diff - np.sum(got[gname][0] * v)) <= 1e-7 * (1 + abs(diff)), gname
