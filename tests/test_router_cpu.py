"""The balance loss and the router's and combine's gradients without a GPU: the
oracle's gradients against central differences, worked cases, and every
refusal, made before the first CUDA call."""
import numpy as np
import pytest
import torch

from oracle import moe as M
from oracle import router as R


@pytest.fixture(scope="module")
def moe():
    from expert_offload_serving_b200 import build
    build.build()
    import expert_offload_serving_b200 as m
    m.lib()
    return m


def differences(f, x, h=1e-5):
    """Central differences of the scalar f at x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, E, k = 7, 9, 3
    l = rng.standard_normal((T, E))
    idx, _ = M.route_topk(l.astype(np.float32), k)
    off, mask = [1, 4, 4, 6], np.array([1, 1, 0, 1, 1, 1, 1])
    dl, dg = [0.7, 0.3], rng.standard_normal((T, k))
    loss, counts, _, coef = R.balance(l, idx, off, mask)

    def gates(v):
        s = np.take_along_axis(v, idx.astype(np.int64), 1)
        z = np.exp(s - s.max(1, keepdims=True))
        return z / z.sum(1, keepdims=True)

    live = np.zeros(T)
    for ts in R.tokens_of(T, off, mask):
        live[ts] = 1

    def value(v):
        a = R.balance(v, idx, off, mask)[0]
        return dl[0] * a[0] + dl[1] * a[1] + (live[:, None] * dg * gates(v)).sum()
    got = R.router_backward(l, idx, gates(l), dg, counts, coef, dl, off, mask)
    # central differences at h = 1e-5 are off by h^2 f''' / 6 ~ 1e-10 and by rounding ~ 1e-16 / 1e-5
    assert np.abs(got - differences(value, l)).max() < 1e-8
    assert (got[live == 0] == 0).all()


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(1)
    T, k, d, E = 3, 2, 4, 5
    idx = np.array([[0, 4], [2, 0], [3, 1]])
    slot = np.array([0, 1, -1, 2, 3])
    gate, y, dout = rng.random((T, k)), rng.standard_normal((T * k, d)), rng.standard_normal((T, d))
    _, _, inv = M.permute(idx, E)

    def out(g, v):
        return sum((g[t, j] * v[inv[t * k + j]] * dout[t]).sum() for t in range(T) for j in range(k)
                   if slot[idx[t, j]] >= 0)
    dgate, dy = R.combine_backward(y, idx, gate, inv, slot, dout, np.zeros_like(y))
    assert np.abs(dgate - differences(lambda g: out(g, y), gate)).max() < 1e-8
    assert np.abs(dy - differences(lambda v: out(gate, v), y)).max() < 1e-8


def test_uniform_routing_has_loss_one():
    E, k, T = 6, 2, 12
    idx = np.array([[t % E, (t + 3) % E] for t in range(T)])
    loss, counts, prob, coef = R.balance(np.zeros((T, E)), idx)
    assert abs(loss[0] - 1) < 1e-12 and abs(loss[1] - np.log(E) ** 2) < 1e-12
    assert (counts == 4).all() and np.allclose(prob, 1 / E)


def test_empty_sequences_masked_tokens_and_dead_rows():
    l = np.full((4, 3), -np.inf)
    l[1] = [0.0, -np.inf, 0.0]
    l[2] = np.nan
    idx = np.array([[0], [2], [1], [1]])
    loss, counts, prob, coef = R.balance(l, idx, [0, 0, 2, 4], [1, 1, 0, 0])
    assert counts.tolist() == [[0, 0, 0], [1, 0, 1], [0, 0, 0]]
    assert np.allclose(prob, [[0, 0, 0], [0.25, 0, 0.25], [0, 0, 0]])
    assert np.allclose(loss, [3 / 2 * 0.5, np.log(2) ** 2 / 2]) and coef.tolist() == [0, 3 / 4, 0, 0.5]
    assert R.balance(l[:0], idx[:0])[0].tolist() == [0, 0]


@pytest.fixture()
def p():
    raw = np.zeros(1 << 16, dtype=np.uint8)
    p.keep = raw
    return raw.ctypes.data + (-raw.ctypes.data) % 256


p.keep = None


def _balance(moe, p, T=4, E=8, k=2, S=1, ws=1 << 20, logits=0, idx=0, seq=None, mask=None, loss=0, counts=0, prob=0,
             coef=0, work=0):
    at = lambda v: None if v is None else p + v
    return moe.lib().moe_balance_loss(at(logits), T, E, at(idx), k, at(seq), S, at(mask), at(loss), at(counts), at(prob),
                                      at(coef), at(work), ws, None, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=33), dict(T=1 << 24), dict(S=0),
    dict(S=2), dict(S=(1 << 20) + 1, seq=0), dict(S=2, seq=2), dict(logits=None), dict(idx=None), dict(loss=None),
    dict(counts=None), dict(prob=None), dict(coef=None), dict(work=None), dict(work=8), dict(logits=2), dict(coef=1)])
def test_balance_refusals(moe, p, bad):
    assert _balance(moe, p, **bad) == moe.MOE_ERR_INVALID_ARG


def test_balance_workspace(moe, p):
    need = moe.moe_balance_loss_workspace_bytes(4, 8, 1)
    assert need > 0 and _balance(moe, p, ws=need - 1) == moe.MOE_ERR_CAPACITY
    for bad in ((-1, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0), ((1 << 24) + 1, 8, 1)):
        assert moe.moe_balance_loss_workspace_bytes(*bad) == 0
    sizes = [moe.moe_balance_loss_workspace_bytes(T, 256, 4) for T in (1, 100, 5000, 60000, 1 << 20)]
    assert max(sizes) < 64 << 20


def _router(moe, p, T=4, E=8, k=2, S=1, logits=0, idx=0, gate=0, dgate=0, seq=None, mask=None, counts=0, coef=0,
            dloss=0, dlogits=0):
    at = lambda v: None if v is None else p + v
    return moe.lib().moe_router_backward(at(logits), T, E, at(idx), at(gate), at(dgate), k, at(seq), S, at(mask),
                                         at(counts), at(coef), at(dloss), at(dlogits), None, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=1025), dict(k=9), dict(S=3), dict(dlogits=None), dict(logits=None), dict(counts=None),
    dict(coef=None), dict(gate=None), dict(idx=None), dict(dlogits=2), dict(dgate=1), dict(dloss=2)])
def test_router_backward_refusals(moe, p, bad):
    assert _router(moe, p, **bad) == moe.MOE_ERR_INVALID_ARG
    assert _router(moe, p, T=0) == moe.MOE_OK


def _combine(moe, p, T=4, k=2, d=8, E=8, y=0, idx=0, gate=0, inv=0, slot=0, dout=0, dgate=0, dy=0):
    at = lambda v: None if v is None else p + v
    return moe.lib().moe_combine_backward(at(y), at(idx), at(gate), at(inv), at(slot), at(dout), T, k, d, E, at(dgate),
                                          at(dy), None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(k=0), dict(k=33), dict(d=6), dict(d=0), dict(E=0), dict(E=1025), dict(T=1 << 24), dict(y=None),
    dict(idx=None), dict(gate=None), dict(inv=None), dict(dout=None), dict(dgate=None), dict(y=4), dict(dout=8),
    dict(dy=4), dict(inv=2), dict(slot=1)])
def test_combine_backward_refusals(moe, p, bad):
    assert _combine(moe, p, **bad) == moe.MOE_ERR_INVALID_ARG
    assert _combine(moe, p, T=0) == moe.MOE_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would launch on host pointers")
def test_valid_arguments_reach_the_device(moe, p):
    for r in (_balance(moe, p), _balance(moe, p, T=0, logits=None, idx=None), _balance(moe, p, S=3, seq=4, mask=1),
              _router(moe, p), _router(moe, p, dloss=None, logits=None, counts=None, coef=None),
              _router(moe, p, dgate=None, gate=None, idx=None), _combine(moe, p), _combine(moe, p, dy=None, gate=None),
              _combine(moe, p, slot=None)):
        assert r == moe.MOE_ERR_CUDA
