"""moe_balance_loss, moe_router_backward and moe_combine_backward against the
float64 oracle, at the sizes and masks where they can go wrong.

Tolerances.  A probability is an fp32 exponential of a difference (each within a
few steps of 2^-24) over a sum of E of them in log2(32) + E/32 adds: within
(E/32 + 16) 2^-23 of its value, plus |logit - max| 2^-24 for the rounded
difference (logits here stay below 16 apart: 2^-20 covers it).  Averages over
tokens add at most n/8/592 + 8 fp32 steps more before the 64-bit sum.  Below:
P = (E/32 + 48) 2^-23 for probabilities, means, lse^2 and the losses; a gradient
is a product of such a probability with a difference of like terms, bounded by P
times the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from oracle import moe as M
from oracle import router as R
from tests.gpu_util import load_moe, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    return load_moe()


def routing(T, E, k, seed=0):
    rng = np.random.default_rng(seed * 7919 + T * 31 + E)
    l = (rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    idx, gate = M.route_topk(l, k)
    return rng, l, idx, gate.astype(np.float32)


def dev(a, dt=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)


def run_balance(moe, l, idx, off=None, mask=None, status=None, ws=None, **kw):
    T, E = l.shape
    S = 1 if off is None else len(off) - 1
    o = dict(loss=torch.full((2,), -7.0, device="cuda"), counts=torch.full((S, E), -7, dtype=torch.int32, device="cuda"),
             prob=torch.full((S, E), -7.0, device="cuda"), coef=torch.full((S + 1,), -7.0, device="cuda"))
    if ws is None:
        ws = torch.full((moe.moe_balance_loss_workspace_bytes(T, E, S),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(dev(l), dev(idx), o["loss"], o["counts"], o["prob"], o["coef"], ws,
                         seq_offsets=None if off is None else dev(np.asarray(off, dtype=np.int32)),
                         mask=None if mask is None else dev(np.asarray(mask, dtype=bool)), dev_status=status, **kw)
    return o


def check_balance(o, l, idx, off=None, mask=None):
    E = l.shape[1]
    P = (E / 32 + 48) * 2.0 ** -23
    loss, counts, prob, coef = R.balance(l, idx, off, mask)
    assert np.array_equal(o["counts"].cpu().numpy(), counts)
    assert (np.abs(o["prob"].double().cpu().numpy() - prob) <= P * prob + 2.0 ** -126).all()
    assert (np.abs(o["coef"].double().cpu().numpy() - coef) <= 2.0 ** -23 * coef).all()
    assert (np.abs(o["loss"].double().cpu().numpy() - loss) <= P * np.abs(loss)).all(), (o["loss"], loss)


SIZES = [(1, 1, 1), (1, 8, 2), (7, 33, 4), (64, 128, 8), (65, 64, 3), (200, 256, 6), (33, 512, 8), (19, 1000, 32),
         (5, 1024, 1), (3000, 60, 5)]


@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance_one_sequence(moe, T, E, k):
    _, l, idx, _ = routing(T, E, k)
    check_balance(run_balance(moe, l, idx), l, idx)


@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance_sequences_and_mask(moe, T, E, k):
    """Ragged sequences, empty ones, tokens before the first and behind the last,
    masked tokens whose logits are NaN, a sequence with nothing left."""
    rng, l, idx, _ = routing(T, E, k, 1)
    cuts = np.sort(rng.integers(0, T + 1, 9))
    off = np.concatenate([cuts[:3], cuts[2:3], cuts[2:]])
    mask = rng.random(T) < 0.8
    mask[off[4]:off[5]] = False
    l[~mask] = np.nan
    check_balance(run_balance(moe, l, idx, off, mask), l, idx, off, mask)


def test_balance_many_short_sequences(moe):
    T = 5000
    _, l, idx, _ = routing(T, 40, 2, 2)
    off = np.arange(T + 1)
    check_balance(run_balance(moe, l, idx, off), l, idx, off)
    check_balance(run_balance(moe, l, idx, off[::-1][:1].tolist() * 2000 + [T]), l, idx, [T] * 2001)


def test_balance_nothing_left(moe):
    _, l, idx, _ = routing(6, 16, 2, 3)
    check_balance(run_balance(moe, l, idx, None, np.zeros(6, dtype=bool)), l, idx, None, np.zeros(6, dtype=bool))
    o = run_balance(moe, l[:0], idx[:0])
    assert o["loss"].tolist() == [0, 0] and (o["counts"] == 0).all() and (o["prob"] == 0).all()
    assert o["coef"].tolist() == [0, 1]


def test_balance_infinite_and_lowest_logits(moe):
    """-inf switches an expert off; the type's lowest value is a number; a row of
    -inf has no probabilities."""
    _, l, idx, _ = routing(40, 70, 4, 4)
    l[:, 5] = -np.inf
    l[3] = -np.inf
    l[4, 10:] = -np.inf
    l[6, :60] = np.finfo(np.float32).min
    l[7] = -80.0
    for T in (40, 4):
        check_balance(run_balance(moe, l[:T], idx[:T]), l[:T], idx[:T])


def test_bad_ids_and_offsets_are_recorded(moe):
    _, l, idx, _ = routing(50, 20, 3, 5)
    bad = idx.copy()
    bad[7, 1], bad[9, 0] = 20, -3
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_balance(run_balance(moe, l, bad, status=st), l, bad)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check_status(st)
    assert e.value.status == moe.MOE_ERR_DEVICE
    for off in ([0, 30, 20, 50], [-1, 10], [0, 51], [40, 10]):
        run_balance(moe, l, idx, off, status=st)
        with pytest.raises(moe.MoeError):
            moe.moe_check_status(st)
        dl = torch.zeros((50, 20), device="cuda")
        S = len(off) - 1
        moe.moe_router_backward(dev(l), dev(idx), dl, counts=torch.zeros((S, 20), dtype=torch.int32, device="cuda"),
                                coef=torch.zeros(S + 1, device="cuda"), dloss=torch.ones(2, device="cuda"),
                                seq_offsets=dev(np.asarray(off, dtype=np.int32)))
    torch.cuda.synchronize()


def run_router(moe, l, idx, gate=None, dgate=None, counts=None, coef=None, dloss=None, off=None, mask=None, **kw):
    out = torch.full(l.shape, -7.0, device="cuda")
    f = lambda a: None if a is None else dev(a, torch.float32)
    moe.moe_router_backward(dev(l), dev(idx), out, gate=f(gate), dgate=f(dgate),
                            counts=None if counts is None else dev(counts, torch.int32), coef=f(coef), dloss=f(dloss),
                            seq_offsets=None if off is None else dev(np.asarray(off, dtype=np.int32)),
                            mask=None if mask is None else dev(np.asarray(mask, dtype=np.uint8)), **kw)
    return out


def check_router(out, l, idx, gate, dgate, counts, coef, dloss, off, mask):
    T, E = l.shape
    P = (E / 32 + 48) * 2.0 ** -23
    ref = R.router_backward(l, idx, gate, dgate, counts, coef, dloss, off, mask)
    size = np.zeros((T, E))
    for s, ts in enumerate(R.tokens_of(T, off, mask)):
        if dloss is not None and ts:
            p, lse = R.softmax_rows(l[ts])
            c = np.asarray(counts[s], dtype=np.float64)
            size[ts] += p * (abs(dloss[0]) * coef[s] * (c + (c * p).sum(1, keepdims=True))
                             + 2 * abs(dloss[1]) * coef[-1] * np.abs(lse)[:, None])
        if dgate is not None:
            for t in ts:
                for j, e in enumerate(idx[t]):
                    if 0 <= e < E:
                        size[t, e] += gate[t, j] * (abs(dgate[t, j]) + (gate[t] * np.abs(dgate[t])).sum())
    assert (np.abs(out.double().cpu().numpy() - ref) <= P * size + 2.0 ** -126).all()


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("parts", ["both", "gates", "loss"])
def test_router_backward(moe, T, E, k, parts):
    rng, l, idx, gate = routing(T, E, k, 6)
    for ragged in (False, True):
        off = mask = None
        if ragged:
            off = np.sort(rng.integers(0, T + 1, 6))
            mask = rng.random(T) < 0.8
            l[~mask] = np.nan
            gate[~mask] = np.nan
        _, counts, _, coef = R.balance(l, idx, off, mask)
        a = dict(counts=counts, coef=coef, dloss=np.array([0.6, -0.2], dtype=np.float32)) if parts != "gates" else \
            dict(counts=None, coef=None, dloss=None)
        a.update(dict(gate=gate, dgate=rng.standard_normal((T, k)).astype(np.float32)) if parts != "loss" else
                 dict(gate=None, dgate=None))
        if a["coef"] is not None:
            a["coef"] = a["coef"].astype(np.float32)
        out = run_router(moe, l, idx, off=off, mask=mask, **a)
        check_router(out, l, idx, a["gate"], a["dgate"], a["counts"], a["coef"], a["dloss"], off, mask)


def test_router_backward_infinite_logits_and_bad_ids(moe):
    rng, l, idx, gate = routing(30, 50, 4, 7)
    l[:, 11] = -np.inf
    l[3] = -np.inf
    idx[5, 2] = 50
    idx[6, 0] = -1
    _, counts, _, coef = R.balance(l, idx)
    coef = coef.astype(np.float32)
    dg = rng.standard_normal((30, 4)).astype(np.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run_router(moe, l, idx, gate, dg, counts, coef, np.array([1, 1], dtype=np.float32), dev_status=st)
    check_router(out, l, idx, gate, dg, counts, coef, [1.0, 1.0], None, None)
    with pytest.raises(moe.MoeError):
        moe.moe_check_status(st)


def test_gradient_against_differences_of_the_loss(moe):
    """The forward's own loss, moved along a direction, changes by <dlogits, v>.
    The loss is fp32 (a step is 2^-24 of ~6) and h = 2^-5 leaves h^2/6 f''' of the
    third derivative, each far below 2e-3 of the change's size."""
    rng, l, idx, _ = routing(24, 16, 2, 8)
    off = [0, 10, 24]
    o = run_balance(moe, l, idx, off)
    d = run_router(moe, l, idx, counts=o["counts"].cpu().numpy(), coef=o["coef"].cpu().numpy(),
                   dloss=np.array([1.0, 0.5], dtype=np.float32), off=off)
    v = np.sign(d.cpu().numpy()).astype(np.float32)
    f = lambda a: float((run_balance(moe, a.astype(np.float32), idx, off)["loss"].double().cpu() *
                         torch.tensor([1.0, 0.5])).sum())
    h = 2.0 ** -5
    got = (f(l + h * v) - f(l - h * v)) / (2 * h)
    want = float((d.double().cpu().numpy() * v).sum())
    assert abs(got - want) <= 2e-3 * abs(want)


@pytest.mark.parametrize("T,k,d,E", [(1, 1, 4, 1), (1, 8, 2048, 128), (5, 3, 260, 16), (17, 9, 1028, 40), (64, 8, 512, 128),
                                     (3, 32, 64, 1024), (300, 6, 36, 256), (2, 2, 16384, 8)])
def test_combine_backward(moe, T, k, d, E):
    """dgate is an fp32 sum of d products: (d/1024 + 16) 2^-23 of the sum of their
    magnitudes; dy is one product: half a step."""
    rng, _, idx, gate = routing(T, E, k, 9)
    _, _, inv = M.permute(idx, E)
    y, dout = (rng.standard_normal(s).astype(np.float32) for s in ((T * k, d), (T, d)))
    slot = np.where(rng.random(E) < 0.3, -1, np.arange(E)).astype(np.int32)
    for sl in (slot, None):
        for want_dy in (True, False):
            y2 = y.copy()
            if sl is not None:                              # rows that no term reads may hold anything
                for p_, e in enumerate(idx.ravel()):
                    if sl[e] < 0:
                        y2[inv[p_]] = np.nan
            dg = torch.full((T, k), -7.0, device="cuda")
            dy = torch.full((T * k, d), -7.0, device="cuda") if want_dy else None
            moe.moe_combine_backward(dev(y2), dev(idx), dev(gate), dev(inv), dev(sl), dev(dout), E, dg, dy_perm=dy)
            rg, rdy = R.combine_backward(y2, idx, gate, inv, sl, dout, np.full((T * k, d), -7.0))
            size = R.combine_backward(np.abs(y2), idx, gate, inv, sl, np.abs(dout), np.zeros((T * k, d)))[0]
            assert (np.abs(dg.double().cpu().numpy() - rg) <= (d / 1024 + 16) * 2.0 ** -23 * size).all()
            if want_dy:
                assert (np.abs(dy.double().cpu().numpy() - rdy) <= 2.0 ** -24 * np.abs(rdy)).all()


def test_combine_backward_bad_indices(moe):
    """inv_perm or an id out of range drops the pair, as the combine does."""
    rng, _, idx, gate = routing(6, 8, 2, 10)
    _, _, inv = M.permute(idx, 8)
    y, dout = (rng.standard_normal(s).astype(np.float32) for s in ((12, 16), (6, 16)))
    inv, idx = inv.copy(), idx.copy()
    inv[3], inv[4], idx[0, 1] = 12, -1, 9
    slot = np.arange(8, dtype=np.int32)
    dg = torch.full((6, 2), -7.0, device="cuda")
    dy = torch.full((12, 16), -7.0, device="cuda")
    moe.moe_combine_backward(dev(y), dev(idx), dev(gate), dev(inv), dev(slot), dev(dout), 8, dg, dy_perm=dy)
    rg, rdy = R.combine_backward(y, idx, gate, inv, slot, dout, np.full((12, 16), -7.0))
    assert np.allclose(dg.cpu().numpy(), rg, atol=1e-5) and np.allclose(dy.cpu().numpy(), rdy, atol=1e-6)


def test_same_bits_graphs_and_streams(moe):
    """Two eager calls, a call on another stream and a replayed graph (forward and
    gradient in one) agree bit for bit."""
    _, l, idx, gate = routing(900, 100, 4, 11)
    off = [0, 100, 555, 900]
    L, I, G = dev(l), dev(idx), dev(gate)
    offs = dev(np.asarray(off, dtype=np.int32))
    dgate = torch.randn((900, 4), device="cuda")
    dloss = torch.tensor([0.5, 0.1], device="cuda")

    def step(stream=None):
        o = [torch.empty(2, device="cuda"), torch.empty((3, 100), dtype=torch.int32, device="cuda"),
             torch.empty((3, 100), device="cuda"), torch.empty(4, device="cuda"), torch.empty((900, 100), device="cuda")]
        ws = torch.empty(moe.moe_balance_loss_workspace_bytes(900, 100, 3), dtype=torch.uint8, device="cuda")
        moe.moe_balance_loss(L, I, *o[:4], ws, seq_offsets=offs, stream=stream)
        moe.moe_router_backward(L, I, o[4], gate=G, dgate=dgate, counts=o[1], coef=o[3], dloss=dloss, seq_offsets=offs,
                                stream=stream)
        return o + [ws]
    first, second = step(), step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    third = step(side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fourth = step()
    for _ in range(2):
        for t in fourth[:5]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for other in (second, third, fourth):
            for a, b in zip(first[:5], other[:5]):
                assert torch.equal(a, b)


def test_binding_refusals(moe):
    l, i = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    o = [torch.empty(2, device="cuda"), torch.empty((1, 8), dtype=torch.int32, device="cuda"),
         torch.empty((1, 8), device="cuda"), torch.empty(2, device="cuda")]
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(4, 8, 1), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_balance_loss(l.half(), i, *o, ws)
    with pytest.raises(ValueError):
        moe.moe_balance_loss(l, i, *o, ws, seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))   # S = 2
    with pytest.raises(ValueError):
        moe.moe_balance_loss(l, i, *o, ws, mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, i, *o, ws[:64])
    with pytest.raises(ValueError):
        moe.moe_router_backward(l, i, l[:3])
    with pytest.raises(moe.MoeError):
        moe.moe_router_backward(l, i, l.clone(), dgate=torch.zeros((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_combine_backward(l, i, o[2], i, None, l, 8, o[2])


def test_outputs_overlap_nothing_else_of_the_call(moe):
    l, i = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    o = [torch.empty(2, device="cuda"), torch.empty((1, 8), dtype=torch.int32, device="cuda"),
         torch.empty((1, 8), device="cuda"), torch.empty(2, device="cuda")]
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(4, 8, 1), dtype=torch.uint8, device="cuda")
    for bad in ((l.view(-1)[:2], *o[1:], ws), (o[0], i.view(1, 8), *o[2:], ws), (o[0], o[1], l[3:], o[3], ws),
                (o[0], o[1], o[2], o[0], ws), (*o, l.view(torch.uint8).view(-1)), (o[2].view(-1)[:2], *o[1:], ws)):
        with pytest.raises(ValueError, match="overlaps"):
            moe.moe_balance_loss(l, i, *bad)
    g = torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        moe.moe_router_backward(l, i, l, gate=g, dgate=g)
    big = torch.zeros(40, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        moe.moe_router_backward(l, i, big[:32].view(4, 8), gate=g, dgate=big[30:38].view(4, 2))
    moe.moe_router_backward(l, i, big[:32].view(4, 8), gate=g, dgate=big[32:40].view(4, 2))
    y, inv, dout = torch.zeros((8, 8), device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda"), l
    for dg, dy in ((g, None), (torch.empty_like(g), y), (y[0].view(4, 2), None), (y[0].view(4, 2), torch.empty_like(y))):
        with pytest.raises(ValueError, match="overlaps"):
            moe.moe_combine_backward(y, i, g, inv, None, dout, 8, dg, dy_perm=dy)
    with pytest.raises(ValueError, match="overlaps"):
        moe.moe_combine_backward(y, i, g, inv, None, y[:4], 8, torch.empty_like(g), dy_perm=y)


@pytest.mark.parametrize("T", [40, 300])
def test_z_loss_of_rows_whose_logsumexp_is_near_zero(moe, T):
    """A z-loss drives lse = max + log(sum) to 0, where only absolute errors are left.
    E equal logits near -log E: the sum is E exactly and log is off by a step of its
    value at most.  Logits 0 and -a: the sum 1 + exp(-a) is off by half a step of 1,
    2^-24, and 2^-20 of the exponential; log passes that on.  The z-loss is lse^2 within
    a few 2^-23 and its gradient 2 lse p / T within 2^-20 more (p)."""
    rows = [(np.full(E, -np.log(E) + 1e-4), lambda l: np.spacing(np.float32(np.log(len(l))))) for E in range(3, 40)]
    rows += [(np.array([0.0, -a]), lambda l: 2.0 ** -24 + 2.0 ** -20 * np.exp(l[1])) for a in np.linspace(2.0, 12.0, 21)]
    for row, err in rows:
        l = np.repeat(row.astype(np.float32)[None], T, 0)
        idx = np.zeros((T, 1), dtype=np.int32)
        o = run_balance(moe, l, idx)
        r = l[0].astype(np.float64)
        lse = np.log(np.exp(r).sum())
        off = float(err(r)) + 2.0 ** -22 * abs(lse)
        z = float(o["loss"][1].double().cpu())
        assert abs(np.sqrt(z) - abs(lse)) <= off, (row[:2], np.sqrt(z) - abs(lse), off)
        d = run_router(moe, l, idx, counts=o["counts"].cpu().numpy(), coef=o["coef"].cpu().numpy(),
                       dloss=np.array([0.0, 1.0], dtype=np.float32))
        p = np.exp(r - lse)
        assert (np.abs(d.double().cpu().numpy() - 2 * lse * p / T) <= (2 * off + 2.0 ** -20 * abs(lse)) * p / T).all()


def test_the_status_word_lies_apart_from_the_outputs(moe):
    """dev_status is written by a call, too: it may lie in nothing that the call reads
    or writes."""
    l, i = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    o = [torch.empty(2, device="cuda"), torch.empty((1, 8), dtype=torch.int32, device="cuda"),
         torch.empty((1, 8), device="cuda"), torch.empty(2, device="cuda")]
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(4, 8, 1), dtype=torch.uint8, device="cuda")
    for st in (o[1].view(-1)[3:4], o[2].view(torch.int32).view(-1)[:1], ws[16:20].view(torch.int32), i.view(-1)[7:],
               l.view(torch.int32).view(-1)[:1]):
        with pytest.raises(ValueError, match="dev_status overlaps"):
            moe.moe_balance_loss(l, i, *o, ws, dev_status=st)
    g, dl = torch.zeros((4, 2), device="cuda"), torch.zeros((4, 8), device="cuda")
    for st in (dl.view(torch.int32).view(-1)[31:], g.view(torch.int32).view(-1)[:1]):
        with pytest.raises(ValueError, match="dev_status overlaps"):
            moe.moe_router_backward(l, i, dl, gate=g, dgate=torch.zeros_like(g), dev_status=st)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    c, s = torch.zeros((16, 32), dtype=torch.uint8, device="cuda"), torch.ones((16, 2), dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros((2, 24), device="cuda")
    for st in (wide.view(torch.int32).view(-1)[25:26], x.view(torch.int32).view(-1)[:1], c.view(-1)[:4].view(torch.int32),
               s.view(-1)[:2].view(torch.int32)):
        with pytest.raises(ValueError, match="dev_status overlaps"):
            moe.moe_linear_w4(x, c, s, wide[:, :16], group=32, dev_status=st)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_balance_loss(l, i, *o, ws, dev_status=st)
    moe.moe_router_backward(l, i, dl, gate=g, dgate=torch.zeros_like(g), dev_status=st)
    moe.moe_linear_w4(x, c, s, wide[:, :16], group=32, dev_status=st)
    moe.moe_check_status(st)
    gap = wide.view(torch.int32).view(-1)[16:17]                       # between out's rows
    moe.moe_linear_w4(x, c, s, wide[:, :16], group=32, dev_status=gap)
    moe.moe_check_status(gap)


@pytest.mark.parametrize("E", [20, 512, 516, 1000])
def test_balance_where_one_cta_gives_way_to_two_kernels(moe, E):
    """48, 64 and 128 tokens and one more, one sequence and two, by offsets or none."""
    for T in (48, 49, 64, 65, 128, 129):
        rng, l, idx, _ = routing(T, E, 4, 13)
        mask = rng.random(T) < 0.8
        l[~mask] = np.nan
        for off in (None, [0, T], [3, T - 2], [T // 2, T // 2], [0, 5, T], [0, 0, T]):
            check_balance(run_balance(moe, l, idx, off, mask), l, idx, off, mask)


def test_balance_of_few_tokens_in_many_sequences_is_not_slow(moe):
    """64 tokens in 64 sequences may not take 64 times those in one: they are 3 times
    as slow in two kernels, 40 times where one CTA walks the sequences; 10 is between."""
    _, l, idx, _ = routing(64, 128, 8, 14)
    L, I = dev(l), dev(idx)
    times = []
    for S in (1, 64):
        off = torch.arange(S + 1, dtype=torch.int32, device="cuda") * (64 // S)
        o = [torch.empty(2, device="cuda"), torch.empty((S, 128), dtype=torch.int32, device="cuda"),
             torch.empty((S, 128), device="cuda"), torch.empty(S + 1, device="cuda")]
        ws = torch.empty(moe.moe_balance_loss_workspace_bytes(64, 128, S), dtype=torch.uint8, device="cuda")
        moe.moe_balance_loss(L, I, *o, ws, seq_offsets=off)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(50):
                moe.moe_balance_loss(L, I, *o, ws, seq_offsets=off)
        best = float("inf")
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[1] <= 10 * times[0], times


def test_no_tokens_in_several_sequences(moe):
    l, idx = np.zeros((0, 24), dtype=np.float32), np.zeros((0, 3), dtype=np.int32)
    check_balance(run_balance(moe, l, idx, [0, 0, 0, 0]), l, idx, [0, 0, 0, 0])
    out = torch.empty((0, 24), device="cuda")
    moe.moe_router_backward(dev(l), dev(idx), out, gate=torch.empty((0, 3), device="cuda"),
                            dgate=torch.empty((0, 3), device="cuda"))
