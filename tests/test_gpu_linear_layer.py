"""The dense 4-bit linear, the balance loss and the gradients where a layer uses
them: a layer with a shared expert, one router training step of a layer with
frozen experts, and the bounded-wait path of the tcgen05 linear kernel."""
import time

import numpy as np
import pytest
import torch

import synth
from oracle import linear as O
from oracle import moe as M
from oracle import router as R
from tests.gpu_util import Built, check_tol, load_moe, require_gpu
from tests.test_gpu_linear import cuda, make, oracle_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    return load_moe()


def shared_expert(fmt, group, d, I, T_max, seed=0):
    from expert_offload_serving_b200.layer import SharedExpert
    gu, _ = make(fmt, group, 2 * I, d, 1, zeros=fmt == "int4", seed=seed)
    dn, _ = make(fmt, group, d, I, 1, zeros=fmt == "int4", seed=seed + 1)
    if fmt == "nvfp4":
        gu["tensor_scale"] = dn["tensor_scale"] = 2e-5
    c, e = cuda(gu), cuda(dn)
    s = SharedExpert((c["codes"], c["scales"], c["zeros"]), (e["codes"], e["scales"], e["zeros"]), fmt=fmt, group=group,
                     tensor_scales=(gu["tensor_scale"], dn["tensor_scale"]), T_max=T_max)
    return s, oracle_weights(gu), oracle_weights(dn)


@pytest.mark.parametrize("fmt,group", [("int4", 64), ("mxfp4", 32), ("nvfp4", 16)])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_layer_with_a_shared_expert(moe, fmt, group, T):
    """out = routed experts + shared expert (+ host partial), in one forward()."""
    cfg = synth.LayerConfig("shared", E=8, k=2, d=512, I=256, fmt="bf16")
    b = Built(cfg, T, seed=3)
    ref = b.oracle()["out"]
    sh, wgu, wd = shared_expert(fmt, group, 512, 192, T)
    a = O.linear(b.x.double().numpy(), wgu, swiglu=True)
    a = torch.from_numpy(a).to(torch.bfloat16).double().numpy()        # the activations between the products
    ref = ref + O.linear(a, wd)
    from expert_offload_serving_b200.layer import MoeLayer
    layer = MoeLayer(8, 512, 256, "bf16", 2, T, device_pool=b.layer.pool, shared=sh)
    layer.slot.copy_(b.layer.slot)
    out = layer.forward(b.logits.cuda(), b.x.cuda())
    check_tol(out.cpu().numpy(), ref)
    hp = torch.randn((T, 512), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = layer.forward(b.logits.cuda(), b.x.cuda(), host_partial=hp, stream=side)
    side.synchronize()
    check_tol(out.cpu().numpy(), ref + hp.double().cpu().numpy())
    moe.moe_check_status(layer.status)
    moe.moe_check_status(sh.status)


def test_shared_expert_refusals(moe):
    from expert_offload_serving_b200.layer import MoeLayer, SharedExpert
    sh, _, _ = shared_expert("int4", 64, 512, 192, 4)
    with pytest.raises(ValueError):
        sh.add(torch.zeros((5, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((5, 512), device="cuda"))
    with pytest.raises(ValueError):
        sh.add(torch.zeros((2, 512), dtype=torch.float16, device="cuda"), torch.zeros((2, 512), device="cuda"))
    with pytest.raises(ValueError):
        SharedExpert(sh.down, sh.gate_up)
    with pytest.raises(ValueError):
        SharedExpert(sh.gate_up, sh.down, fmt="bf16")
    with pytest.raises(ValueError):
        MoeLayer(8, 256, 256, "bf16", 2, 4, device_pool=torch.empty((8, moe.moe_expert_blob_bytes(
            moe.shape(8, 256, 256, "bf16"))), dtype=torch.uint8, device="cuda"), shared=sh)


@pytest.mark.parametrize("ragged", [False, True])
def test_router_training_step_with_frozen_experts(moe, ragged):
    """forward -> balance -> router_grad: the gradient of <dout, out> + dloss . loss
    with respect to the logits, by the oracle (experts in float64) and against
    differences of the layer itself."""
    cfg = synth.LayerConfig("router", E=8, k=2, d=512, I=256, fmt="bf16")
    T = 24
    b = Built(cfg, T, seed=4, experts=range(8))
    logits, x = b.logits.cuda(), b.x.cuda()
    out = b.layer.forward(logits, x).clone()
    off = torch.tensor([0, 9, 9, T], dtype=torch.int32, device="cuda") if ragged else None
    mask = (torch.arange(T, device="cuda") % 5 != 3) if ragged else None
    bal = b.layer.balance(logits, seq_offsets=off, mask=mask)
    dloss = torch.tensor([0.05, 0.01], device="cuda")
    dout = torch.randn((T, 512), device="cuda") * 0.1
    if mask is not None:
        dout[~mask] = 0
    got = b.layer.router_grad(logits, dout, bal, dloss, seq_offsets=off, mask=mask)
    moe.moe_check_status(b.layer.status)

    idx, gate = M.route_topk(b.logits.numpy(), 2)
    y = M.per_pair_outputs(b.x.double().numpy(), b.logits.numpy(), 2, b.weights)
    dg = np.einsum("td,tjd->tj", dout.double().cpu().numpy(), np.asarray(y).reshape(T, 2, 512))
    o = None if off is None else off.tolist()
    m = None if mask is None else mask.cpu().numpy()
    _, counts, _, coef = R.balance(b.logits.numpy(), idx, o, m)
    assert np.array_equal(bal["counts"].cpu().numpy(), counts)
    ref = R.router_backward(b.logits.numpy(), idx, gate, dg, counts, coef, dloss.tolist(), o, m)
    check_tol(got.cpu().numpy(), ref, 1e-4, 1e-5)

    # differences: the routing must not change, so move within the gaps of the top-2
    v = torch.sign(got)
    srt = torch.sort(logits, dim=1, descending=True).values
    h = min(2.0 ** -4, float((srt[:, :2] - srt[:, 1:3]).min()) / 4)

    def value(l):
        r = b.layer.forward(l, x)
        q = b.layer.balance(l, seq_offsets=off, mask=mask)
        return float((r.double() * dout.double()).sum() + (q["loss"].double() * dloss.double()).sum())
    change = (value(logits + h * v) - value(logits - h * v)) / (2 * h)
    want = float((got.double() * v).sum())
    assert torch.equal(b.layer.forward(logits, x), out)
    # the values are sums of ~1e4 fp32 products of 1e-2: 1e-6 of rounding, over 2h >= 1e-4
    assert abs(change - want) <= 2e-2 * abs(want) + 1e-2 * h


def test_router_grad_parts_and_refusals(moe):
    cfg = synth.LayerConfig("router", E=8, k=2, d=512, I=256, fmt="bf16")
    b = Built(cfg, 6, seed=5)
    logits = b.logits.cuda()
    b.layer.forward(logits, b.x.cuda())
    bal = b.layer.balance(logits)
    dout, dloss = torch.randn((6, 512), device="cuda"), torch.ones(2, device="cuda")
    both = b.layer.router_grad(logits, dout, bal, dloss)
    apart = b.layer.router_grad(logits, dout) + b.layer.router_grad(logits, balance=bal, dloss=dloss)
    assert torch.allclose(both, apart, rtol=1e-5, atol=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = b.layer.router_grad(logits, dout, b.layer.balance(logits, stream=side), dloss, stream=side)
    side.synchronize()
    assert torch.equal(both, again)
    with pytest.raises(ValueError):
        b.layer.router_grad(logits, dout, bal)
    with pytest.raises(ValueError):
        b.layer.router_grad(logits, dout[:, :256])
    nv = Built(synth.LayerConfig("nv", E=8, k=2, d=512, I=256, fmt="nvfp4", act="nvfp4"), 6, seed=6, act="nvfp4")
    nv.run()
    with pytest.raises(RuntimeError):
        nv.layer.router_grad(nv.logits.cuda(), dout)
    assert torch.isfinite(nv.layer.router_grad(nv.logits.cuda(), balance=nv.layer.balance(nv.logits.cuda()),
                                               dloss=dloss)).all()


@pytest.mark.parametrize("T", [8, 24, 300])
def test_wait_expiry_of_the_linear_is_reported(moe, monkeypatch, T):
    """With the testing aids on, CTA 0's workers wait on a barrier nothing arrives
    on: the call reports MOE_ERR_TIMEOUT, and the next one is right again."""
    monkeypatch.setenv("MOE_LINEAR", "tc")
    w, x = make("int4", 128, 256, 2048, T, zeros=True, seed=13)
    d, xs = cuda(w), x.cuda()
    out, st = torch.empty((T, 256), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(fmt="int4", group=128, zeros=d["zeros"], dev_status=st)
    prev = moe.moe_set_wait_limit_ns(5_000_000)
    moe.moe_set_test_stall(True)
    try:
        t0 = time.perf_counter()
        moe.moe_linear_w4(xs, d["codes"], d["scales"], out, **args)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_check_status(st)
        assert e.value.status == moe.MOE_ERR_TIMEOUT and time.perf_counter() - t0 < 30
    finally:
        moe.moe_set_test_stall(False)
        moe.moe_set_wait_limit_ns(prev)
    for _ in range(2):
        moe.moe_linear_w4(xs, d["codes"], d["scales"], out, **args)
        moe.moe_check_status(st)
        check_tol(out.cpu().numpy(), O.linear(x.double().numpy(), oracle_weights(w)), 1e-4, 1e-5)


@pytest.mark.parametrize("path", ["warp", "tc"])
@pytest.mark.parametrize("fmt,group", [("int4", 32), ("int4", 128), ("mxfp4", 32), ("nvfp4", 16)])
def test_both_kernels_at_every_token_count(moe, monkeypatch, path, fmt, group):
    """MOE_LINEAR forces a kernel where the rule would take the other."""
    from tests.test_gpu_linear import DT, call, check
    monkeypatch.setenv("MOE_LINEAR", path)
    for T in (1, 3, 16, 17, 31, 64, 65, 129, 257):
        for x in ("bf16", "f16"):
            w, xs = make(fmt, group, 200, 1056, T, x=x, zeros=fmt == "int4", seed=14)
            out = torch.empty((T, 200), dtype=DT["f32"], device="cuda")
            call(moe, cuda(w), xs.cuda(), out)
            check(out, w, xs, "f32")


def test_results_on_a_stream_take_no_memory_that_another_still_uses(moe):
    """balance() and router_grad() with a stream of their own: their tensors come
    from that stream, not from a block that the current one has yet to write."""
    T, E = 4096, 256
    from expert_offload_serving_b200.layer import MoeLayer
    layer = MoeLayer(E, 512, 256, "bf16", 4, T, device_pool=torch.zeros(
        (1, moe.moe_expert_blob_bytes(moe.shape(E, 512, 256, "bf16"))), dtype=torch.uint8, device="cuda"))
    logits = torch.randn((T, E), device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    layer.route(logits)
    dloss = torch.ones(2, device="cuda")
    want = layer.router_grad(logits, balance=layer.balance(logits), dloss=dloss).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bal = layer.balance(logits, stream=side)
    torch.cuda.synchronize()
    junk = [torch.empty((T, E), device="cuda") for _ in range(4)]
    torch.cuda._sleep(200_000_000)                     # ~0.1 s: the fills are pending while the gradient is formed
    for j in junk:
        j.fill_(float("nan"))
    del junk, j
    got = layer.router_grad(logits, balance=bal, dloss=dloss, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("q", [0.0, 0.5])
def test_split_step_adds_the_shared_expert(moe, q):
    """A cached layer's split step: routed experts (filled, or computed by the host)
    + shared expert."""
    from expert_offload_serving_b200.layer import MoeLayer, pack_pool
    cfg = synth.LayerConfig("shared_split", E=16, k=4, d=512, I=256, fmt="mxfp4", bias_std=0.5, n_slots=12)
    w = synth.make_experts(cfg, range(16), 8, device="cpu")
    sh, wgu, wd = shared_expert("int4", 128, 512, 256, 3, seed=9)
    layer = MoeLayer(16, 512, 256, "mxfp4", 4, 3, host_pool=pack_pool(16, 512, 256, "mxfp4", w, range(16)), n_slots=12,
                     shared=sh)
    for t in range(2):
        logits, x = synth.make_routing(cfg, 3, 20 + t)
        layer.split_step(t, logits.cuda(), x.cuda(), q=q, threads=2)
        ref = M.moe_layer(x.double().numpy(), logits.numpy(), 4, lambda e: M.dequant_expert("mxfp4", w, e))["out"]
        a = torch.from_numpy(O.linear(x.double().numpy(), wgu, swiglu=True)).to(torch.bfloat16).double().numpy()
        out = layer.out[:3].cpu().numpy()
        check_tol(out, ref + O.linear(a, wd))
        # the routed part, 1e-3 of the sum: what is left of it after fp32 rounding (1e-7 of the sum) is good to 1e-3
        alone = sh.add(x.cuda(), torch.empty((3, 512), device="cuda"), accumulate=False)
        check_tol(out.astype(np.float64) - alone.double().cpu().numpy(), ref)
        moe.moe_check_status(layer.status)


def test_a_timeout_of_the_shared_expert_reaches_the_layer(moe, monkeypatch):
    monkeypatch.setenv("MOE_LINEAR", "tc")
    cfg = synth.LayerConfig("shared", E=8, k=2, d=512, I=256, fmt="bf16")
    b = Built(cfg, 4, seed=3)
    sh, _, _ = shared_expert("int4", 128, 512, 256, 4)
    from expert_offload_serving_b200.layer import MoeLayer
    layer = MoeLayer(8, 512, 256, "bf16", 2, 4, device_pool=b.layer.pool, shared=sh)
    layer.slot.copy_(b.layer.slot)
    prev = moe.moe_set_wait_limit_ns(5_000_000)
    moe.moe_set_test_stall(True)
    try:
        sh.add(b.x.cuda(), torch.zeros((4, 512), device="cuda"), dev_status=layer.status)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_check_status(layer.status)
        assert e.value.status == moe.MOE_ERR_TIMEOUT
    finally:
        moe.moe_set_test_stall(False)
        moe.moe_set_wait_limit_ns(prev)
    layer.forward(b.logits.cuda(), b.x.cuda())
    moe.moe_check_status(layer.status)


def test_captured_step_with_shared_expert_and_router_gradient(moe):
    """forward, balance and router_grad in one graph while an eager pass of the same
    layer lives: replays of new inputs agree with eager passes."""
    cfg = synth.LayerConfig("graph", E=8, k=2, d=512, I=256, fmt="bf16")
    T = 20
    b = Built(cfg, T, seed=11, experts=range(8))
    sh, _, _ = shared_expert("mxfp4", 32, 512, 192, T, seed=3)
    from expert_offload_serving_b200.layer import MoeLayer
    layer = MoeLayer(8, 512, 256, "bf16", 2, T, device_pool=b.layer.pool, shared=sh)
    layer.slot.copy_(b.layer.slot)
    logits, x = b.logits.cuda(), b.x.cuda()
    dout, dloss = torch.randn((T, 512), device="cuda"), torch.tensor([0.3, 0.2], device="cuda")

    def step():
        out = layer.forward(logits, x)
        bal = layer.balance(logits)
        return out, bal["loss"], layer.router_grad(logits, dout, bal, dloss)
    eager = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for seed in (1, 2):
        l2, x2 = synth.make_routing(cfg, T, 40 + seed)
        logits.copy_(l2)
        x.copy_(x2)
        want = [t.clone() for t in step()]
        for t in captured:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(want, captured):
            assert torch.equal(a, c)
    del eager


def test_split_step_runs_the_shared_expert_beside_the_host_share(moe, monkeypatch):
    """The shared expert needs only x, so its products are on the stream before the CPU
    share is waited for.  The host's kernel stands in here for a slow one: it waits
    (10 s at most) until the shared expert has been enqueued."""
    import threading

    from expert_offload_serving_b200 import layer as L
    cfg = synth.LayerConfig("shared_split", E=16, k=4, d=512, I=256, fmt="mxfp4", bias_std=0.5, n_slots=12)
    w = synth.make_experts(cfg, range(16), 8, device="cpu")
    sh, _, _ = shared_expert("int4", 128, 512, 256, 3, seed=9)
    layer = L.MoeLayer(16, 512, 256, "mxfp4", 4, 3, host_pool=L.pack_pool(16, 512, 256, "mxfp4", w, range(16)), n_slots=12,
                       shared=sh)
    logits, x = synth.make_routing(cfg, 3, 20)
    enqueued, seen = threading.Event(), []
    add, host = sh.add, L.moe_host_expert_ffn

    def add_and_tell(*a, **kw):
        r = add(*a, **kw)
        enqueued.set()
        return r

    def slow_host(*a, **kw):
        seen.append(enqueued.wait(10))
        return host(*a, **kw)
    monkeypatch.setattr(sh, "add", add_and_tell)
    monkeypatch.setattr(L, "moe_host_expert_ffn", slow_host)
    assert layer.split_step(0, logits.cuda(), x.cuda(), q=0.0, threads=2)["host"]
    assert seen == [True]


@pytest.mark.parametrize("T", [3, 300])
def test_fused_fp4_layer_with_a_shared_expert(moe, T):
    """act="nvfp4" adds its experts into the output itself: with the shared expert (and a
    host partial) it is the plain layer's output plus their sum, to fp32 rounding of
    adds whose order may differ."""
    cfg = synth.LayerConfig("nv", E=8, k=2, d=512, I=256, fmt="nvfp4", act="nvfp4")
    b = Built(cfg, T, seed=6, act="nvfp4")
    sh, wgu, wd = shared_expert("nvfp4", 16, 512, 192, T, seed=4)
    from expert_offload_serving_b200.layer import MoeLayer
    layer = MoeLayer(8, 512, 256, "nvfp4", 2, T, device_pool=b.layer.pool, act="nvfp4", shared=sh)
    layer.slot.copy_(b.layer.slot)
    logits, x, hp = b.logits.cuda(), b.x.cuda(), torch.randn((T, 512), device="cuda")
    plain = b.layer.forward(logits, x).double().cpu().numpy()
    a = torch.from_numpy(O.linear(b.x.double().numpy(), wgu, swiglu=True)).to(torch.bfloat16).double().numpy()
    ref = plain + O.linear(a, wd)
    check_tol(layer.forward(logits, x).cpu().numpy(), ref)
    check_tol(layer.forward(logits, x, host_partial=hp).cpu().numpy(), ref + hp.double().cpu().numpy())
    moe.moe_check_status(layer.status)
