"""router_grad(dout) on layers whose experts come and go: the gradient belongs to
the slots of the step whose output it differentiates, not to the table as later
fills have left it, and a step that left chosen experts to the host has none.

A cached layer runs the kernels of a resident one on the same blobs, so its
gradient has the same bits."""
import numpy as np
import pytest
import torch

import synth
from oracle import moe as M
from tests.gpu_util import load_moe, require_gpu

pytestmark = pytest.mark.gpu

E, D, I, K, T = 16, 512, 256, 2, 5


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    return load_moe()


class Cached:
    """Layers over one cache of few slots, a resident twin of each, and a routing."""

    def __init__(self, n_layers=1, n_slots=T * K, fmt="mxfp4"):
        from expert_offload_serving_b200.layer import ExpertCache, MoeLayer, pack_pool
        from expert_offload_serving_b200 import shape
        cfg = synth.LayerConfig("offloaded", E=E, k=K, d=D, I=I, fmt=fmt)
        pools = [pack_pool(E, D, I, fmt, synth.make_experts(cfg, range(E), 30 + l, device="cpu"), range(E))
                 for l in range(n_layers)]
        self.cache = ExpertCache(shape(E, D, I, fmt), n_slots, pools)
        self.layers = [MoeLayer(E, D, I, fmt, K, T, cache=self.cache, layer_id=l) for l in range(n_layers)]
        self.twins = [MoeLayer(E, D, I, fmt, K, T, device_pool=p.cuda()) for p in pools]
        g = torch.Generator().manual_seed(77)
        self.in_ = []
        for l in range(n_layers):
            logits, x = synth.make_routing(cfg, T, 60 + l)
            self.in_.append((logits.cuda(), x.cuda(), (0.1 * torch.randn((T, D), generator=g)).cuda()))
        self.step = 0

    def chosen(self, l):
        return sorted(set(M.route_topk(self.in_[l][0].cpu().numpy(), K)[0].ravel().tolist()))

    def prepare(self, l, experts):
        self.layers[l].prepare(self.step, list(experts))
        self.step += 1

    def twin_grad(self, l, slots=None):
        """The resident twin's gradient, with only `slots` in its table (None: all)."""
        twin, (logits, x, dout) = self.twins[l], self.in_[l]
        table = torch.arange(E, dtype=torch.int32)
        if slots is not None:
            table[[e for e in range(E) if e not in slots]] = -1
        twin.slot.copy_(table)
        twin.forward(logits, x)
        return twin.router_grad(logits, dout)


@pytest.mark.parametrize("steps", ["forward", "stepwise"])
def test_gradient_after_later_layers_evicted_the_experts(moe, steps):
    """Forward through three layers over a cache that holds one step, then the
    gradients from the last layer to the first."""
    c = Cached(n_layers=3)
    for l, layer in enumerate(c.layers):
        logits, x, _ = c.in_[l]
        c.prepare(l, c.chosen(l))
        if steps == "forward":
            layer.forward(logits, x)
        else:
            layer.route(logits)
            layer.permute(T)
            layer.ffn(x)
            layer.combine(T)
    assert all(c.layers[0].slot.cpu()[e] < 0 for e in c.chosen(0)[:2])       # evicted by now
    for l in (2, 1, 0):
        assert torch.equal(c.layers[l].router_grad(c.in_[l][0], c.in_[l][2]), c.twin_grad(l))
    for layer in c.layers:
        moe.moe_check_status(layer.status)


def test_an_expert_filled_after_the_step_is_not_part_of_it(moe):
    """A step that runs with some chosen experts absent (and no host share) adds
    nothing for them; fills that follow do not change its gradient."""
    c = Cached()
    layer, (logits, x, dout) = c.layers[0], c.in_[0]
    u = c.chosen(0)
    c.prepare(0, u[:-2])
    layer.y_perm.fill_(float("nan"))                    # rows that the step does not write
    layer.forward(logits, x)
    c.prepare(0, u)
    torch.cuda.synchronize()
    assert (layer.slot.cpu()[u] >= 0).all()
    got = layer.router_grad(logits, dout)
    assert torch.isfinite(got).all() and torch.equal(got, c.twin_grad(0, u[:-2]))


@pytest.mark.parametrize("q", [0.0, 1.0])
def test_split_step(moe, q):
    """Every miss on the host: no gradient of the gates (the losses' part stays);
    every miss filled: the resident layer's."""
    c = Cached()
    layer, (logits, x, dout) = c.layers[0], c.in_[0]
    r = layer.split_step(0, logits, x, q=q, threads=2)
    assert bool(r["host"]) == (q == 0.0)
    if q == 0.0:
        with pytest.raises(RuntimeError, match="host"):
            layer.router_grad(logits, dout)
    else:
        assert torch.equal(layer.router_grad(logits, dout), c.twin_grad(0))
    dloss = torch.ones(2, device="cuda")
    assert torch.isfinite(layer.router_grad(logits, balance=layer.balance(logits), dloss=dloss)).all()
    # the same experts filled afterwards do not make up for the host's outputs
    c.step = 1
    c.prepare(0, c.chosen(0))
    if q == 0.0:
        with pytest.raises(RuntimeError, match="host"):
            layer.router_grad(logits, dout)


@pytest.mark.parametrize("cached", [True, False])
@pytest.mark.parametrize("steps", ["forward", "stepwise"])
def test_callers_host_partial(moe, cached, steps):
    """A host_partial beside chosen experts that have no slot holds their outputs:
    refused.  With every chosen expert in a slot it is some other term."""
    c = Cached()
    (logits, x, dout), u = c.in_[0], c.chosen(0)
    layer = c.layers[0] if cached else c.twins[0]
    hp = torch.randn((T, D), device="cuda")

    def have(experts):
        if cached:
            c.prepare(0, experts)
        else:
            layer.slot.fill_(-1)
            layer.slot[torch.tensor(experts, device="cuda")] = torch.tensor(experts, dtype=torch.int32, device="cuda")

    def run():
        if steps == "forward":
            layer.forward(logits, x, host_partial=hp)
        else:
            layer.route(logits)
            layer.permute(T)
            layer.ffn(x)
            layer.combine(T, host_partial=hp)
    have(u[:-1])
    run()
    have(u)
    with pytest.raises(RuntimeError, match="host"):
        layer.router_grad(logits, dout)
    run()
    got = layer.router_grad(logits, dout)
    layer.forward(logits, x)
    assert torch.equal(got, layer.router_grad(logits, dout))
    if cached:
        assert torch.equal(got, c.twin_grad(0))


def test_captured_step(moe):
    """In a graph the refusal is recorded in the status word; a replay after another
    step's fills is that of the slots it ran with."""
    c = Cached()
    (logits, x, dout), u, layer = c.in_[0], c.chosen(0), c.layers[0]
    hp = torch.zeros((T, D), device="cuda")
    c.prepare(0, u)
    layer.forward(logits, x, host_partial=hp)
    want = layer.router_grad(logits, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(logits, x, host_partial=hp)
        got = layer.router_grad(logits, dout)
    g.replay()
    moe.moe_check_status(layer.status)
    assert torch.equal(got, want)
    layer.slot[u[0]] = -1                               # what a fill of another layer does
    g.replay()
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check_status(layer.status)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED


def test_logits_and_balance_of_another_shape_are_refused(moe):
    """Narrower logits would leave results in the wrong columns; counts and coef of
    other sequences would be read as this batch's."""
    c = Cached()
    layer, (logits, x, dout) = c.twins[0], c.in_[0]
    layer.forward(logits, x)
    dloss = torch.ones(2, device="cuda")
    off = torch.tensor([0, 2, T], dtype=torch.int32, device="cuda")
    bal, bal2 = layer.balance(logits), layer.balance(logits, seq_offsets=off)
    for bad in (logits[:, :E // 2].contiguous(), torch.cat([logits, logits], 1), logits.double(), logits.cpu()):
        with pytest.raises(ValueError, match="logits: expected a contiguous"):
            layer.balance(bad)
        with pytest.raises(ValueError, match="logits: expected a contiguous"):
            layer.router_grad(bad, dout)
        with pytest.raises(ValueError, match="logits: expected a contiguous"):
            layer.router_grad(bad, balance=bal, dloss=dloss)
    with pytest.raises(ValueError, match="counts"):
        layer.router_grad(logits, balance=bal2, dloss=dloss)
    with pytest.raises(ValueError, match="counts"):
        layer.router_grad(logits, balance=bal, dloss=dloss, seq_offsets=off)
    with pytest.raises(ValueError, match="coef"):
        layer.router_grad(logits, balance=dict(bal, coef=bal2["coef"]), dloss=dloss)
    layer.router_grad(logits, balance=bal2, dloss=dloss, seq_offsets=off)


@pytest.mark.parametrize("inside", [True, False])
def test_layer_built_in_inference_mode(moe, inside):
    """Its steps run within that mode and outside of it."""
    with torch.inference_mode():
        c = Cached()
    layer, (logits, x, dout) = c.layers[0], c.in_[0]
    hp = torch.zeros((T, D), device="cuda")
    with torch.inference_mode(inside):
        c.prepare(0, c.chosen(0))
        want = layer.forward(logits, x).clone()
        got = layer.router_grad(logits, dout)
        assert torch.equal(layer.forward(logits, x, host_partial=hp), want)
        assert torch.equal(layer.router_grad(logits, dout), got)
