"""What is measured of the dense 4-bit linear and of the router's training operators.

Each operator has a plain form (elementary torch operations in 32 bits) and the
call a user makes of this package; `own` picks between them.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = {"mxfp4": 32, "nvfp4": 16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token through the down projection of a small shared expert (d = 2048, I = 768): a call of latency
        dict(name="w4_int4_T1_2048x768", op="linear", fmt="int4", group=128, zeros=True, T=1, N=2048, K=768,
             x="bf16", y="f32", swiglu=False),
        # one token through the gate and up projections of a large shared expert (d = 4096, I = 2048)
        dict(name="w4_mxfp4_T1_swiglu", op="linear", fmt="mxfp4", group=32, zeros=False, T=1, N=4096, K=4096,
             x="bf16", y="bf16", swiglu=True),
        # a decode batch of 8 through that expert's down projection
        dict(name="w4_nvfp4_T8_4096x2048", op="linear", fmt="nvfp4", group=16, zeros=False, T=8, N=4096, K=2048,
             x="bf16", y="f32", swiglu=False),
        # an output head over a vocabulary of odd size for a decode batch of 13
        dict(name="w4_int4_T13_head", op="linear", fmt="int4", group=64, zeros=False, T=13, N=128001, K=4096,
             x="f16", y="f32", swiglu=False),
        # a decode batch of 64 through a wide dense projection
        dict(name="w4_int4_T64_16384x4096", op="linear", fmt="int4", group=128, zeros=True, T=64, N=16384, K=4096,
             x="bf16", y="bf16", swiglu=False),
        # a prompt of 1000 tokens through the large shared expert's gate and up projections
        dict(name="w4_int4_T1000_swiglu", op="linear", fmt="int4", group=32, zeros=True, T=1000, N=4096, K=4096,
             x="bf16", y="bf16", swiglu=True),
        # the load statistics of one decode batch (E = 128, top 8)
        dict(name="balance_T64_E128", op="balance", T=64, E=128, k=8, S=1, masked=0.0),
        # a training batch of packed ragged sequences with padding (E = 256, top 6)
        dict(name="balance_T50000_E256", op="balance", T=50000, E=256, k=6, S=29, masked=0.1),
        # the router's gradient for a small batch and for that training batch
        dict(name="router_grad_T61_E128", op="router_grad", T=61, E=128, k=8, S=1, masked=0.0),
        dict(name="router_grad_T50000_E256", op="router_grad", T=50000, E=256, k=6, S=29, masked=0.1),
        # the combine's gradient for a small batch, and for a prefill-sized one with 30 % of the experts on the host
        dict(name="combine_grad_T16_d2048", op="combine_grad", T=16, E=128, k=8, d=2048, host=0.0),
        dict(name="combine_grad_T4096_d4096", op="combine_grad", T=4096, E=256, k=6, d=4096, host=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "balance", "router_grad", "combine_grad"])
    if op == "linear":
        fmt = rng.choice(["int4", "int4", "mxfp4", "nvfp4"])
        group = rng.choice([32, 64, 128]) if fmt == "int4" else GROUP[fmt]
        T = _log(rng, 1, 1000)
        K = 32 * _log(rng, 4, 512)
        most = min(128001 * 4096 // K, 1000 * 4096 * 4096 // (K * T))
        N = _log(rng, 64, max(65, min(131072, most)))
        swiglu = rng.random() < 0.3
        x = rng.choice(["bf16", "f16"])
        return dict(op=op, fmt=fmt, group=group, zeros=fmt == "int4" and rng.random() < 0.5, T=T,
                    N=N - N % 2 if swiglu else N, K=K, x=x, y=rng.choice(["f32", x]), swiglu=swiglu)
    E = rng.choice([8, 60, 64, 128, 160, 256, 384, 512])
    k = rng.randint(1, 8)
    if op == "combine_grad":
        d = 4 * _log(rng, 64, 2048)
        most = 4096 * 4096 * 6 // (d * k)
        return dict(op=op, T=_log(rng, 1, min(8192, most)), E=E, k=k, d=d, host=rng.choice([0.0, 0.3]))
    T = _log(rng, 1, 50000 * 256 // max(E, 256))
    return dict(op=op, T=T, E=E, k=k, S=_log(rng, 1, max(1, min(T, 64))), masked=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _codes(g, N, K, fmt):
    """Codes of weights drawn from a normal distribution, two to a byte (even element in the low nibble)."""
    out = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    rows = max(1, (1 << 26) // K)
    for n in range(0, N, rows):
        w = torch.randn((min(rows, N - n), K), generator=g, device="cuda")
        if fmt == "int4":
            q = (w * 2.6 + 8).round().clamp(0, 15).to(torch.uint8)
        else:
            mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
            q = torch.bucketize(w.abs() * 2, mids).to(torch.uint8) + 8 * (w < 0).to(torch.uint8)
        out[n:n + rows] = q[:, 0::2] | (q[:, 1::2] << 4)
    return out


def _linear_inputs(c, g):
    N, K, T, fmt = c["N"], c["K"], c["T"], c["fmt"]
    G = -(-K // c["group"])
    spread = torch.randn((N, G), generator=g, device="cuda") * 0.3
    st = dict(codes=_codes(g, N, K, fmt), zeros=None, tensor_scale=1.0)
    if fmt == "int4":
        st["scales"] = (0.008 * spread.exp()).to(DTYPES[c["x"]])
        if c["zeros"]:
            st["zeros"] = torch.randint(6, 11, (N, G), generator=g, device="cuda", dtype=torch.uint8)
    elif fmt == "mxfp4":
        st["scales"] = (127 + torch.floor(spread - 6.0)).to(torch.uint8)
    else:
        st["scales"] = (40 * spread.exp()).to(torch.float8_e4m3fn).view(torch.uint8)
        st["tensor_scale"] = 2.0 ** -12 * 1.3
    st["x"] = torch.randn((T, K), generator=g, device="cuda").to(DTYPES[c["x"]])
    st["out"] = torch.empty((T, N // 2 if c["swiglu"] else N), dtype=DTYPES[c["y"]], device="cuda")
    return st


def _routing(c, g):
    """Logits with a per-expert bias, the top k of each token and their gates."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((E,), generator=g, device="cuda")
    v, idx = torch.topk(logits, k, dim=1)
    return logits, idx.to(torch.int32), torch.softmax(v, dim=1)


def _sequences(c, g):
    """Offsets of S ragged sequences over the T tokens, and the mask of the tokens that count."""
    T, S = c["T"], c["S"]
    if S == 1:
        off = None
    else:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
    mask = None
    if c["masked"]:
        mask = torch.rand((T,), generator=g, device="cuda") >= c["masked"]
    return off, mask


def _members(T, S, off, mask):
    """[S, T] in {0, 1}: the tokens that count for each sequence."""
    t = torch.arange(T, device="cuda")
    if off is None:
        m = torch.ones((1, T), dtype=torch.bool, device="cuda")
    else:
        m = (t >= off[:-1, None]) & (t < off[1:, None])
    return m if mask is None else m & mask


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "linear":
        return dict(case=c, **_linear_inputs(c, g))
    logits, idx, gate = _routing(c, g)
    T, E, k = c["T"], c["E"], c["k"]
    st = dict(case=c, logits=logits, idx=idx, gate=gate)
    if c["op"] == "combine_grad":
        order = torch.sort(idx.reshape(-1), stable=True).indices
        st["inv_perm"] = torch.empty((T * k,), dtype=torch.int32, device="cuda")
        st["inv_perm"][order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        st["slot"] = torch.arange(E, dtype=torch.int32, device="cuda")
        if c["host"]:
            st["slot"][torch.rand((E,), generator=g, device="cuda") < c["host"]] = -1
        st["y_perm"] = torch.randn((T * k, c["d"]), generator=g, device="cuda")
        st["dout"] = torch.randn((T, c["d"]), generator=g, device="cuda")
        st["dgate"] = torch.empty((T, k), device="cuda")
        st["dy_perm"] = torch.zeros((T * k, c["d"]), device="cuda")   # rows of experts on the host stay as they are
        return st
    S = c["S"]
    st["seq_offsets"], st["mask"] = _sequences(c, g)
    if c["op"] == "balance":
        st["loss"] = torch.empty((2,), device="cuda")
        st["counts"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
        st["prob"] = torch.empty((S, E), device="cuda")
        st["coef"] = torch.empty((S + 1,), device="cuda")
        return st
    # what the forward pass left: per-sequence counts and the two gradients' factors
    m = _members(T, S, st["seq_offsets"], st["mask"])
    chosen = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, idx.long(), 1.0)
    st["counts"] = torch.matmul(m.double(), chosen).to(torch.int32)
    n = m.sum(1).double()
    there = (n > 0).sum().clamp(min=1)
    st["coef"] = torch.cat([torch.where(n > 0, E / (k * n.clamp(min=1) ** 2 * there), 0.0),
                            1 / n.sum().clamp(min=1).reshape(1)]).float()
    st["dloss"] = torch.tensor([0.01, 0.001], device="cuda") * (1 + torch.rand((2,), generator=g, device="cuda"))
    st["dgate"] = torch.randn((T, k), generator=g, device="cuda") * 0.1 / T
    st["dlogits"] = torch.empty((T, E), device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def _weights(st):
    """The weights as 32-bit floats [N, K]."""
    c = st["case"]
    q = torch.stack([st["codes"] & 15, st["codes"] >> 4], dim=2).reshape(c["N"], c["K"])
    if c["fmt"] == "int4":
        z = 8.0 if st["zeros"] is None else st["zeros"].float().repeat_interleave(c["group"], 1)[:, :c["K"]]
        w, s = q.float() - z, st["scales"].float()
    else:
        mag = torch.tensor(E2M1, device="cuda")[(q & 7).long()]
        w = torch.where(q >= 8, -mag, mag)
        if c["fmt"] == "mxfp4":
            s = torch.exp2(st["scales"].float() - 127)
        else:
            s = st["scales"].view(torch.float8_e4m3fn).float() * st["tensor_scale"]
    return w * s.repeat_interleave(c["group"], 1)[:, :c["K"]]


def _linear(st):
    c = st["case"]
    y = torch.matmul(st["x"].float(), _weights(st).t())
    if c["swiglu"]:
        h, u = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
        y = h / (1 + torch.exp(-h)) * u
    return y.to(DTYPES[c["y"]])


def _probabilities(logits):
    top = logits.max(1, keepdim=True).values
    z = torch.exp(logits - top)
    total = z.sum(1, keepdim=True)
    return z / total, (top + torch.log(total)).squeeze(1)


def _balance(st):
    c = st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    m = _members(T, S, st["seq_offsets"], st["mask"]).float()
    p, lse = _probabilities(st["logits"])
    chosen = torch.zeros((T, E), device="cuda").scatter_(1, st["idx"].long(), 1.0)
    counts = torch.matmul(m, chosen)
    n = m.sum(1)
    some = n.clamp(min=1)
    prob = torch.matmul(m, p) / some[:, None]
    there = (n > 0).sum().clamp(min=1)
    coef = torch.where(n > 0, E / (k * some * some * there), 0.0)
    total = n.sum().clamp(min=1)
    loss = torch.stack([(coef * some * (counts * prob).sum(1)).sum(),
                        (m.amax(0) * lse * lse).sum() / total])
    return {"loss": loss, "counts": counts.to(torch.int32), "prob": prob,
            "coef": torch.cat([coef, 1 / total.reshape(1)])}


def _router_grad(st):
    c = st["case"]
    m = _members(c["T"], c["S"], st["seq_offsets"], st["mask"]).float()
    p, lse = _probabilities(st["logits"])
    f = torch.matmul(m.t(), st["counts"].float() * st["coef"][:-1, None])
    live = m.amax(0)
    d = p * (st["dloss"][0] * (f - (f * p).sum(1, keepdim=True))
             + (2 * st["dloss"][1] * st["coef"][-1] * live * lse)[:, None])
    dg = st["gate"] * (st["dgate"] - (st["gate"] * st["dgate"]).sum(1, keepdim=True))
    return d.scatter_add(1, st["idx"].long(), dg * live[:, None])


def _combine_grad(st):
    c = st["case"]
    idx, rows = st["idx"].long(), st["inv_perm"].long()
    there = st["slot"][idx.reshape(-1)] >= 0
    y = st["y_perm"][rows].reshape(c["T"], c["k"], c["d"])
    dgate = (y * st["dout"][:, None, :]).sum(2) * there.reshape(c["T"], c["k"])
    dy = torch.zeros((c["T"] * c["k"], c["d"]), device="cuda")
    dy[rows[there]] = (st["gate"][:, :, None] * st["dout"][:, None, :]).reshape(-1, c["d"])[there]
    return {"dgate": dgate, "dy_perm": dy}


def run(st):
    c = st["case"]
    if not own:
        return {"linear": _linear, "balance": _balance, "router_grad": _router_grad,
                "combine_grad": _combine_grad}[c["op"]](st)
    import expert_offload_serving_b200 as moe
    if c["op"] == "linear":
        moe.moe_linear_w4(st["x"], st["codes"], st["scales"], st["out"], fmt=c["fmt"], group=c["group"],
                          zeros=st["zeros"], tensor_scale=st["tensor_scale"], swiglu=c["swiglu"])
        return st["out"]
    if c["op"] == "balance":
        if "workspace" not in st:
            st["workspace"] = torch.empty((moe.moe_balance_loss_workspace_bytes(c["T"], c["E"], c["S"]),),
                                          dtype=torch.uint8, device="cuda")
        moe.moe_balance_loss(st["logits"], st["idx"], st["loss"], st["counts"], st["prob"], st["coef"],
                             st["workspace"], seq_offsets=st["seq_offsets"], mask=st["mask"])
        return {"loss": st["loss"], "counts": st["counts"], "prob": st["prob"], "coef": st["coef"]}
    if c["op"] == "router_grad":
        moe.moe_router_backward(st["logits"], st["idx"], st["dlogits"], gate=st["gate"], dgate=st["dgate"],
                                counts=st["counts"], coef=st["coef"], dloss=st["dloss"],
                                seq_offsets=st["seq_offsets"], mask=st["mask"])
        return st["dlogits"]
    moe.moe_combine_backward(st["y_perm"], st["idx"], st["gate"], st["inv_perm"], st["slot"], st["dout"], c["E"],
                             st["dgate"], dy_perm=st["dy_perm"])
    return {"dgate": st["dgate"], "dy_perm": st["dy_perm"]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, T = case, case["T"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "linear":
        G = -(-c["K"] // c["group"])
        per = (2 if c["fmt"] == "int4" else 1) + (1 if c["zeros"] else 0)
        out = c["N"] // 2 if c["swiglu"] else c["N"]
        return {"bytes": c["N"] * (c["K"] // 2 + G * per) + T * c["K"] * size[c["x"]] + T * out * size[c["y"]],
                "flops": 2 * T * c["N"] * c["K"]}
    E, k = c["E"], c["k"]
    live = 1 - c.get("masked", 0.0)
    if c["op"] == "balance":
        return {"bytes": live * T * (E + k) * 4 + T * (c["masked"] > 0) + c["S"] * (E * 8 + 8), "flops": 6 * T * E}
    if c["op"] == "router_grad":
        return {"bytes": live * T * (E + 3 * k) * 4 + T * E * 4 + T * (c["masked"] > 0) + c["S"] * (E * 4 + 8),
                "flops": 10 * T * E}
    there = 1 - c["host"]
    return {"bytes": there * T * k * c["d"] * 8 + T * c["d"] * 4 + T * k * 16, "flops": 3 * there * T * k * c["d"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_linear(c, st):
    N, K, g = c["N"], c["K"], c["group"]
    y = torch.zeros((c["T"], N), dtype=torch.float64, device="cuda")
    x = st["x"].double()
    rows = max(1, (1 << 27) // K)
    for n in range(0, N, rows):
        b = st["codes"][n:n + rows].to(torch.int32)
        w = torch.empty((b.shape[0], K), dtype=torch.float64, device="cuda")
        s = st["scales"][n:n + rows]
        for odd, code in ((0, b % 16), (1, b // 16)):
            if c["fmt"] == "int4":
                w[:, odd::2] = code.double()
            else:
                e, man = (code % 8) // 2, code % 2
                mag = torch.where(e == 0, man.double() / 2, (1 + man.double() / 2) * torch.pow(2.0, e.double() - 1))
                w[:, odd::2] = mag * (1 - 2 * (code // 8).double())
        if c["fmt"] == "mxfp4":
            s = torch.pow(torch.full((), 2.0, dtype=torch.float64, device="cuda"), s.double() - 127)
        elif c["fmt"] == "nvfp4":
            i = s.to(torch.int32)
            e, man = (i % 128) // 8, (i % 8).double()
            s = torch.where(e == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.pow(2.0, e.double() - 7))
            s = s * (1 - 2 * (i // 128).double()) * st["tensor_scale"]
        for j in range(s.shape[1]):
            part = w[:, j * g:(j + 1) * g]
            if c["fmt"] == "int4":
                part -= 8 if st["zeros"] is None else st["zeros"][n:n + rows, j:j + 1].double()
            part *= s[:, j:j + 1].double()
        y[:, n:n + rows] = x @ w.t()
    if c["swiglu"]:
        y = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:]
    return y


def _spans(c, st):
    off = [0, c["T"]] if st["seq_offsets"] is None else st["seq_offsets"].tolist()
    live = torch.ones((c["T"],), dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
    return [torch.arange(a, b, device="cuda")[live[a:b]] for a, b in zip(off[:-1], off[1:])]


def _exact_balance(c, st):
    E, k = c["E"], c["k"]
    logits, spans = st["logits"].double(), _spans(c, st)
    some = sum(len(t) > 0 for t in spans)
    total = sum(len(t) for t in spans)
    loss, z = torch.zeros((2,), dtype=torch.float64, device="cuda")
    counts, prob, coef = [], [], []
    for t in spans:
        counts.append(torch.bincount(st["idx"][t].reshape(-1).long(), minlength=E))
        prob.append(torch.softmax(logits[t], 1).sum(0) / max(1, len(t)))
        coef.append(E / (k * len(t) ** 2 * some) if len(t) else 0.0)
        loss = loss + coef[-1] * len(t) * (counts[-1] * prob[-1]).sum()
        z = z + torch.logsumexp(logits[t], 1).square().sum() / max(1, total)
    return {"loss": torch.stack([loss, z]), "counts": torch.stack(counts).to(torch.int32), "prob": torch.stack(prob),
            "coef": torch.tensor(coef + [1 / max(1, total)], dtype=torch.float64, device="cuda")}


def _exact_router_grad(c, st):
    d = torch.zeros((c["T"], c["E"]), dtype=torch.float64, device="cuda")
    a, b = st["dloss"].double()
    coef = st["coef"].double()
    for s, t in enumerate(_spans(c, st)):
        p = torch.softmax(st["logits"][t].double(), 1)
        lse = torch.logsumexp(st["logits"][t].double(), 1)
        n = st["counts"][s].double()
        d[t] = a * coef[s] * p * (n - (p @ n)[:, None]) + 2 * b * coef[-1] * lse[:, None] * p
        g, dg = st["gate"][t].double(), st["dgate"][t].double()
        for j in range(c["k"]):
            d[t, st["idx"][t, j].long()] += g[:, j] * (dg[:, j] - (g * dg).sum(1))
    return d


def _exact_combine_grad(c, st):
    k = c["k"]
    dgate = torch.zeros((c["T"], k), dtype=torch.float64, device="cuda")
    dy = torch.zeros((c["T"] * k, c["d"]), dtype=torch.float64, device="cuda")
    dout = st["dout"].double()
    for j in range(k):
        t = torch.nonzero(st["slot"][st["idx"][:, j].long()] >= 0).reshape(-1)
        q = st["inv_perm"][t * k + j].long()
        dgate[t, j] = torch.einsum("td,td->t", dout[t], st["y_perm"][q].double())
        dy[q] = st["gate"][t, j].double()[:, None] * dout[t]
    return {"dgate": dgate, "dy_perm": dy}


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _exact_linear, "balance": _exact_balance, "router_grad": _exact_router_grad,
            "combine_grad": _exact_combine_grad}[case["op"]](dict(case), st)
