"""moe_linear_w4 against the float64 oracle: formats, groups, types, token
counts from one to many, odd sizes, strides, epilogues, graphs and streams.

Tolerance.  Products are exact and the sums fp32: a step of the tensor cores
adds 16 products to a running sum with an error of at most one step, 2^-23, of
the largest magnitude in it, and the partial sums of a split add as many errors
as there are parts (at most 32).  With K/16 steps, an element is off by at most
(K/16 + 32) 2^-23 S, S = sum |w x| (no partial sum exceeds it), and as partial
sums of terms of random sign stay near the size of the result, the whole output
by (K/16 + 32) 2^-23 in norm.  Rounding y to bf16 or fp16 adds half a step of
the value: 2^-8 or 2^-11 of it.  SwiGLU is smooth: |silu'| <= 1.1, so its two
factors' errors add, each times the other factor (plus 2^-20 of the value for
the exponential and the quotient)."""
import numpy as np
import pytest
import torch

from oracle import linear as O
from tests.gpu_util import load_moe, require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    return load_moe()


def make(fmt, group, N, K, T, x="bf16", zeros=False, scale="bf16", seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + N * 31 + K * 7 + T)
    G = -(-K // group)
    w = dict(fmt=fmt, group=group, zeros=None, tensor_scale=1.0)
    w["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    if fmt == "int4":
        w["scales"] = (0.01 * (0.3 * torch.randn((N, G), generator=g)).exp()).to(DT[scale])
        if zeros:
            w["zeros"] = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8)
    elif fmt == "mxfp4":
        w["scales"] = torch.randint(115, 127, (N, G), generator=g, dtype=torch.uint8)
    else:
        w["scales"] = torch.randint(0, 127, (N, G), generator=g, dtype=torch.uint8)      # every finite positive E4M3
        w["tensor_scale"] = 0.0123
    return w, torch.randn((T, K), generator=g).to(DT[x])


def oracle_weights(w):
    s = w["scales"]
    s = s.double().numpy() if w["fmt"] == "int4" else s.numpy()
    z = None if w["zeros"] is None else w["zeros"].numpy()
    return O.weights(w["fmt"], w["codes"].numpy(), s, w["group"], z, w["tensor_scale"])


def call(moe, w, x, out, **kw):
    moe.moe_linear_w4(x, w["codes"], w["scales"], out, fmt=w["fmt"], group=w["group"], zeros=w["zeros"],
                      tensor_scale=w["tensor_scale"], **kw)


def cuda(w):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in w.items()}


def check(got, w, x, y, swiglu=False, y0=None):
    """got [T, N] against the oracle, by the tolerance above."""
    W, X = oracle_weights(w), x.double().numpy()
    ref = O.linear(X, W, swiglu, None if y0 is None else y0.double().numpy())
    got = got.double().cpu().numpy()
    step = (W.shape[1] / 16 + 32) * 2.0 ** -23
    S = np.abs(X) @ np.abs(W).T
    if swiglu:
        half = W.shape[0] // 2
        h, u = X @ W[:half].T, X @ W[half:].T
        tol = step * (1.1 * S[:, :half] * np.abs(u) + np.abs(O.silu(h)) * S[:, half:]) + 2.0 ** -20 * np.abs(ref)
    else:
        tol = step * S
    tol = tol + 2 * HALF_STEP[y] * np.abs(ref) + 2.0 ** -126
    if y0 is not None:
        tol = tol + 2.0 ** -23 * np.abs(ref - y0.double().numpy())
    if y == "f16":
        tol = tol + 2.0 ** -24
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"off by {(err / tol).max():.3g} of the tolerance"
    norm = np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-30)
    assert norm <= (3 if swiglu else 1) * step + 2 * HALF_STEP[y], f"off by {norm:.3g} in norm"


FORMATS = [("int4", 32, False), ("int4", 64, True), ("int4", 128, True), ("int4", 128, False), ("mxfp4", 32, False),
           ("nvfp4", 16, False)]


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 8, 9, 17, 33, 64, 65, 130])
def test_formats_and_token_counts(moe, fmt, group, zeros, T):
    w, x = make(fmt, group, 80, 512, T, zeros=zeros)
    out = torch.empty((T, 80), device="cuda")
    call(moe, cuda(w), x.cuda(), out)
    check(out, w, x, "f32")


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("N,K", [(1, 32), (7, 64), (16, 96), (17, 160), (33, 224), (250, 1120), (513, 2080), (3, 8192)])
def test_odd_sizes(moe, fmt, group, zeros, N, K):
    """Rows that end inside a tile, K that ends inside a group, a stage or a
    warp's share."""
    for T in (1, 11, 70):
        w, x = make(fmt, group, N, K, T, zeros=zeros, seed=1)
        out = torch.empty((T, N), device="cuda")
        call(moe, cuda(w), x.cuda(), out)
        check(out, w, x, "f32")


@pytest.mark.parametrize("x,y,scale", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f16"), ("f16", "f16", "f16"),
                                       ("f16", "f32", "f32"), ("f16", "f16", "bf16"), ("bf16", "bf16", "f32")])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_types(moe, fmt, group, zeros, x, y, scale):
    for T in (3, 80):
        w, xs = make(fmt, group, 96, 1024, T, x=x, zeros=zeros, scale=scale, seed=2)
        out = torch.empty((T, 96), dtype=DT[y], device="cuda")
        call(moe, cuda(w), xs.cuda(), out)
        check(out, w, xs, y)


@pytest.mark.parametrize("T", [1, 5, 40, 129])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("N", [2, 26, 256, 530])
def test_swiglu(moe, fmt, group, zeros, N, T):
    w, x = make(fmt, group, N, 352, T, zeros=zeros, seed=3)
    if fmt == "nvfp4":
        w["tensor_scale"] = 1e-4                       # h and u of ordinary size
    for y in ("f32", "bf16"):
        out = torch.empty((T, N // 2), dtype=DT[y], device="cuda")
        call(moe, cuda(w), x.cuda(), out, swiglu=True)
        check(out, w, x, y, swiglu=True)


@pytest.mark.parametrize("T", [1, 7, 50, 200])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_strides_and_accumulate(moe, T, y, swiglu):
    """Rows of x and out apart, the gaps untouched, y added to what is there."""
    w, x = make("int4", 64, 90, 288, T, zeros=True, seed=4)
    wide = torch.full((T, 288 + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :288] = x.cuda()
    n = 45 if swiglu else 90
    y0 = torch.randn((T, n)).to(DT[y])
    buf = torch.full((T + 1, n + 5), 7.0, dtype=DT[y], device="cuda")
    buf[:T, :n] = y0.cuda()
    call(moe, cuda(w), wide[:, :288], buf[:T, :n], swiglu=swiglu, accumulate=True)
    check(buf[:T, :n], w, x, y, swiglu=swiglu, y0=y0)
    assert (buf[T] == 7).all() and (buf[:, n:] == 7).all()


def test_scale_ranges(moe):
    """E8M0 scales over the whole range fp32 can hold, 255 as NaN; zeros above 15
    count by their low four bits."""
    K = 64
    w, x = make("mxfp4", 32, 17, K, 2, seed=5)
    w["scales"] = torch.tensor([[0, 1], [253, 20], [1, 200], [127, 127]] * 5, dtype=torch.uint8)[:17].contiguous()
    for T in (2, 66):
        xs = (torch.randn((T, K)) * 0.01).to(torch.bfloat16)
        out = torch.empty((T, 17), device="cuda")
        call(moe, cuda(w), xs.cuda(), out)
        ref = O.linear(xs.double().numpy(), oracle_weights(w))
        S = np.abs(xs.double().numpy()) @ np.abs(oracle_weights(w)).T
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= 36 * 2.0 ** -23 * S + 2.0 ** -140).all()
        bad = dict(w, scales=w["scales"].clone())
        bad["scales"][3, 1] = 255
        call(moe, cuda(bad), xs.cuda(), out)
        assert torch.isnan(out[:, 3]).all() and not torch.isnan(out[:, 4:]).any()
        z, xz = make("int4", 32, 20, K, T, zeros=True, seed=6)
        got = torch.empty((T, 20), device="cuda")
        call(moe, cuda(z), xz.cuda(), got)
        high = dict(z, zeros=z["zeros"] + 16 * 3)
        again = torch.empty_like(got)
        call(moe, cuda(high), xz.cuda(), again)
        assert torch.equal(got, again)


def test_negative_and_subnormal_e4m3_scales(moe):
    w, x = make("nvfp4", 16, 24, 256, 9, seed=7)
    w["scales"] = torch.arange(24 * 16, dtype=torch.int64).remainder(254).to(torch.uint8).reshape(24, 16)
    w["scales"][w["scales"] == 127] = 0
    for T in (9, 100):
        for dt in ("bf16", "f16"):
            xs = torch.randn((T, 256)).to(DT[dt])
            out = torch.empty((T, 24), device="cuda")
            call(moe, cuda(w), xs.cuda(), out)
            check(out, w, xs, "f32")


def test_non_finite_x_stays_in_its_row(moe):
    for T in (6, 90):
        w, x = make("int4", 128, 48, 256, T, seed=8)
        x[2, 100] = float("inf")
        x[4, 7] = float("nan")
        out = torch.empty((T, 48), device="cuda")
        call(moe, cuda(w), x.cuda(), out)
        fine = [t for t in range(T) if t not in (2, 4)]
        assert torch.isfinite(out[fine]).all()
        assert torch.isnan(out[4]).all() and not torch.isfinite(out[2]).all()


def test_no_tokens_and_no_second_row(moe):
    w, x = make("int4", 32, 16, 64, 1, seed=9)
    d = cuda(w)
    call(moe, d, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 16), device="cuda"))
    out = torch.empty((1, 16), device="cuda")
    call(moe, d, x.cuda(), out)
    check(out, w, x, "f32")


@pytest.mark.parametrize("T", [1, 16, 100])
def test_same_call_same_bits_and_graph(moe, T):
    """Two eager calls, a call on another stream and a replayed graph agree bit for bit."""
    w, x = make("int4", 128, 300, 4096, T, zeros=True, seed=10)
    d, xs = cuda(w), x.cuda()
    outs = [torch.empty((T, 300), device="cuda") for _ in range(4)]
    call(moe, d, xs, outs[0])
    call(moe, d, xs, outs[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(moe, d, xs, outs[2], stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(moe, d, xs, outs[3])
    outs[3].zero_()
    g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(outs[0], o)
    check(outs[0], w, x, "f32")


def test_offsets_past_31_bits(moe):
    """Code and output offsets above 2^31."""
    N, K, T = 1 << 20, 8192, 1                          # 4 GiB of codes
    d = dict(fmt="mxfp4", group=32, zeros=None, tensor_scale=1.0)
    d["codes"] = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda")      # every code 1.0
    d["scales"] = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    d["codes"][-1] = 0x44                                                              # 2.0
    x = torch.ones((T, K), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((T, N), device="cuda")
    call(moe, d, x, out)
    assert (out[0, :-1] == K).all() and out[0, -1] == 2 * K
    del d["codes"], out
    rows = 40000                                       # rows 65536 apart: offsets of x and y above 2^31
    x = torch.zeros((rows, 65536), dtype=torch.bfloat16, device="cuda")
    x[:, :32] = 1
    small, _ = make("int4", 32, 8, 32, 1, seed=11)
    y = torch.zeros((rows, 65536), dtype=torch.bfloat16, device="cuda")
    call(moe, cuda(small), x[:, :32], y[:, :8])
    ref = oracle_weights(small).sum(1)
    got = y[[0, rows - 1], :8].double().cpu().numpy()
    assert np.allclose(got, ref[None], rtol=2.0 ** -7, atol=1e-6)
    assert torch.equal(y[0, :8], y[rows - 1, :8]) and (y[:, 8:16] == 0).all()


def test_binding_refusals(moe):
    w, x = make("int4", 32, 16, 64, 2, seed=12)
    d, xs, out = cuda(w), x.cuda(), torch.empty((2, 16), device="cuda")
    for kw in (dict(x=xs.t().contiguous().t()), dict(out=torch.empty((2, 15), device="cuda")),
               dict(out=torch.empty((2, 16), dtype=torch.float64, device="cuda")), dict(x=xs.float()),
               dict(out=torch.empty((2, 16), dtype=torch.float16, device="cuda")), dict(group=64, scales=d["scales"][:8]),
               dict(scales=d["scales"].double()), dict(codes=d["codes"][:, :16]), dict(zeros=torch.zeros((16, 1),
               dtype=torch.uint8, device="cuda")), dict(out=torch.empty((1, 16), device="cuda").expand(2, 16)),
               dict(tensor_scale=1.0, fmt="mxfp4"), dict(zeros=torch.zeros((8, 4), dtype=torch.uint8, device="cuda"))):
        a = dict(x=xs, codes=d["codes"], scales=d["scales"], out=out, fmt="int4", group=32, zeros=None)
        a.update(kw)
        with pytest.raises((ValueError, moe.MoeError)):
            moe.moe_linear_w4(**a)


def test_out_overlaps_nothing_that_is_read(moe):
    """x and out as columns of one buffer are apart; any common element is refused."""
    N, K, T = 24, 64, 5
    w, x = make("int4", 32, N, K, T, seed=15)
    d = cuda(w)
    buf = torch.empty((T, 96), dtype=torch.bfloat16, device="cuda")
    buf[:, :K] = x.cuda()
    want = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    args = dict(fmt="int4", group=32)
    moe.moe_linear_w4(buf[:, :K], d["codes"], d["scales"], want, **args)
    moe.moe_linear_w4(buf[:, :K], d["codes"], d["scales"], buf[:, 64:88], **args)
    assert torch.equal(buf[:, 64:88], want) and torch.equal(buf[:, :K].cpu(), x)
    for t, out in ((T, buf[:, 63:87]), (T, buf[:, :N]), (1, buf[:1, 8:32])):
        with pytest.raises(ValueError, match="overlaps"):
            moe.moe_linear_w4(buf[:t, :K], d["codes"], d["scales"], out, **args)
    rows = torch.zeros((2 * T, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):                  # out's second row on x's first
        moe.moe_linear_w4(rows[1:3], d["codes"], d["scales"], rows[:2, :N], **args)
    with pytest.raises(ValueError, match="overlaps"):
        moe.moe_linear_w4(buf[:1, :K], d["codes"], d["scales"], d["scales"].view(-1)[:N].view(1, N), **args)
    moe.moe_linear_w4(rows[:0], d["codes"], d["scales"], rows[:0, :N], **args)
    with pytest.raises((ValueError, moe.MoeError)):                    # no K at all
        moe.moe_linear_w4(rows[:2, :0], d["codes"][:, :0], d["scales"][:, :0], want[:2], **args)


@pytest.mark.parametrize("T", [5, 24, 100])
def test_calls_at_once_from_two_threads(moe, T):
    """Two threads, a stream each, over the same weights: every result has the bits of
    a call alone."""
    import threading
    w, x = make("int4", 64, 1024, 2048, T, seed=16)
    d, xs = cuda(w), x.cuda()
    want = torch.empty((T, 1024), device="cuda")
    call(moe, d, xs, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.full((T, 1024), -1.0, device="cuda") for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    errors = []

    def run(s, os):
        try:
            for o in os:
                call(moe, d, xs, o, stream=s)
        except Exception as e:                                         # raised below, on the test's thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=a) for a in zip(streams, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for o in outs[0] + outs[1]:
        assert torch.equal(o, want)


def test_the_first_call_of_a_process_can_be_captured(moe):
    """Kernel attributes and the clusters' number are asked for inside the capture."""
    import subprocess
    import sys
    code = ("import torch, expert_offload_serving_b200 as m\n"
            "T, N, K = 24, 1024, 2048\n"
            "x = torch.randn((T, K), device='cuda').to(torch.bfloat16)\n"
            "c = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device='cuda')\n"
            "s = torch.ones((N, K // 64), dtype=torch.bfloat16, device='cuda')\n"
            "a, b = torch.zeros((T, N), device='cuda'), torch.zeros((T, N), device='cuda')\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n"
            "    m.moe_linear_w4(x, c, s, a, group=64)\n"
            "g.replay()\n"
            "m.moe_linear_w4(x, c, s, b, group=64)\n"
            "torch.cuda.synchronize()\n"
            "assert a.abs().max() > 0 and torch.equal(a, b)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("path", ["warp", "tc"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_fp32_scales_keep_their_bits_for_an_fp32_y(moe, monkeypatch, path, group):
    """bf16 x, fp32 scales: exact products and fp32 sums on both kernels.  At K = 4096
    the up to 8 additions of a group cut off up to a step of 2^-23 each, half of that
    on average: 8 2^-24 = 4.8e-7 of the group's sum and so of the whole (the groups'
    signs are random); 32 to 128 fp32 roundings of the running sum, each up to 2^-24,
    add as random errors do, at most sqrt(128 / 3) 2^-24 = 3.9e-7.  Below 1e-6 in norm
    together.  (A weight within 2^-14.8 of itself, 2^-16 on average, would be off by
    more than that.)"""
    monkeypatch.setenv("MOE_LINEAR", path)
    for T in (5, 24, 64, 130):
        w, x = make("int4", group, 200, 4096, T, zeros=True, scale="f32", seed=17)
        out = torch.empty((T, 200), device="cuda")
        call(moe, cuda(w), x.cuda(), out)
        check(out, w, x, "f32")
        ref = O.linear(x.double().numpy(), oracle_weights(w))
        norm = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert norm <= 1e-6, (T, norm)
