"""moe_linear_w4 where a CTA walks several tiles, where the 32-row and 16-token
instances run, and over long sums: every element against float64 (formed on the
GPU from the formats' definitions, as the matrices are large).

Tolerance: that of test_gpu_linear.py, element by element and in norm."""
import numpy as np
import pytest
import torch

from oracle import linear as O
from tests.gpu_util import load_moe, require_gpu
from tests.test_gpu_linear import DT, HALF_STEP, call

pytestmark = pytest.mark.gpu

FORMATS = [("int4", 32, True), ("int4", 64, False), ("int4", 64, True), ("int4", 128, True), ("mxfp4", 32, False),
           ("nvfp4", 16, False)]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    return load_moe()


def make(fmt, group, zeros, N, K, seed, scale="bf16"):
    g = torch.Generator("cuda").manual_seed(seed)
    w = dict(fmt=fmt, group=group, zeros=None, tensor_scale=1.0)
    w["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    G = -(-K // group)
    if fmt == "int4":
        w["scales"] = (0.01 * (0.3 * torch.randn((N, G), generator=g, device="cuda")).exp()).to(DT[scale])
        if zeros:
            w["zeros"] = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8, device="cuda")
    elif fmt == "mxfp4":
        w["scales"] = torch.randint(115, 123, (N, G), generator=g, dtype=torch.uint8, device="cuda")
    else:
        w["scales"] = torch.randint(0, 127, (N, G), generator=g, dtype=torch.uint8, device="cuda")
        w["tensor_scale"] = 1.5e-4
    return w, g


def dequant(w, rows):
    """Rows of W in float64."""
    c = w["codes"][rows]
    q = torch.stack([c & 15, c >> 4], 2).reshape(c.shape[0], -1)
    K = q.shape[1]
    if w["fmt"] == "int4":
        z = 8.0 if w["zeros"] is None else w["zeros"][rows].double().repeat_interleave(w["group"], 1)[:, :K]
        v, s = q.double() - z, w["scales"][rows].double()
    else:
        m = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[(q & 7).long()]
        v = torch.where(q >= 8, -m, m)
        s = w["scales"][rows]
        ts = float(np.float32(w["tensor_scale"]))                     # the call takes it in fp32
        s = torch.exp2(s.double() - 127) if w["fmt"] == "mxfp4" else s.view(torch.float8_e4m3fn).double() * ts
    return v * s.repeat_interleave(w["group"], 1)[:, :K]


def test_the_reference_is_the_oracles(moe):
    for fmt, group, zeros in FORMATS:
        w, _ = make(fmt, group, zeros, 20, 160, 1)
        cpu = {k: v.cpu() if torch.is_tensor(v) else v for k, v in w.items()}
        s = cpu["scales"].double().numpy() if fmt == "int4" else cpu["scales"].numpy()
        ref = O.weights(fmt, cpu["codes"].numpy(), s, group, None if cpu["zeros"] is None else cpu["zeros"].numpy(),
                        w["tensor_scale"])
        assert np.array_equal(dequant(w, slice(None)).cpu().numpy(), ref)


def products(w, x):
    """x W^T and |x| |W|^T in float64."""
    N, X = w["codes"].shape[0], x.double()
    y, s = (torch.empty((x.shape[0], N), dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, (1 << 26) // (2 * w["codes"].shape[1]))
    for n in range(0, N, step):
        W = dequant(w, slice(n, n + step))
        y[:, n:n + step], s[:, n:n + step] = X @ W.t(), X.abs() @ W.abs().t()
    return y, s


def check(got, y, S, K, dtype, swiglu=False, y0=None):
    step = (K / 16 + 32) * 2.0 ** -23
    if swiglu:
        half = y.shape[1] // 2
        h, u = y[:, :half], y[:, half:]
        ref = h * torch.sigmoid(h) * u
        tol = step * (1.1 * S[:, :half] * u.abs() + (h * torch.sigmoid(h)).abs() * S[:, half:]) + 2.0 ** -20 * ref.abs()
    else:
        ref, tol = y, step * S
    if y0 is not None:
        tol = tol + 2.0 ** -23 * ref.abs()
        ref = ref + y0.double()
    tol = tol + 2 * HALF_STEP[dtype] * ref.abs() + (2.0 ** -24 if dtype == "f16" else 2.0 ** -126)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), f"off by {float((err / tol).max()):.3g} of the tolerance"
    norm = float(err.norm() / ref.norm())
    assert norm <= (3 if swiglu else 1) * step + 2 * HALF_STEP[dtype], f"off by {norm:.3g} in norm"
    return norm


@pytest.mark.parametrize("path", ["warp", "tc"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("K", [1056, 1312])
def test_few_tokens_and_more_tiles_than_sms(moe, monkeypatch, path, fmt, group, zeros, K):
    """N just above a tile of 128 rows for every SM, the last tile partial; 9 or 11
    stages of 128 (5 or 6 of 256), the last partial.  Both x types, SwiGLU, and rows
    apart with accumulation."""
    monkeypatch.setenv("MOE_LINEAR", path)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for N in (128 * sms + 75, 128 * sms + 74):
        swiglu = N % 2 == 0
        n = N // 2 if swiglu else N
        w, g = make(fmt, group, zeros, N, K, 2)
        X = torch.randn((16, K), generator=g, device="cuda")
        for xt in ("bf16", "f16"):
            x = X.to(DT[xt])
            y, S = products(w, x)
            for T in (1, 8, 13, 16):
                out = torch.empty((T, n), device="cuda")
                call(moe, w, x[:T], out, swiglu=swiglu)
                check(out, y[:T], S[:T], K, "f32", swiglu)
            T = 11
            y0 = torch.randn((T, n), generator=g, device="cuda").to(DT[xt])
            buf = torch.full((T, n + 9), 7.0, dtype=DT[xt], device="cuda")
            buf[:, :n] = y0
            xs = torch.full((T, K + 8), float("nan"), dtype=DT[xt], device="cuda")
            xs[:, :K] = x[:T]
            call(moe, w, xs[:, :K], buf[:, :n], swiglu=swiglu, accumulate=True)
            check(buf[:, :n], y[:T], S[:T], K, xt, swiglu, y0)
            assert (buf[:, n:] == 7).all()


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("T", [24, 64, 200])
def test_many_tokens_and_more_tiles_than_sms(moe, monkeypatch, fmt, group, zeros, T):
    """The same of the kernel for more tokens: CTAs walk several tiles of 9 stages, so
    the sets' roles change from tile to tile."""
    monkeypatch.setenv("MOE_LINEAR", "tc")
    sms, K = torch.cuda.get_device_properties(0).multi_processor_count, 1056
    for N in (128 * sms + 75, 128 * sms + 74):
        swiglu = N % 2 == 0
        n = N // 2 if swiglu else N
        w, g = make(fmt, group, zeros, N, K, 3)
        for xt, yt in (("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")):
            x = torch.randn((T, K), generator=g, device="cuda").to(DT[xt])
            y, S = products(w, x)
            out = torch.empty((T, n), dtype=DT[yt], device="cuda")
            call(moe, w, x, out, swiglu=swiglu)
            check(out, y, S, K, yt, swiglu)


@pytest.mark.parametrize("T", [24, 64, 130])
@pytest.mark.parametrize("fmt,group,zeros", [("int4", 64, True), ("mxfp4", 32, False), ("nvfp4", 16, False)])
@pytest.mark.parametrize("K", [16384, 16384 + 128, 16384 + 256, 16384 + 1024 + 32])
@pytest.mark.parametrize("wide", [False, True])
def test_long_sums_of_an_fp32_y_are_added_in_registers(moe, fmt, group, zeros, T, K, wide):
    """At most 1024 of K run through the tensor cores' truncating additions: 4.8e-7 of
    the norm measured at K = 16384, and 2.4e-6 (shared by a cluster) or 7.7e-6 (not)
    where the sums run through all of K; the bound lies between.  wide: enough rows that
    no cluster shares a tile."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N = 128 * sms if wide else 384
    w, g = make(fmt, group, zeros, N, K, 4)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((T, N), device="cuda")
    call(moe, w, x, out)
    assert check(out, *products(w, x), K, "f32") <= 1e-6


@pytest.mark.parametrize("path", ["warp", "tc"])
@pytest.mark.parametrize("T,N", [(1 << 20, 24), (1, 1 << 24), (20, 1 << 24)])
def test_the_most_tokens_and_the_most_rows(moe, monkeypatch, path, T, N):
    monkeypatch.setenv("MOE_LINEAR", path)
    w, g = make("int4", 32, True, N, 32, 5)
    x = torch.randn((T, 32), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((T, N), device="cuda")
    call(moe, w, x, out)
    for t in range(0, T, 1 << 18):
        for n in range(0, N, 1 << 22):
            part = dict(w, codes=w["codes"][n:n + (1 << 22)], scales=w["scales"][n:n + (1 << 22)],
                        zeros=w["zeros"][n:n + (1 << 22)])
            y, S = products(part, x[t:t + (1 << 18)])
            check(out[t:t + (1 << 18), n:n + (1 << 22)], y, S, 32, "f32")


@pytest.mark.parametrize("path", ["warp", "tc"])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_subnormal_x(moe, monkeypatch, path, fmt, group, zeros):
    """x below the type's normal range counts with its value (a flushed one would be 0)."""
    monkeypatch.setenv("MOE_LINEAR", path)
    for xt, size in (("bf16", 2.0 ** -126), ("f16", 2.0 ** -14)):
        for T in (5, 40):
            w, g = make(fmt, group, zeros, 96, 512, 6)
            x = (torch.randint(-127, 128, (T, 512), generator=g, device="cuda") * (size / 128)).to(DT[xt])
            assert bool((x.float().abs() < size).all()) and bool((x != 0).any())
            if fmt == "mxfp4":
                w["scales"] += 127 + 30 - 115                          # the results are normal fp32 values
            elif fmt == "nvfp4":
                w["tensor_scale"] = 2.0 ** 30
            else:
                w["scales"] = (w["scales"].float() * 2.0 ** 40).to(torch.bfloat16)
            out = torch.empty((T, 96), device="cuda")
            call(moe, w, x, out)
            check(out, *products(w, x), 512, "f32")
