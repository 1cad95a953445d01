"""The 8-bit activation path on the GPU against the fp64 oracle.

Tolerances, u = 2^-24 (half a step of fp32) and 2^-8 half a step of bf16:

  norm     sum of squares: at most 40 fp32 additions and fused steps deep for
           any value (lane, tree over lanes and waves), every addend positive,
           so its relative error is below 40 u and that of its root below 20 u;
           mean, root, reciprocal, gain and the last product add 6 u.  Scales
           add the division by 127 and one product.  Below: 32 u for values
           and scales.
  silu     exp within 1.5 ulp (3 u), 1 + e (1 u), reciprocal within 1 ulp
           (2 u), two products (2 u): 8 u, and 2^-118 |u_max| where the reciprocal
           of a number past 2^126 is flushed.
  integers to the bit for the norm and quantize (the definition rounds every
           step in fp32); for silu p carries 8 u and the step another 10 u:
           an integer may move by one where p / s is within 127 * 20 u of a tie.
  product  the integer sum is exact; its conversion, the product of the scales
           and the scaling are 1 u each, the bias one more rounding of y:
           3.1 u |product| + 1.1 u |y|.
"""
import itertools
import random
import sys

import numpy as np
import pytest
import torch

import workloads
from oracle import int8 as o8
from oracle import products

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_canonical_amd as uw  # noqa: E402

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}


def _say(msg):
    print(f"[gpu-int8] {msg}", flush=True)
    sys.stdout.flush()


def f64(t):
    return t.detach().double().cpu().numpy()


def inside(rows, cols, dtype, pad=0, shift=0, fill=0x5A):
    """A [rows, cols] view with row stride cols + pad, `shift` elements into a
    larger buffer whose other bytes all hold `fill`; (view, check that they
    still do)."""
    n = rows * (cols + pad) + shift + 64
    raw = torch.full((n * torch.empty(0, dtype=dtype).element_size(),), fill, dtype=torch.uint8, device=DEV)
    flat = raw.view(dtype)
    view = flat[shift: shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    def untouched():
        view.view(dtype).copy_(torch.zeros_like(view))
        rest = flat.clone()
        m = torch.ones_like(flat, dtype=torch.bool)
        m[shift: shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False
        got = rest[m].view(torch.uint8)
        return bool((got == fill).all())

    return view, untouched


def rand(rows, cols, dtype, seed, pad=0, shift=0, loud=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if loud and cols > 8:
        x[:, :: max(1, cols // 5)] *= 17
    v, _ = inside(rows, cols, dtype, pad, shift)
    v.copy_(x.to(dtype))
    return v


def check(got, ref, rel, dtype, what, floor=0.0):
    got, ref = f64(got), np.asarray(ref, np.float64)
    bad = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what + ": NaN pattern"
    err = np.abs(got - ref)
    lim = np.abs(ref) * (rel * (1 + HALF[dtype]) + (HALF[dtype] if dtype != torch.float32 else 0)) + floor
    over = (err > lim) & ~bad
    assert not over.any(), f"{what}: {over.sum()} of {over.size} off, worst {np.nanmax(np.where(bad, 0, err / np.maximum(lim, 1e-300))):.3g} of the tolerance"


NORM_COLS = [1, 7, 8, 9, 64, 511, 512, 513, 1000, 1024, 1025, 2048, 2056, 4096, 5001, 8192, 8200, 14336, 16384, 32768, 32769, 40003]


def run_norm(b, cols, x, res, gain, out, pad=0, shift=0, seed=1, X=None, R=None):
    X = rand(b, cols, DT[x], seed, pad, shift) if X is None else X
    if R is None and res != "none":
        R = rand(b, cols, DT[res], seed + 1, pad, shift)
    g = None
    if gain != "none":
        g = (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed + 2))).to(DT[gain]).to(DEV)
    Y, y_ok = inside(b, cols, DT[out], pad, shift)
    H, h_ok = (None, None) if R is None else inside(b, cols, R.dtype, pad, shift)
    scale = torch.full((b + 2,), 7.0, device=DEV)
    sc = scale[1: b + 1] if out == "i8" else None
    uw.uw_rmsnorm(X, g, Y, scale=sc, residual=R, residual_out=H, eps=EPS)
    torch.cuda.synchronize()
    what = f"norm b={b} cols={cols} x={x} res={res} gain={gain} out={out} pad={pad} shift={shift}"
    h = o8.norm_h(f64(X), None if R is None else f64(R), R is not None and R.dtype == torch.bfloat16)
    if H is not None:
        assert np.array_equal(f64(H), h, equal_nan=True), what + ": h"
    gn = None if g is None else f64(g)
    if out == "i8":
        p = h.astype(np.float32) if gn is None else (h.astype(np.float32) * gn.astype(np.float32))
        q, s = o8.quantize(p)
        assert np.array_equal(Y.cpu().numpy(), q), f"{what}: {(Y.cpu().numpy() != q).sum()} integers differ"
        check(sc, s.astype(np.float64) * o8.rstd(h, EPS), 32 * U, torch.float32, what + ": scale")
        assert scale[0] == 7 and scale[-1] == 7
    else:
        check(Y, o8.rmsnorm(h, gn, EPS), 32 * U, DT[out], what)
    assert y_ok(), what + ": wrote outside Y"
    if H is not None:
        assert h_ok(), what + ": wrote outside h"


@pytest.mark.parametrize("cols", NORM_COLS)
def test_norm_widths(cols):
    _say(f"norm cols={cols}")
    for b, (x, res, out) in zip((1, 3, 5, 2, 4, 1), (("bf16", "bf16", "i8"), ("bf16", "none", "bf16"), ("f32", "bf16", "i8"),
                                                     ("bf16", "f32", "f32"), ("f32", "f32", "bf16"), ("f32", "none", "i8"))):
        run_norm(b, cols, x, res, "bf16" if x == "bf16" else "f32", out, seed=cols)


@pytest.mark.parametrize("x,res,gain,out", list(itertools.product(("bf16", "f32"), ("none", "bf16", "f32"), ("none", "bf16", "f32"), ("i8", "bf16", "f32"))))
def test_norm_types(x, res, gain, out):
    run_norm(3, 777, x, res, gain, out, seed=5)
    run_norm(2, 4096, x, res, gain, out, pad=8, seed=6)


@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 1), (5, 3), (16, 7)])
@pytest.mark.parametrize("cols", [5, 500, 1333, 4097, 33001])
def test_norm_strides_and_offsets(cols, pad, shift):
    run_norm(4, cols, "bf16", "bf16", "bf16", "i8", pad, shift)
    run_norm(4, cols, "f32", "bf16", "bf16", "bf16", pad, shift)
    run_norm(4, cols, "bf16", "f32", "f32", "f32", pad, shift)


def test_norm_many_rows():
    run_norm(1111, 4096, "bf16", "bf16", "bf16", "i8")
    run_norm(2049, 96, "bf16", "f32", "bf16", "bf16")
    # streams of over 16 MiB
    run_norm(2100, 4096, "bf16", "bf16", "bf16", "i8")
    run_norm(1030, 4101, "bf16", "f32", "bf16", "bf16", pad=3, shift=1)
    run_norm(140, 33000, "f32", "f32", "f32", "f32")


def special_rows(cols, dtype):
    """Rows of zeros, tiny values, one loud value, infinities and NaN."""
    X = torch.randn(9, cols, generator=torch.Generator().manual_seed(3))
    X[0] = 0
    X[1] *= 1e-30
    X[2] = 0
    X[2, -1] = 3.0
    X[3] *= 1e-3
    X[3, cols // 2] = 1e15
    X[4, 0] = float("inf")
    X[5, -1] = float("nan")
    X[6] = float("-inf")
    X[7] = -0.0
    X[8] = 1e-40
    return X.to(dtype).to(DEV)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 33000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_rows(cols, dtype):
    X = special_rows(cols, dtype)
    xn = f64(X).astype(np.float32)
    # 8 bits of the rows themselves
    Q, s = uw.i8_rows(9, cols), torch.empty(9, device=DEV)
    uw.uw_i8_quantize(X, Q, s)
    q, sn = o8.quantize(xn)
    assert np.array_equal(Q.cpu().numpy(), q)
    assert np.array_equal(s.cpu().numpy(), sn, equal_nan=True)
    # the norm: rows with an infinity or a NaN give a NaN scale, zeros stay zeros
    uw.uw_rmsnorm(X, None, Q, scale=s, eps=EPS)
    assert np.array_equal(Q.cpu().numpy(), q)
    s = s.cpu().numpy()
    fine = np.isfinite(xn).all(axis=1)
    assert np.isnan(s[~fine]).all() and np.isfinite(s[fine]).all()
    Y = torch.empty(9, cols, device=DEV)
    uw.uw_rmsnorm(X, None, Y, eps=EPS)
    y = Y.cpu().numpy()
    assert np.isnan(y[5]).all() and np.isnan(y[4, 0]) and (y[4, 1:] == 0).all() and np.isnan(y[6]).all()
    check(Y[:4], o8.rmsnorm(f64(X)[:4], None, EPS), 32 * U, torch.float32, "special norm")
    assert (y[[0, 7]] == 0).all()
    # their product is NaN, the others' is not
    W, ws = rand_i8(33, cols, 4)
    out = torch.empty(9, 33, device=DEV)
    uw.uw_i8_gemm(W, ws, Q, torch.from_numpy(s).to(DEV), out)
    out = out.cpu().numpy()
    assert np.isnan(out[~fine]).all() and np.isfinite(out[fine]).all()


def test_norm_squares_past_fp32():
    X = torch.full((2, 300), 3e38, device=DEV)
    X[1] = 1.0
    Y, Q, s = torch.empty(2, 300, device=DEV), uw.i8_rows(2, 300), torch.empty(2, device=DEV)
    uw.uw_rmsnorm(X, None, Y)
    uw.uw_rmsnorm(X, None, Q, scale=s)
    assert (Y[0] == 0).all() and s[0] == 0 and (Y[1] > 0.99).all()


@pytest.mark.parametrize("cols", [96, 4096, 5003, 34000])
def test_norm_in_place(cols):
    for dt in (torch.bfloat16, torch.float32):
        X, R = rand(3, cols, dt, 1), rand(3, cols, dt, 2)
        g = torch.ones(cols, device=DEV)
        Y0, H0 = torch.empty(3, cols, dtype=dt, device=DEV), torch.empty(3, cols, dtype=dt, device=DEV)
        uw.uw_rmsnorm(X, g, Y0, residual=R, residual_out=H0)
        # the stream updated in place
        R1, Y = R.clone(), torch.empty_like(Y0)
        uw.uw_rmsnorm(X, g, Y, residual=R1, residual_out=R1)
        assert torch.equal(R1, H0) and torch.equal(Y, Y0)
        # h into X
        X1, Y = X.clone(), torch.empty_like(Y0)
        uw.uw_rmsnorm(X1, g, Y, residual=R, residual_out=X1)
        assert torch.equal(X1, H0) and torch.equal(Y, Y0)
        # y into X, h into the residual
        X1, R1 = X.clone(), R.clone()
        uw.uw_rmsnorm(X1, g, X1, residual=R1, residual_out=R1)
        assert torch.equal(X1, Y0) and torch.equal(R1, H0)
        # y into X, h not kept; and the same tensor twice
        X1 = X.clone()
        uw.uw_rmsnorm(X1, g, X1, residual=R)
        assert torch.equal(X1, Y0)
        X1, Y1 = X.clone(), torch.empty_like(Y0)
        uw.uw_rmsnorm(X1, g, Y1, residual=X1, residual_out=X1)
        assert torch.equal(X1, (X.float() * 2).to(dt))


def run_silu(b, cols, x, out, pad=0, shift=0, seed=1, halves=False, scale_by=3.0):
    if halves:
        GU = rand(b, 2 * cols, DT[x], seed, pad, shift)
        G, V = GU[:, :cols], GU[:, cols:]
    else:
        G, V = rand(b, cols, DT[x], seed, pad, shift), rand(b, cols, DT[x], seed + 1, 2 * pad, shift)
    G.copy_(G * scale_by)
    Y, y_ok = inside(b, cols, DT[out], pad, shift)
    s = torch.empty(b, device=DEV) if out == "i8" else None
    uw.uw_silu_mul(G, V, Y, scale=s)
    torch.cuda.synchronize()
    p = o8.silu_mul(f64(G), f64(V))
    what = f"silu b={b} cols={cols} x={x} out={out} pad={pad} shift={shift}"
    floor = 2.0 ** -118 * max(1e-30, float(np.abs(f64(V)).max()))
    if out == "i8":
        top = np.abs(p).max(axis=1)
        step = np.maximum(top / 127, 2.0 ** -126)
        check(s, step, 10 * U, torch.float32, what + ": scale", floor)
        q = Y.cpu().numpy().astype(np.float64)
        want = p / step[:, None]
        off = np.abs(q - want)
        assert (off <= 0.5 + 127 * 20 * U).all(), f"{what}: integer off by {off.max()}"
    else:
        check(Y, p, 8 * U, DT[out], what, floor)
    assert y_ok(), what + ": wrote outside Y"


@pytest.mark.parametrize("cols", [1, 7, 8, 65, 512, 520, 1024, 1500, 2048, 4096, 4104, 8192, 14336, 16385, 32768, 33333])
def test_silu_widths(cols):
    _say(f"silu cols={cols}")
    for b, (x, out) in zip((1, 2, 3, 5, 4, 2), itertools.product(("bf16", "f32"), ("i8", "bf16", "f32"))):
        run_silu(b, cols, x, out, seed=cols)


@pytest.mark.parametrize("pad,shift", [(1, 1), (8, 0), (13, 5)])
def test_silu_strides(pad, shift):
    for cols in (100, 1001, 4096, 14336):
        run_silu(4, cols, "bf16", "i8", pad, shift, halves=True)
        run_silu(3, cols, "f32", "bf16", pad, shift)


def test_silu_extremes():
    run_silu(3, 1000, "f32", "f32", scale_by=400.0)  # exp over- and underflows on both sides
    G = torch.tensor([[0.0, -0.0, 100.0, -100.0, float("inf"), 1.0, float("nan")]], device=DEV)
    V = torch.tensor([[2.0, 2.0, 2.0, 2.0, 2.0, float("inf"), 1.0]], device=DEV)
    Y = torch.empty_like(G)
    uw.uw_silu_mul(G, V, Y)
    y = Y.cpu().numpy()[0]
    assert y[0] == 0 and y[1] == 0 and y[2] == 200 and abs(y[3]) < 1e-40 and np.isinf(y[4]) and np.isinf(y[5]) and np.isnan(y[6])
    X = rand(2, 640, torch.bfloat16, 9)
    Y = torch.empty_like(X)
    uw.uw_silu_mul(X, X, Y)  # one tensor for both
    X1 = X.clone()
    uw.uw_silu_mul(X1, X, X1)  # in place
    assert torch.equal(X1, Y)


@pytest.mark.parametrize("rows,cols,x,pad,shift", [
    (1, 1, "f32", 0, 0), (3, 5, "bf16", 1, 1), (37, 1001, "f32", 0, 0), (64, 4096, "bf16", 0, 0), (5, 14336, "bf16", 8, 0),
    (2, 40000, "f32", 3, 1), (1000, 64, "bf16", 0, 0), (300, 513, "bf16", 7, 3)])
def test_quantize_and_back(rows, cols, x, pad, shift):
    X = rand(rows, cols, DT[x], 3, pad, shift)
    Q, q_ok = inside(rows, cols, torch.int8, pad, shift)
    s = torch.empty(rows, device=DEV)
    uw.uw_i8_quantize(X, Q, s)
    q, sn = o8.quantize(f64(X).astype(np.float32))
    assert np.array_equal(Q.cpu().numpy(), q) and np.array_equal(s.cpu().numpy(), sn)
    for out in ("f32", "bf16"):
        Y, y_ok = inside(rows, cols, DT[out], pad, shift)
        uw.uw_i8_dequantize(Q, s, Y)
        v = q.astype(np.float32) * sn[:, None]  # one fp32 rounding, then the type's
        assert np.array_equal(f64(Y), v.astype(np.float64) if out == "f32" else o8.to_bf16(v.astype(np.float64)))
        # the value is half a step away at most (and the fp32 roundings of p * (1 / s))
        if out == "f32":
            assert (np.abs(f64(Y) - f64(X)) <= sn.astype(np.float64)[:, None] * (0.5 + 127 * 4 * U)).all()
        assert y_ok()
    assert q_ok()


def test_quantize_more_rows_than_a_launch_holds():
    rows = (1 << 21) + 5
    X = torch.randn(rows, 8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    Q, s = torch.zeros(rows, 16, dtype=torch.int8, device=DEV)[:, :8], torch.zeros(rows, device=DEV)
    uw.uw_i8_quantize(X, Q, s)
    for at in (slice(0, 7), slice((1 << 21) - 3, rows)):
        q, sn = o8.quantize(X[at].cpu().numpy())
        assert np.array_equal(Q[at].cpu().numpy(), q) and np.array_equal(s[at].cpu().numpy(), sn)
    Y = torch.empty(rows, 8, device=DEV)
    uw.uw_i8_dequantize(Q, s, Y)
    assert torch.equal(Y, Q.float() * s[:, None])


# -- product -------------------------------------------------------------------

def rand_i8(rows, cols, seed, pad=None, shift=0, extreme=False):
    """Integers over the whole range (-128 too), rows at multiples of 16 bytes unless pad says otherwise."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-128, 128, (rows, cols), generator=g, dtype=torch.int16).to(torch.int8)
    if extreme:
        q = torch.full((rows, cols), -128, dtype=torch.int8)
    v, _ = inside(rows, cols, torch.int8, (-cols) % 16 if pad is None else pad, shift)
    v.copy_(q)
    return v, (0.01 + torch.rand(rows, generator=g)).to(DEV)


def run_gemm(b, rows, cols, out="f32", bias=False, shape=0, ks=0, pad=None, shift=0, ypad=0, seed=1, extreme=False):
    W, ws = rand_i8(rows, cols, seed, pad, shift, extreme)
    X, xs = rand_i8(b, cols, seed + 1, pad, shift, extreme)
    bb = torch.randn(rows, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) * 100 if bias else None
    Y, y_ok = inside(b, rows, DT[out], ypad, shift)
    if shape:
        uw.uw_i8_gemm_shaped(W, ws, X, xs, Y, shape, ks, bias=bb)
    else:
        uw.uw_i8_gemm(W, ws, X, xs, Y, bias=bb)
    torch.cuda.synchronize()
    y, prod = o8.gemm(W.cpu().numpy(), f64(ws), X.cpu().numpy(), f64(xs), None if bb is None else f64(bb))
    what = f"gemm b={b} rows={rows} cols={cols} out={out} bias={bias} shape={shape} ks={ks} pad={pad} shift={shift}"
    half = HALF[DT[out]] if out == "bf16" else 0.0
    lim = (3.1 * U * np.abs(prod) + 1.1 * U * np.abs(y)) * (1 + half) + half * np.abs(y)
    err = np.abs(f64(Y) - y)
    assert (err <= lim).all(), f"{what}: {(err > lim).sum()} of {err.size} off"
    assert y_ok(), what + ": wrote outside Y"


SIZES = [(1, 1, 1), (1, 16, 64), (2, 3, 5), (5, 17, 63), (16, 16, 256), (17, 33, 257), (31, 100, 129), (33, 65, 1000),
         (64, 64, 128), (65, 130, 384), (100, 200, 1023), (129, 257, 640), (3, 1000, 4100), (300, 72, 515), (257, 513, 127)]


@pytest.mark.parametrize("shape", range(1, uw.uw_i8_gemm_shape_count()))
@pytest.mark.parametrize("b,rows,cols", SIZES)
def test_gemm_shapes(b, rows, cols, shape):
    _say(f"gemm shape={shape} b={b} rows={rows} cols={cols}")
    run_gemm(b, rows, cols, "f32", bias=True, shape=shape)
    run_gemm(b, rows, cols, "bf16", shape=shape, ypad=5, shift=16)


@pytest.mark.parametrize("ks", range(1, 9))
@pytest.mark.parametrize("cols", [100, 256, 1500, 4096])
def test_gemm_direct_waves(ks, cols):
    run_gemm(20, 48, cols, "f32", shape=1, ks=ks)


@pytest.mark.parametrize("shape", range(4, uw.uw_i8_gemm_shape_count()))
def test_gemm_whole_lines(shape):
    """Rows of Y at multiples of 128 bytes (the others above mostly are not), with the row's end inside a line."""
    for b, rows, out in ((300, 512, "bf16"), (300, 320, "f32"), (130, 500, "bf16"), (70, 250, "f32")):
        run_gemm(b, rows, 384, out, bias=True, shape=shape, ypad=-rows % (64 if out == "bf16" else 32))


@pytest.mark.parametrize("b", [1, 2, 8, 15, 16, 17, 32, 33, 48, 64, 65, 96, 128, 200, 256])
@pytest.mark.parametrize("rows,cols", [(1024, 1024), (1000, 4100), (517, 333)])
def test_gemm_auto(b, rows, cols):
    run_gemm(b, rows, cols, "bf16" if b % 2 else "f32", bias=b % 3 == 0)


@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (3, 5), (16, 3), (8, 8)])
@pytest.mark.parametrize("b", [1, 20, 70])
def test_gemm_unaligned_operands(b, pad, shift):
    for cols in (333, 256, 1025):
        run_gemm(b, 130, cols, "f32", pad=pad, shift=shift, bias=True)
        run_gemm(b, 37, cols, "bf16", pad=pad, shift=shift, ypad=3)
        for shape in range(1, 4):
            run_gemm(b, 130, cols, "f32", pad=pad, shift=shift, shape=shape)


def test_gemm_unaligned_large():
    run_gemm(2100, 2100, 130, "bf16", pad=0, shift=3, bias=True)
    run_gemm(300, 1000, 4100, "f32", pad=0)


def test_gemm_mlp_sizes():
    run_gemm(1, 14336, 4096, "bf16")
    run_gemm(32, 4096, 14336, "f32")
    run_gemm(300, 4096, 4096, "bf16", bias=True)


def test_gemm_longest_sum_is_exact():
    # every product is 128 * 128: the sum is 131071 * 2^14, just under 2^31
    run_gemm(3, 20, 131071, "f32", extreme=True)
    run_gemm(70, 40, 131071, "f32", extreme=True)
    for shape in range(1, uw.uw_i8_gemm_shape_count()):
        run_gemm(2, 16, 131071, "f32", shape=shape, extreme=True)


def test_gemm_offsets_past_32_bits():
    """Operands whose last rows start beyond 2^31 (staged shapes) and 2^32 bytes (direct)."""
    cols = 200
    for ld, rows, shape in (((1 << 22) - 16, 600, 0), ((1 << 22) - 16, 600, uw.uw_i8_gemm_shape_count() - 1), ((1 << 30) + 3, 5, 0)):
        raw = torch.empty((rows - 1) * ld + cols, dtype=torch.int8, device=DEV)
        W = torch.as_strided(raw, (rows, cols), (ld, 1))
        W0, ws = rand_i8(rows, cols, 5)
        W.copy_(W0)
        X, xs = rand_i8(70, cols, 6)
        Y, Y0 = torch.empty(70, rows, device=DEV), torch.empty(70, rows, device=DEV)
        if shape:
            uw.uw_i8_gemm_shaped(W, ws, X, xs, Y, shape)
        else:
            uw.uw_i8_gemm(W, ws, X, xs, Y)
        uw.uw_i8_gemm(W0, ws, X, xs, Y0)
        assert torch.equal(Y, Y0)
        # the same operand as the activations
        Y, Y0 = torch.empty(rows, 70, device=DEV), torch.empty(rows, 70, device=DEV)
        uw.uw_i8_gemm(X, xs, W, ws, Y)
        uw.uw_i8_gemm(X, xs, W0, ws, Y0)
        assert torch.equal(Y, Y0)
        del raw, W


def test_rows_offsets_past_32_bits():
    cols, ld = 1000, (1 << 31) + 24
    raw = torch.empty(ld + cols, dtype=torch.bfloat16, device=DEV)
    X = torch.as_strided(raw, (2, cols), (ld, 1))
    X0 = rand(2, cols, torch.bfloat16, 8)
    X.copy_(X0)
    Y, Y0 = torch.empty(2, cols, device=DEV), torch.empty(2, cols, device=DEV)
    uw.uw_rmsnorm(X, None, Y)
    uw.uw_rmsnorm(X0, None, Y0)
    assert torch.equal(Y, Y0)
    uw.uw_rmsnorm(X0, None, X, residual=X0)  # written there
    uw.uw_rmsnorm(X0, None, Y0, residual=X0)
    assert torch.equal(X.float(), Y0.to(torch.bfloat16).float())


# -- together ------------------------------------------------------------------

class Mlp:
    """norm -> gate and up in one product -> silu -> down, all in 8 bits."""

    def __init__(self, b, dim, hid, seed=1, dev=DEV):
        g = torch.Generator().manual_seed(seed)
        mk = lambda *s: (0.05 * torch.randn(*s, generator=g)).to(torch.bfloat16).to(dev)  # noqa: E731
        self.gu, self.down = uw.Int8Matrix.from_weights(mk(2 * hid, dim)), uw.Int8Matrix.from_weights(mk(dim, hid))
        self.x, self.r = mk(b, dim) * 20, mk(b, dim) * 20
        self.gain = (1 + mk(dim))
        self.hid = hid
        self.h = torch.empty_like(self.r)
        self.q, self.qs = uw.i8_rows(b, dim, dev), torch.empty(b, device=dev)
        self.GU = torch.empty(b, 2 * hid, dtype=torch.bfloat16, device=dev)
        self.a, self.as_ = uw.i8_rows(b, hid, dev), torch.empty(b, device=dev)
        self.y = torch.empty(b, dim, device=dev)

    def run(self, stream=None):
        uw.uw_rmsnorm(self.x, self.gain, self.q, scale=self.qs, residual=self.r, residual_out=self.h, stream=stream)
        self.gu.gemm(self.q, self.qs, self.GU, stream=stream)
        uw.uw_silu_mul(self.GU[:, : self.hid], self.GU[:, self.hid:], self.a, scale=self.as_, stream=stream)
        self.down.gemm(self.a, self.as_, self.y, stream=stream)


@pytest.mark.parametrize("b,dim,hid", [(1, 1024, 2816), (7, 256, 1000), (70, 512, 1536)])
def test_mlp_together(b, dim, hid):
    m = Mlp(b, dim, hid)
    m.run()
    torch.cuda.synchronize()
    # step by step against the oracle, each from the operands the step read
    h = o8.norm_h(f64(m.x), f64(m.r), True)
    assert np.array_equal(f64(m.h), h)
    q, s = o8.quantize(h.astype(np.float32) * f64(m.gain).astype(np.float32))
    assert np.array_equal(m.q.cpu().numpy(), q)
    check(m.qs, s * o8.rstd(h, EPS), 32 * U, torch.float32, "scale")
    gu, _ = o8.gemm(m.gu.q.cpu().numpy(), f64(m.gu.scale), q, f64(m.qs))
    check(m.GU, gu, 4 * U, torch.bfloat16, "gate and up")
    got = f64(m.GU)
    p = o8.silu_mul(got[:, :hid], got[:, hid:])
    assert (np.abs(f64(m.a) * f64(m.as_)[:, None] - p) <= f64(m.as_)[:, None] * (0.5 + 127 * 20 * U)).all()
    y, prod = o8.gemm(m.down.q.cpu().numpy(), f64(m.down.scale), m.a.cpu().numpy(), f64(m.as_))
    check(m.y, y, 4 * U, torch.float32, "down")
    # and against the MLP in fp64 over the same bf16 inputs: each 8-bit operand is half a step (1 / 254 of its row's
    # largest) off at most; over random rows that is well under 5 % of the output's size
    wg, wd = f64(m.gu.dequantize(out_dtype=torch.float32)), f64(m.down.dequantize(out_dtype=torch.float32))
    n = o8.rmsnorm(h, f64(m.gain), EPS)
    full = n @ wg.T
    ref = o8.silu_mul(full[:, :hid], full[:, hid:]) @ wd.T
    assert np.linalg.norm(f64(m.y) - ref) <= 0.05 * np.linalg.norm(ref)


def test_int8_from_compressed_weights():
    """The lossless form taken to 8 bits, next to the lossless product of the same norm."""
    w = workloads.weights("gate", rows=768, cols=1024, seed=12)
    m = uw.CompressedMatrix.from_weights(w, device="cuda:0")
    q8 = uw.Int8Matrix.from_compressed(m)
    wf = products.bf16_to_f32(w.numpy().view(np.uint16))
    q, s = o8.quantize(wf)
    assert np.array_equal(q8.q.cpu().numpy(), q) and np.array_equal(q8.scale.cpu().numpy(), s)
    p8 = uw.Int8Matrix.from_compressed(m.transcode_palette())
    assert torch.equal(p8.q, q8.q) and torch.equal(p8.scale, q8.scale)
    X = rand(4, 1024, torch.bfloat16, 3, loud=False)
    g = torch.ones(1024, dtype=torch.bfloat16, device=DEV)
    n16, n8, ns = torch.empty_like(X), uw.i8_rows(4, 1024), torch.empty(4, device=DEV)
    uw.uw_rmsnorm(X, g, n16)
    uw.uw_rmsnorm(X, g, n8, scale=ns)
    lossless, eight = m.gemm(n16.contiguous()), q8.gemm(n8, ns)
    assert torch.linalg.norm(lossless - eight) <= 0.03 * torch.linalg.norm(lossless)
    m.close()


def test_mlp_in_a_graph_replayed():
    m, other = Mlp(3, 512, 1024), Mlp(40, 256, 640, seed=5)
    m.run()
    other.run()
    torch.cuda.synchronize()
    inputs = [(torch.randn_like(m.x), torch.randn_like(m.r)) for _ in range(4)]
    want = []
    for x, r in inputs:
        m.x.copy_(x)
        m.r.copy_(r)
        m.run()
        want.append((m.y.clone(), m.h.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=side):
        m.run()
    with torch.cuda.graph(g2, stream=side):
        other.run()
    y2 = other.y.clone()
    for (x, r), (y, h) in list(zip(inputs, want)) * 2:
        m.x.copy_(x)
        m.r.copy_(r)
        other.y.zero_()
        g1.replay()
        g2.replay()
        uw.uw_silu_mul(x, r, torch.empty_like(x))  # the program's own eager work between replays
        torch.cuda.synchronize()
        assert torch.equal(m.y, y) and torch.equal(m.h, h) and torch.equal(other.y, y2)


def test_mlp_on_two_streams_at_once():
    a, b = Mlp(4, 512, 2048, seed=1), Mlp(33, 512, 1024, seed=2)
    a.run()
    b.run()
    torch.cuda.synchronize()
    ya, yb = a.y.clone(), b.y.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.y.zero_()
        b.y.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            a.run(stream=s1)
            b.run(stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a.y, ya) and torch.equal(b.y, yb)


def test_refusals_name_the_operand():
    x, y = torch.zeros(4, 64, device=DEV), torch.zeros(4, 64, device=DEV)
    q, s = uw.i8_rows(4, 64), torch.zeros(4, device=DEV)
    for call in (
        lambda: uw.uw_rmsnorm(x, None, y[:3]),
        lambda: uw.uw_rmsnorm(x, None, y[:, ::2]),
        lambda: uw.uw_rmsnorm(x, None, torch.zeros(64, 4, device=DEV).t()),
        lambda: uw.uw_rmsnorm(x, None, q),                                  # no scale
        lambda: uw.uw_rmsnorm(x, None, y, scale=s),                         # nothing to scale
        lambda: uw.uw_rmsnorm(x, None, q, scale=s[:3]),
        lambda: uw.uw_rmsnorm(x, None, q, scale=s.double()),
        lambda: uw.uw_rmsnorm(x, torch.ones(63, device=DEV), y),
        lambda: uw.uw_rmsnorm(x, torch.ones(64), y),                        # gain on the host
        lambda: uw.uw_rmsnorm(x, None, y, residual_out=x),
        lambda: uw.uw_rmsnorm(x, None, y, residual=x, residual_out=x.bfloat16()),
        lambda: uw.uw_rmsnorm(x, None, x[0].expand(4, 64)),                 # rows overlap
        lambda: uw.uw_rmsnorm(x[0], None, y[0]),
        lambda: uw.uw_silu_mul(x, x[:2], y),
        lambda: uw.uw_i8_quantize(x, q, s[:2]),
        lambda: uw.uw_i8_dequantize(q, s, y[:, :60]),
        lambda: uw.uw_i8_gemm(q, s, q[:, :60], s, torch.zeros(4, 4, device=DEV)),
        lambda: uw.uw_i8_gemm(q, s, q, s, torch.zeros(4, 5, device=DEV)),
        lambda: uw.uw_i8_gemm(q, s, q, s[:1], torch.zeros(4, 4, device=DEV)),
        lambda: uw.uw_i8_gemm(q, s, q, s, torch.zeros(4, 4, device=DEV), bias=s[:3]),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: uw.uw_silu_mul(x, x.bfloat16(), y),
        lambda: uw.uw_rmsnorm(x.half(), None, y),
        lambda: uw.uw_rmsnorm(x, None, y.half()),
        lambda: uw.uw_i8_quantize(x, y, s),
        lambda: uw.uw_i8_dequantize(x, s, y),
        lambda: uw.uw_i8_gemm(x, s, q, s, torch.zeros(4, 4, device=DEV)),
        lambda: uw.uw_i8_gemm(q, s, x, s, torch.zeros(4, 4, device=DEV)),
    ):
        with pytest.raises(TypeError):
            call()
    for call in (
        lambda: uw.uw_rmsnorm(x, None, y, stream="s"),
        lambda: uw.uw_rmsnorm(x, None, y, eps="e"),
        lambda: uw.uw_rmsnorm([1.0], None, y),
    ):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(uw.UwError):
        uw.uw_rmsnorm(x, None, y, eps=0.0)
    with pytest.raises(uw.UwError):
        uw.uw_i8_gemm_shaped(q, s, q, s, torch.zeros(4, 4, device=DEV), 1 << 40)
    raw = torch.cuda.current_stream().cuda_stream
    uw.uw_rmsnorm(x, None, y, stream=raw)
    uw.uw_rmsnorm(x[:0], None, y[:0])  # no rows: nothing to do
    uw.uw_i8_gemm(q, s, q[:0], s[:0], torch.zeros(0, 4, device=DEV))


# -- defined to the bit ----------------------------------------------------------

@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("b,rows,cols", [(1, 64, 256), (33, 100, 300), (70, 257, 1025)])
def test_gemm_bias_to_the_bit_in_every_shape(b, rows, cols, out):
    """The sum, the scaling and the bias are rounded one after the other, in fp32, whichever shape runs."""
    W, ws = rand_i8(rows, cols, 11)
    X, xs = rand_i8(b, cols, 12)
    bias = torch.randn(rows, device=DEV, generator=torch.Generator(device=DEV).manual_seed(13)) * 1000
    sums = (X.cpu().numpy().astype(np.int64) @ W.cpu().numpy().astype(np.int64).T).astype(np.float32)
    step = xs.cpu().numpy()[:, None] * ws.cpu().numpy()[None, :]
    y = sums * step + bias.cpu().numpy()[None, :]
    assert y.dtype == np.float32
    want = torch.from_numpy(y).to(DT[out])
    for shape in range(uw.uw_i8_gemm_shape_count()):
        for ypad in (0, 5):  # whole lines or not
            Y, _ = inside(b, rows, DT[out], ypad + (-rows % 64 if ypad == 0 else 0))
            if shape:
                uw.uw_i8_gemm_shaped(W, ws, X, xs, Y, shape, bias=bias)
            else:
                uw.uw_i8_gemm(W, ws, X, xs, Y, bias=bias)
            got = Y.cpu()
            assert torch.equal(got, want), f"shape {shape}: {(got != want).sum()} of {want.numel()} differ"
    # operands off 16-byte boundaries
    W1, _ = inside(rows, cols, torch.int8, 1, 3)
    W1.copy_(W)
    Y = torch.empty(b, rows, dtype=DT[out], device=DEV)
    uw.uw_i8_gemm(W1, ws, X, xs, Y, bias=bias)
    assert torch.equal(Y.cpu(), want)


# -- outputs over inputs -----------------------------------------------------------

@pytest.mark.parametrize("cols", [96, 4096, 34000])
def test_norm_over_the_residual(cols):
    """y into the residual, h not kept or kept elsewhere."""
    for dt in (torch.bfloat16, torch.float32):
        X, R = rand(3, cols, dt, 1, pad=8), rand(3, cols, dt, 2, pad=3)
        Y0, H0 = torch.empty(3, cols, dtype=dt, device=DEV), torch.empty(3, cols, dtype=dt, device=DEV)
        uw.uw_rmsnorm(X, None, Y0, residual=R, residual_out=H0)
        for keep in (None, "apart", "x"):
            R1, _ = inside(3, cols, dt, 3)
            R1.copy_(R)
            X1 = X.clone()
            H = None if keep is None else X1 if keep == "x" else torch.empty_like(H0)
            uw.uw_rmsnorm(X1, None, R1, residual=R1, residual_out=H)
            assert torch.equal(R1, Y0) and (H is None or torch.equal(H, H0))


def test_rows_between_the_rows_of_another_operand():
    GU = rand(5, 2 * 700, torch.bfloat16, 4)
    G, V = GU[:, :700], GU[:, 700:]
    Y = torch.empty(5, 700, dtype=torch.bfloat16, device=DEV)
    uw.uw_silu_mul(G, V, Y)
    keep = V.clone()
    uw.uw_silu_mul(G, V, G)  # the gate's half in place, the other half beside it
    assert torch.equal(G, Y) and torch.equal(V, keep)
    # every second row read, every fourth written
    B = rand(16, 300, torch.float32, 5)
    X, Y = B[0:8:2], B[1:16:4]
    want = torch.empty(4, 300, device=DEV)
    uw.uw_rmsnorm(X.clone(), None, want)
    rest = B[2:16:4].clone()
    uw.uw_rmsnorm(X, None, Y)
    assert torch.equal(Y, want) and torch.equal(B[2:16:4], rest)


def test_overlaps_are_refused():
    x = torch.zeros(4, 64, device=DEV)
    s = torch.zeros(4, device=DEV)
    q = x.view(torch.int8)  # rows of 256 integers over x
    for call in (
        lambda: uw.uw_rmsnorm(x[:3], None, x[1:]),
        lambda: uw.uw_rmsnorm(x.clone(), None, q[:, :64], scale=s, residual=x),
        lambda: uw.uw_rmsnorm(x.clone(), None, torch.zeros_like(x), residual=x[:, :64], residual_out=x.view(-1)[1:].as_strided((4, 64), (63, 1))),
        lambda: uw.uw_silu_mul(x[:, :32], x[:, 32:], x[:, 16:48]),
        lambda: uw.uw_i8_quantize(x, q[:, :64], s),
        lambda: uw.uw_i8_dequantize(q[:, :64], s, x),
        lambda: uw.uw_i8_gemm(q[:, :64], s, torch.zeros(4, 64, dtype=torch.int8, device=DEV), s.clone(), x[:, :4]),
    ):
        with pytest.raises((uw.UwError, ValueError)):
            call()
    assert not x.any()


# -- outputs of calls on another stream ----------------------------------------------

def test_outputs_belong_to_the_stream_that_writes_them():
    """An output that is not passed in takes no block of the current stream's, and goes back to the other's."""
    c = uw.CompressedMatrix.from_weights(workloads.weights("gate", rows=768, cols=1024, seed=12), device="cuda:0")
    p = c.transcode_palette(attach=False)
    m = uw.Int8Matrix.from_compressed(c)
    q, qs = rand_i8(37, 1024, 4)
    x = torch.randn(37, 1024, device=DEV).bfloat16()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls = {
        "int8 gemm": lambda s: m.gemm(q, qs, stream=s), "dequantize": lambda s: m.dequantize(stream=s),
        "gemm": lambda s: c.gemm(x[:4], stream=s), "gemv": lambda s: c.gemv(x[0], stream=s),
        "decompress": lambda s: c.decompress(stream=s), "palette gemm": lambda s: p.gemm(x[:4], stream=s),
        "palette gemv": lambda s: p.gemv(x[0], stream=s), "palette decompress": lambda s: p.decompress(stream=s),
    }
    for name, call in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        size, dtype = want.shape, want.dtype
        for stream in (side, side.cuda_stream):
            mine = torch.empty(size, dtype=dtype, device=DEV)  # a block that goes back to the current stream
            at = mine.data_ptr()
            del mine
            got = call(stream)
            assert got.data_ptr() != at, name
            side.synchronize()
            assert torch.equal(got, want), name
            at = got.data_ptr()
            del got
            mine = torch.empty(size, dtype=dtype, device=DEV)
            assert mine.data_ptr() != at, name
            del mine
    with pytest.raises(TypeError):
        m.gemm(q, qs, stream="s")
    c.close()


# -- long sums ---------------------------------------------------------------------------

@pytest.mark.parametrize("value,cols", [(1.2, (1 << 24) + 5), (1.0001, (1 << 22) + 8), (1.37, 1 << 20)])
def test_norm_of_long_rows_of_equal_values(value, cols):
    """Equal squares: every addition of a long chain rounds the same way, so a chain in fp32 shows."""
    X = torch.full((1, cols), value, device=DEV)
    x = float(X[0, 0])
    Y, Q, s = torch.empty_like(X), uw.i8_rows(1, cols), torch.empty(1, device=DEV)
    uw.uw_rmsnorm(X, None, Y, eps=EPS)
    want = x / np.sqrt(x * x + float(np.float32(EPS)))
    for at in (0, cols // 2, cols - 1):
        assert abs(float(Y[0, at]) - want) <= 32 * U * want
    uw.uw_rmsnorm(X, None, Q, scale=s, eps=EPS)
    assert (Q == 127).all() and abs(127 * float(s[0]) - want) <= 32 * U * want


# -- the activation far below zero ------------------------------------------------------------

@pytest.mark.parametrize("x,out", list(itertools.product(("bf16", "f32"), ("f32", "bf16", "i8"))))
@pytest.mark.parametrize("cols", [400, 14336, 40000])
def test_silu_far_below_zero(cols, x, out):
    """exp(-g) near and past the fp32 range, next to values of u that bring the product back into it."""
    gen = torch.Generator().manual_seed(cols)
    G = -80 - 140 * torch.rand(6, cols, generator=gen)
    G[:, ::7] = torch.randn(6, len(range(0, cols, 7)), generator=gen)
    G[0, :5] = torch.tensor([-87.0, -87.25, -88.0, -88.75, -126.0])
    scale = torch.tensor([1.0, 1e3, 1e20, 1e30, 3e38, -3e38])[:, None]
    V = scale * (0.5 + 0.5 * torch.rand(6, cols, generator=gen))
    V[:, ::7] = torch.randn(6, len(range(0, cols, 7)), generator=gen) * 1e-30
    G, V = G.to(DT[x]).to(DEV), V.to(DT[x]).to(DEV)
    p = o8.silu_mul(f64(G), f64(V))
    tiny = 2.0 ** -149  # one step of a denormal number
    if out == "i8":
        Q, s = uw.i8_rows(6, cols), torch.empty(6, device=DEV)
        uw.uw_silu_mul(G, V, Q, scale=s)
        step = np.maximum(np.abs(p).max(axis=1) / 127, 2.0 ** -126)
        check(s, step, 10 * U, torch.float32, "scale", tiny)
        off = np.abs(Q.cpu().numpy().astype(np.float64) - p / step[:, None])
        assert (off <= 0.5 + 127 * 20 * U + 2 * tiny / step[:, None]).all(), off.max()
    else:
        Y = torch.empty(6, cols, dtype=DT[out], device=DEV)
        uw.uw_silu_mul(G, V, Y)
        check(Y, p, 8 * U, DT[out], f"silu {x} {out}", tiny if out == "f32" else 2.0 ** -133)


def test_silu_at_the_ends_of_the_range():
    inf = float("inf")
    G = torch.tensor([[-3e38, -1e5, -301.0, -inf, -90.0, -90.0, -inf, -3e38]], device=DEV)
    V = torch.tensor([[3e38, -3e38, 1.0, 1.0, inf, -inf, inf, 0.0]], device=DEV)
    Y = torch.empty_like(G)
    uw.uw_silu_mul(G, V, Y)
    y = Y.cpu().numpy()[0]
    assert (y[:3] == 0).all() and np.isnan(y[3]) and y[4] == -inf and y[5] == inf and np.isnan(y[6]) and y[7] == 0


# -- more rows than a launch takes ---------------------------------------------------------

def test_rows_past_the_bands_of_each_operator():
    """Rows on both sides of the limit of a launch: 2^24 - 1 for silu and dequantize, 2^21 for the others."""
    rows, edge = (1 << 24) + 9, (1 << 24) - 1
    gen = torch.Generator(device=DEV).manual_seed(2)
    G = torch.randn(rows, 8, device=DEV, generator=gen).bfloat16()
    V = torch.randn(rows, 8, device=DEV, generator=gen).bfloat16()
    Y = torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV)
    uw.uw_silu_mul(G, V, Y)
    for at in (slice(0, 5), slice(edge - 4, edge + 4), slice(rows - 5, rows)):
        check(Y[at], o8.silu_mul(f64(G[at]), f64(V[at])), 8 * U, torch.bfloat16, "silu", 2.0 ** -118)
    del Y
    Q = torch.randint(-127, 128, (rows, 8), dtype=torch.int8, device=DEV, generator=gen)
    s = torch.rand(rows, device=DEV, generator=gen)
    Y = torch.empty(rows, 8, device=DEV)
    uw.uw_i8_dequantize(Q, s, Y)
    assert torch.equal(Y, Q.float() * s[:, None])
    rows, edge = (1 << 21) + 9, 1 << 21
    del Y, Q, s
    G, V = G[:rows].clone(), V[:rows].clone()
    for out in ("bf16", "i8"):
        H = torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV)
        Y = torch.zeros(rows, 8, dtype=DT[out], device=DEV)
        s = torch.zeros(rows, device=DEV)
        uw.uw_rmsnorm(G, None, Y, scale=s if out == "i8" else None, residual=V, residual_out=H)
        S = torch.zeros(rows, device=DEV)
        A = torch.zeros(rows, 8, dtype=torch.int8, device=DEV)
        uw.uw_silu_mul(G, V, A, scale=S)
        for at in (slice(0, 5), slice(edge - 4, edge + 4), slice(rows - 5, rows)):
            h = o8.norm_h(f64(G[at]), f64(V[at]), True)
            assert np.array_equal(f64(H[at]), h)
            if out == "i8":
                q, step = o8.quantize(h.astype(np.float32))
                assert np.array_equal(Y[at].cpu().numpy(), q)
                check(s[at], step * o8.rstd(h, EPS), 32 * U, torch.float32, "scale")
            else:
                check(Y[at], o8.rmsnorm(h, None, EPS), 32 * U, torch.bfloat16, "norm")
            p = o8.silu_mul(f64(G[at]), f64(V[at]))
            assert (np.abs(f64(A[at]) * f64(S[at])[:, None] - p) <= f64(S[at])[:, None] * (0.5 + 127 * 20 * U)).all()


# -- slices whose workgroups start inside the row --------------------------------------------

@pytest.mark.parametrize("shape", [0, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("cols,ld", [(4096, 4096), (4090, 4096), (4001, 4096), (257, 4096), (100, 4096), (8190, 8192), (4097, 12288)])
def test_gemm_slices_at_strides_of_4_kb(cols, ld, shape):
    """The starts wrap around the end of the row, whose last block is masked wherever in the order it comes."""
    rows = 1300
    W, ws = rand_i8(rows, cols, 21, pad=ld - cols)
    for b in (1, 17, 40):
        X, xs = rand_i8(b, cols, 22, pad=ld - cols)
        Y = torch.empty(b, rows, device=DEV)
        if shape:
            uw.uw_i8_gemm_shaped(W, ws, X, xs, Y, shape)
        else:
            uw.uw_i8_gemm(W, ws, X, xs, Y)
        sums = (X.cpu().numpy().astype(np.float64) @ W.cpu().numpy().astype(np.float64).T).astype(np.float32)
        want = sums * (xs.cpu().numpy()[:, None] * ws.cpu().numpy()[None, :])
        assert np.array_equal(Y.cpu().numpy(), want), f"b={b}"


# -- the measured cases ---------------------------------------------------------------------

def measured_cases():
    from perf import operators as ops
    rng = random.Random(17)
    return ops.listed() + [dict(ops.draw(rng), name=f"drawn {i}") for i in range(24)]


@pytest.mark.parametrize("case", measured_cases(), ids=lambda c: c["name"])
def test_measured_cases_against_their_definition(case, monkeypatch):
    """The calls of perf/operators.py, as they are timed, against its definition in 64 bits.  An integer at a tie may go
    either way there (the definition in fp32 is checked to the bit above), so 8-bit values may be one step off."""
    from perf import operators as ops
    monkeypatch.setattr(ops, "own", True)
    _say(f"case {case}")
    state = ops.prepare(case, 5)
    got, ref = ops.run(state), ops.exact(case, 5)
    if case["op"] == "gemm":
        size = ref.abs() + (0 if state["bias"] is None else state["bias"].double().abs())
        lim = 5 * U * size + (HALF[got.dtype] if got.dtype == torch.bfloat16 else 0) * ref.abs()
        assert got.shape == ref.shape and bool(((got.double() - ref).abs() <= lim).all())
        return
    kept, y = got[0], got[1].double()
    assert (kept is None) == (ref[0] is None) and (kept is None or torch.equal(kept.double(), ref[0]))
    assert y.shape == ref[1].shape
    if case["op"] == "mlp":
        # each 8-bit operand is half a step off at most on either side; the rest is as in test_mlp_together
        assert torch.linalg.norm(y - ref[1]) <= 0.05 * torch.linalg.norm(ref[1])
    elif len(got) == 3:
        step = ref[2].unsqueeze(1)
        assert bool(((got[2].double() - ref[2]).abs() <= 40 * U * ref[2]).all())
        assert bool(((y - ref[1]).abs() <= 1.001 * step + 1.01 * 2.0 ** -8 * ref[1].abs()).all())
    else:
        half = HALF[got[1].dtype] if got[1].dtype == torch.bfloat16 else 0
        assert bool(((y - ref[1]).abs() <= (32 * U * (1 + half) + half) * ref[1].abs() + 2.0 ** -126).all())
