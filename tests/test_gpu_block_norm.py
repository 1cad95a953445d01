"""The join of two blocks (uw_block_norm) on the GPU against the fp64 oracle.

Tolerances, u = 2^-24 (half a step of fp32): the first norm's root 20 u and its
mean, reciprocal and products 6 u (the norm's derivation in test_gpu_int8.py),
the gate, its scale and two products 4 u: 30 u of the branch's part of h; the
sum one rounding, then the residual's type.  y is checked from h as the kernel
kept it, as the norm is: 32 u.  Integers to the bit.
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import int4 as o4
from oracle import int8 as o8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_canonical_amd as uw  # noqa: E402
from tests.test_gpu_int8 import DEV, DT, EPS, HALF, NORM_COLS, U, check, f64, inside, rand, special_rows  # noqa: E402


def vector(cols, kind, seed):
    if kind == "none":
        return None
    return (0.7 + 0.4 * torch.randn(cols, generator=torch.Generator().manual_seed(seed))).to(DT[kind]).to(DEV)


def check_h(H, ref, part, what):
    half = HALF[H.dtype] if H.dtype != torch.float32 else 0.0
    # under 2^-126 a step no longer shrinks with the value: half of it is 2^-134 in bf16 (8 significant bits of 2^-126), 2^-150 in
    # fp32, of which the few roundings on the way to h take up to 1e-44 together
    lim = 30 * U * np.abs(part) * (1 + half) + (half + 2 * U) * np.abs(ref) + 1e-44 + (2.0 ** -134 if half else 0.0)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(f64(H)), np.isnan(ref)), what
    over = (np.abs(f64(H) - ref) > lim) & fine
    assert not over.any(), f"{what}: {over.sum()} of {over.size} off"


def run(b, cols, x, res, post, gate, gain, out, pad=0, shift=0, seed=1, branch=1.0, keep=1.0, eps=EPS, post_eps=None, X=None, R=None):
    """post: None (no norm after the block), "none" (no gain) or a type; gate: "none", a type, or a type and "*" (a row per token)."""
    X = rand(b, cols, DT[x], seed, pad, shift) if X is None else X
    R = rand(b, cols, DT[res], seed + 1, pad, shift) if R is None else R
    pg = None if post is None else vector(cols, post, seed + 2)
    gv = vector(cols, gain, seed + 3) if out != "none" else None
    if gate.endswith("*"):
        gt = rand(b, cols, DT[gate[:-1]], seed + 4, pad, shift, loud=False)
    else:
        gt = vector(cols, gate, seed + 4)
    H, h_ok = inside(b, cols, DT[res], pad, shift)
    Y, y_ok = inside(b, cols, DT[out], pad, shift) if out != "none" else (None, lambda: True)
    scale = torch.full((b + 2,), 7.0, device=DEV)
    sc = scale[1: b + 1] if out == "i8" else None
    call = dict(post_gain=pg, gate=gt, gain=gv, Y=Y, scale=sc, post_norm=post is not None, block_scale=branch, residual_scale=keep,
                eps=eps, post_eps=post_eps)
    uw.uw_block_norm(X, R, residual_out=H, **call)
    torch.cuda.synchronize()
    what = f"b={b} cols={cols} x={x} res={res} post={post} gate={gate} gain={gain} out={out} pad={pad} shift={shift}"
    ref, part = o4.join(f64(X), f64(R), post is not None, None if pg is None else f64(pg), eps if post_eps is None else post_eps,
                        None if gt is None else f64(gt), branch, keep)
    check_h(H, ref, part, what + ": h")
    if out != "none":
        h, g = f64(H), None if gv is None else f64(gv)
        if out == "i8":
            q, s = o8.quantize(h.astype(np.float32) if g is None else h.astype(np.float32) * g.astype(np.float32))
            assert np.array_equal(Y.cpu().numpy(), q), f"{what}: {(Y.cpu().numpy() != q).sum()} integers differ"
            check(sc, s.astype(np.float64) * o8.rstd(h, eps), 32 * U, torch.float32, what + ": scale")
            assert scale[0] == 7 and scale[-1] == 7
        else:
            check(Y, o8.rmsnorm(h, g, eps), 32 * U, DT[out], what)
        # h not kept: the same y
        Z = torch.empty_like(Y)
        z = None if sc is None else torch.empty_like(sc)
        uw.uw_block_norm(X, R, **{**call, "Y": Z, "scale": z})
        assert torch.equal(Y, Z) and (sc is None or torch.equal(sc, z)), what + ": h not kept"
        assert y_ok(), what + ": wrote outside Y"
    assert h_ok(), what + ": wrote outside h"


@pytest.mark.parametrize("cols", NORM_COLS)
def test_widths(cols):
    kinds = (("bf16", "bf16", "bf16", "bf16", "bf16", "bf16"), ("bf16", "f32", "bf16", "bf16*", "bf16", "bf16"),
             ("f32", "bf16", None, "none", "f32", "i8"), ("f32", "f32", "f32", "f32*", "none", "f32"),
             ("bf16", "bf16", "none", "f32", "bf16", "none"), ("bf16", "f32", "f32", "bf16", "f32", "i8"))
    for b, kind in zip((1, 3, 5, 2, 4, 1), kinds):
        run(b, cols, *kind, seed=cols, branch=0.5, keep=0.875)


@pytest.mark.parametrize("x,res,out", list(itertools.product(("bf16", "f32"), ("bf16", "f32"), ("i8", "bf16", "f32", "none"))))
def test_types(x, res, out):
    for post, gate, gain in itertools.product((None, "none", "bf16", "f32"), ("none", "bf16", "f32*"), ("none", "bf16", "f32")):
        run(3, 777, x, res, post, gate, gain, out, seed=5)
    run(2, 4096, x, res, "bf16", "f32", "bf16", out, pad=8, seed=6)


@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 1), (5, 3), (16, 7)])
@pytest.mark.parametrize("cols", [5, 500, 1333, 4097, 9001, 33001])
def test_strides_and_offsets(cols, pad, shift):
    run(4, cols, "bf16", "bf16", "bf16", "bf16*", "bf16", "i8", pad, shift)
    run(4, cols, "f32", "bf16", "f32", "f32*", "bf16", "bf16", pad, shift, branch=-1.5)
    run(4, cols, "bf16", "f32", None, "bf16", "f32", "f32", pad, shift, keep=0.25)


def test_many_rows():
    run(1111, 4096, "bf16", "bf16", "bf16", "bf16", "bf16", "i8")
    run(2049, 96, "bf16", "f32", "bf16", "bf16*", "bf16", "bf16")
    # streams of over 16 MiB
    run(2100, 4096, "bf16", "bf16", "bf16", "bf16", "bf16", "bf16")
    run(1030, 4101, "bf16", "f32", "bf16", "bf16*", "bf16", "bf16", pad=3, shift=1)
    run(140, 33000, "f32", "f32", "f32", "f32", "f32", "f32")


def test_scales_and_eps():
    for branch, keep in ((0.0, 1.0), (1.0, 0.0), (0.0, 0.0), (-2.0, 0.1)):
        run(3, 500, "bf16", "f32", "bf16", "bf16", "bf16", "f32", branch=branch, keep=keep)
    run(3, 500, "bf16", "f32", "bf16", "bf16", "bf16", "f32", eps=0.5, post_eps=3.0)
    run(3, 500, "f32", "f32", "none", "none", "none", "f32", eps=1e-30, post_eps=1e-12)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 33000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_rows(cols, dtype):
    """Zeros, tiny and loud values, infinities and NaN in the block's output and in the residual."""
    S = special_rows(cols, dtype)
    C = rand(9, cols, dtype, 2)
    name = "bf16" if dtype == torch.bfloat16 else "f32"
    with np.errstate(all="ignore"):
        for X, R in ((S, C), (C, S), (S, S.clone())):
            for out in ("f32", "i8"):
                H, Y = torch.empty_like(R), torch.empty(9, cols, dtype=DT[out], device=DEV)
                s = torch.empty(9, device=DEV) if out == "i8" else None
                uw.uw_block_norm(X, R, residual_out=H, Y=Y, scale=s, gate=vector(cols, "bf16", 5))
                ref, part = o4.join(f64(X), f64(R), True, None, EPS, f64(vector(cols, "bf16", 5)), 1.0, 1.0)
                check_h(H, ref, part, "special h")
                h = f64(H)
                fine = np.isfinite(h).all(axis=1)
                if out == "i8":
                    q, sn = o8.quantize(h.astype(np.float32))
                    assert np.array_equal(Y.cpu().numpy(), q)
                    assert np.array_equal(np.isnan(f64(s)), ~fine)
                else:
                    check(Y[torch.from_numpy(fine).to(DEV)], o8.rmsnorm(h[fine], None, EPS), 32 * U, torch.float32, "special y")
                    assert np.isnan(f64(Y)[~fine]).any(axis=1).all()
    run(9, cols, name, name, None, "none", "none", "f32", X=C, R=rand(9, cols, dtype, 7))


def test_squares_past_fp32():
    X, R = torch.full((2, 300), 3e38, device=DEV), torch.ones(2, 300, device=DEV)
    X[1] = 1.0
    H, Y = torch.empty(2, 300, device=DEV), torch.empty(2, 300, device=DEV)
    uw.uw_block_norm(X, R, residual_out=H, Y=Y)
    assert (H[0] == 1).all() and torch.allclose(H[1], torch.full_like(H[1], 2.0), rtol=1e-4)
    uw.uw_block_norm(X, R, residual_out=H, Y=Y, post_norm=False)
    assert (H[0] == X[0]).all() and (Y[0] == 0).all() and (Y[1] > 0.99).all()


@pytest.mark.parametrize("cols", [96, 4096, 5003, 34000])
def test_in_place(cols):
    for dt in (torch.bfloat16, torch.float32):
        X, R = rand(3, cols, dt, 1), rand(3, cols, dt, 2)
        kw = dict(post_gain=vector(cols, "bf16", 3), gate=vector(cols, "f32", 4), gain=vector(cols, "f32", 5))
        Y0, H0 = torch.empty(3, cols, dtype=dt, device=DEV), torch.empty(3, cols, dtype=dt, device=DEV)
        uw.uw_block_norm(X, R, residual_out=H0, Y=Y0, **kw)
        R1, Y = R.clone(), torch.empty_like(Y0)  # the stream updated in place
        uw.uw_block_norm(X, R1, residual_out=R1, Y=Y, **kw)
        assert torch.equal(R1, H0) and torch.equal(Y, Y0)
        X1, Y = X.clone(), torch.empty_like(Y0)  # h into X
        uw.uw_block_norm(X1, R, residual_out=X1, Y=Y, **kw)
        assert torch.equal(X1, H0) and torch.equal(Y, Y0)
        X1, R1 = X.clone(), R.clone()  # y into X, h into the residual
        uw.uw_block_norm(X1, R1, residual_out=R1, Y=X1, **kw)
        assert torch.equal(X1, Y0) and torch.equal(R1, H0)
        X1 = X.clone()  # y into X, h not kept
        uw.uw_block_norm(X1, R, Y=X1, **kw)
        assert torch.equal(X1, Y0)
        R1 = R.clone()  # y into the residual, h not kept
        uw.uw_block_norm(X, R1, Y=R1, **kw)
        assert torch.equal(R1, Y0)
        R1 = R.clone()  # no norm behind it
        kw.pop("gain")
        uw.uw_block_norm(X, R1, residual_out=R1, **kw)
        assert torch.equal(R1, H0)
        X1 = X.clone()  # one tensor for block and residual
        uw.uw_block_norm(X1, X1, residual_out=X1, post_norm=False)
        assert torch.equal(X1, (X.float() * 2).to(dt))


def test_agrees_with_rmsnorm_where_nothing_is_gated():
    for cols in (100, 4096, 9000, 40000):
        for x, res, out in itertools.product(("bf16", "f32"), ("bf16", "f32"), ("bf16", "f32", "i8")):
            X, R = rand(5, cols, DT[x], 1), rand(5, cols, DT[res], 2)
            g = vector(cols, "bf16", 3)
            made = []
            for call in (uw.uw_rmsnorm, uw.uw_block_norm):
                H, Y = torch.empty_like(R), torch.empty(5, cols, dtype=DT[out], device=DEV)
                s = torch.empty(5, device=DEV) if out == "i8" else None
                if call is uw.uw_rmsnorm:
                    call(X, g, Y, scale=s, residual=R, residual_out=H)
                else:
                    call(X, R, gain=g, Y=Y, scale=s, residual_out=H, post_norm=False)
                made.append((H, Y, s))
            (h0, y0, s0), (h1, y1, s1) = made
            assert torch.equal(h0, h1) and torch.equal(y0, y1) and (s0 is None or torch.equal(s0, s1)), (cols, x, res, out)


def test_an_expanded_gate_is_a_vector():
    X, R, g = rand(4, 500, torch.bfloat16, 1), rand(4, 500, torch.bfloat16, 2), vector(500, "bf16", 3)
    H = [torch.empty_like(R) for _ in range(3)]
    uw.uw_block_norm(X, R, gate=g, residual_out=H[0])
    uw.uw_block_norm(X, R, gate=g.expand(4, 500), residual_out=H[1])
    uw.uw_block_norm(X, R, gate=g.expand(4, 500).contiguous(), residual_out=H[2])
    assert torch.equal(H[0], H[1]) and torch.equal(H[0], H[2])


def test_more_rows_than_a_launch_holds():
    rows = (1 << 21) + 5
    gen = torch.Generator(device=DEV).manual_seed(1)
    X, R = (torch.randn(rows, 8, device=DEV, generator=gen) for _ in range(2))
    G = torch.rand(rows, 8, device=DEV, generator=gen)
    H, Y, s = torch.empty_like(R), torch.empty(rows, 8, dtype=torch.int8, device=DEV), torch.zeros(rows, device=DEV)
    uw.uw_block_norm(X, R, gate=G, residual_out=H, Y=Y, scale=s)
    for at in (slice(0, 7), slice((1 << 21) - 3, rows)):
        ref, part = o4.join(f64(X[at]), f64(R[at]), True, None, EPS, f64(G[at]), 1.0, 1.0)
        check_h(H[at], ref, part, "band")
        q, sn = o8.quantize(f64(H[at]).astype(np.float32))
        assert np.array_equal(Y[at].cpu().numpy(), q)
        check(s[at], sn * o8.rstd(f64(H[at]), EPS), 32 * U, torch.float32, "band scale")


def test_refusals_name_the_operand():
    x, y = torch.zeros(4, 64, device=DEV), torch.zeros(4, 64, device=DEV)
    r, h, v = torch.zeros(4, 64, device=DEV), torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    q, s = torch.zeros(4, 64, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV)
    for call in (
        lambda: uw.uw_block_norm(x, r),                                       # nothing to write
        lambda: uw.uw_block_norm(x, r[:3], Y=y),
        lambda: uw.uw_block_norm(x, r, Y=y[:, ::2]),
        lambda: uw.uw_block_norm(x, r, Y=q),                                  # no scale
        lambda: uw.uw_block_norm(x, r, Y=y, scale=s),                         # nothing to scale
        lambda: uw.uw_block_norm(x, r, residual_out=h, scale=s),
        lambda: uw.uw_block_norm(x, r, residual_out=h, gain=v),               # a gain without Y
        lambda: uw.uw_block_norm(x, r, Y=y, post_gain=v[:60]),
        lambda: uw.uw_block_norm(x, r, Y=y, gain=v.cpu()),
        lambda: uw.uw_block_norm(x, r, Y=y, gate=v[:60]),
        lambda: uw.uw_block_norm(x, r, Y=y, gate=torch.ones(3, 64, device=DEV)),
        lambda: uw.uw_block_norm(x, r, Y=y, gate=torch.ones(64, 4, device=DEV).t()),
        lambda: uw.uw_block_norm(x, r, residual_out=h.bfloat16()),
        lambda: uw.uw_block_norm(x, r, residual_out=x[0].expand(4, 64)),      # rows overlap
        lambda: uw.uw_block_norm(x[0], r[0], Y=y[0]),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: uw.uw_block_norm(x.half(), r, Y=y),
        lambda: uw.uw_block_norm(x, r.half(), Y=y),
        lambda: uw.uw_block_norm(x, r, Y=y.half()),
        lambda: uw.uw_block_norm(x, r, Y=y, gate=v.half()),
        lambda: uw.uw_block_norm(x, r, Y=y, eps="e"),
        lambda: uw.uw_block_norm(x, r, Y=y, block_scale="b"),
        lambda: uw.uw_block_norm(x, None, Y=y),
        lambda: uw.uw_block_norm(x, r, Y=y, stream="s"),
    ):
        with pytest.raises(TypeError):
            call()
    for k in (dict(eps=0.0), dict(post_eps=-1.0), dict(block_scale=float("nan")), dict(residual_scale=float("inf")),
              dict(post_norm=False, post_gain=v), dict(Y=x, residual_out=x)):
        with pytest.raises(uw.UwError):
            uw.uw_block_norm(x, r, **{"Y": y, **k})
