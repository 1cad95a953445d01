"""4-bit weights on the GPU against the fp64 oracle.

Tolerances, u = 2^-24 (half a step of fp32) and 2^-8 half a step of bf16:

  integers, scales, offsets   to the bit (the definition rounds every step in fp32).
  values back                 to the bit as well: one fp32 product, one sum, one rounding to Y's type.
  product, whole numbers      x whole numbers up to 4, scales and offsets powers of two from 1/2 to 2, so that a group's sums
                              are whole numbers under 2^14 and every term and partial sum of the rest a multiple of 1/16
                              (of an offset: 1/8 of half of one) under 2^19: all are exact in fp32, whatever the order.
  product, any values         a result is the sum over n = cols columns of the terms (q + 8) x s, -8 x s (and m x), whose
                              magnitudes add up to the mass; no order of summation lets a term pass more than 2 cols +
                              groups + 16 additions and 4 roundings, each at most 2 u (the matrix cores' additions may
                              truncate) of a partial sum that the mass bounds: 2 u (2 cols + groups + 20) mass.
                              That holds for the worst signs; roundings of random terms add as their root, and the
                              root mean square of the error is checked against 2 u sqrt(2 cols + groups + 20) of the mass's too.
"""
import itertools
import random
import sys

import numpy as np
import pytest
import torch

import workloads
from oracle import int4 as o4
from oracle import int8 as o8
from oracle import products

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_canonical_amd as uw  # noqa: E402
from tests.test_gpu_int8 import DEV, DT, EPS, U, check, f64, inside, rand  # noqa: E402

SHAPES = range(uw.uw_i4_gemm_shape_count())  # 0: the automatic choice


def _say(msg):
    print(f"[gpu-int4] {msg}", flush=True)
    sys.stdout.flush()


def packed_inside(rows, cols, pad=0):
    """Packed rows with `pad` more 16-byte words between them, in a buffer of 0x5A; (view, check of all other bytes)."""
    ld = ((cols + 31) // 32 + pad) * 16
    raw = torch.full((rows * ld + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    view = raw[32: 32 + rows * ld].view(rows, ld)[:, : (cols + 1) // 2]

    def untouched():
        rest = raw.clone()
        rest[32: 32 + rows * ld].view(rows, ld)[:, : (cols + 1) // 2] = 0x5A
        return bool((rest == 0x5A).all())

    return view, untouched


class Weights:
    """Random 4-bit weights on the device and on the host."""

    def __init__(self, rows, cols, group, affine, st, seed=0, whole=False, pad=0, spad=0):
        rng = np.random.default_rng(seed)
        n = o4.groups(cols, group)
        self.q = rng.integers(-8, 8, (rows, cols)).astype(np.int8)
        if whole:
            s, m = 2.0 ** rng.integers(-1, 2, (n, rows)), 2.0 ** rng.integers(-1, 2, (n, rows)) * rng.choice([-1, 1], (n, rows))
        else:
            s, m = 0.02 * rng.random((n, rows)) + 0.001, 0.02 * rng.standard_normal((n, rows))
        self.W, _ = packed_inside(rows, cols, pad)
        self.W.copy_(torch.from_numpy(o4.pack(self.q)))
        self.scale, self.scale_ok = inside(n, rows, DT[st], pad=spad)
        self.scale.copy_(torch.from_numpy(s))
        self.offset = None
        if affine:
            self.offset, _ = inside(n, rows, DT[st], pad=2 * spad, shift=1)
            self.offset.copy_(torch.from_numpy(m))
        self.s, self.m = f64(self.scale), None if self.offset is None else f64(self.offset)
        self.group, self.rows, self.cols = group, rows, cols

    def run(self, X, Y, shape=0, bias=None, stream=None):
        if shape:
            uw.uw_i4_gemm_shaped(self.W, self.scale, X, Y, shape, self.offset, self.group, bias, stream)
        else:
            uw.uw_i4_gemm(self.W, self.scale, X, Y, self.offset, self.group, bias, stream)

    def ref(self, x, bias=None):
        return o4.gemm(self.q, self.s, self.m, self.group, x, bias)


def tokens(b, cols, seed, whole=False, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-4, 5, (b, cols), generator=g).float() if whole else torch.randn(b, cols, generator=g)
    if not whole and cols > 8:
        x[:, :: max(1, cols // 5)] *= 17
    v, _ = inside(b, cols, torch.bfloat16, pad, shift, fill=0xFF)  # NaN around the rows
    v.copy_(x.bfloat16())
    return v


def run_gemm(b, rows, cols, group, affine, st, out, bias=False, shape=0, whole=False, pad=0, shift=0, seed=1, w=None):
    w = w or Weights(rows, cols, group, affine, st, seed, whole, pad=pad % 3, spad=pad)
    X = tokens(b, cols, seed + 1, whole, pad, shift)
    Y, y_ok = inside(b, rows, DT[out], pad, shift)
    bv = torch.randint(-8, 9, (rows,), generator=torch.Generator().manual_seed(seed)).float().to(DEV) if bias else None
    if shape:
        try:
            w.run(X, Y, shape, bv)
        except uw.UwError as e:
            assert e.status == uw.UW_ERR_UNSUPPORTED
            if not (X.data_ptr() % 16 or (b > 1 and X.stride(0) % 8)):
                assert b > 4  # a shape for few tokens
                return
            # a shape for rows on 16-byte boundaries
            return run_gemm(b, rows, cols, group, affine, st, out, bias, shape, whole, pad + -(cols + pad) % 8, 8 * (shift > 0), seed)
    w.run(X, Y, shape, bv)
    torch.cuda.synchronize()
    what = f"gemm b={b} rows={rows} cols={cols} group={group} affine={affine} st={st} out={out} bias={bias} shape={shape} whole={whole} pad={pad} shift={shift}"
    ref, mass = w.ref(f64(X), None if bv is None else f64(bv))
    got = f64(Y)
    if whole:
        want = ref if out == "f32" else o8.to_bf16(ref)
        assert np.array_equal(got, want), f"{what}: {(got != want).sum()} of {got.size} differ, first at {np.argwhere(got != want)[:3].tolist()}"
    else:
        n = 2 * cols + o4.groups(cols, group) + 20
        half = 0.0 if out == "f32" else 2.0 ** -8
        lim = 2 * U * n * mass + (half + 2 * U) * np.abs(ref)
        over = np.abs(got - ref) > lim
        assert not over.any(), f"{what}: {over.sum()} of {over.size} off, worst {np.max(np.abs(got - ref) / lim):.3g} of the tolerance"
        size = np.sqrt(np.mean(mass ** 2))
        err = np.sqrt(np.mean((got - ref) ** 2))
        assert err <= 2 * U * np.sqrt(n) * size + (half + 2 * U) * np.sqrt(np.mean(ref ** 2)), f"{what}: mean error {err / size:.3g}"
    assert y_ok(), what + ": wrote outside Y"


def takes(w, X, Y, shape):
    """Runs the product; False where the shape is not for so many tokens."""
    try:
        w.run(X, Y, shape)
    except uw.UwError as e:
        assert e.status == uw.UW_ERR_UNSUPPORTED and X.shape[0] > 4
        return False
    return True


WIDTHS = [1, 7, 8, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 160, 192, 255, 256, 257, 384, 511, 512, 640, 1000, 1025, 2048, 4100]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cols", WIDTHS)
def test_gemm_widths(cols, shape):
    for (group, affine), b, rows in zip(itertools.product((32, 64, 128), (False, True)), (1, 2, 16, 17, 5, 3), (1, 15, 16, 33, 64, 70)):
        run_gemm(b, rows, cols, group, affine, "bf16", "f32", shape=shape, whole=True, seed=cols)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("b", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129, 200, 256, 257])
def test_gemm_batches(b, shape):
    for i, (rows, group, affine) in enumerate(((130, 32, True), (257, 128, False), (96, 64, True), (31, 128, True))):
        run_gemm(b, rows, 520, group, affine, ("bf16", "f32")[i % 2], ("f32", "bf16")[i // 2], bias=i % 2 == 1, shape=shape, whole=True, seed=b)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (8, 8), (1, 0), (3, 1), (4, 2), (0, 5), (16, 7)])
def test_gemm_strides_and_offsets(pad, shift, shape):
    for b, rows, cols, group in ((1, 40, 136, 64), (5, 100, 1001, 32), (33, 70, 300, 128), (150, 64, 129, 64)):
        run_gemm(b, rows, cols, group, True, "bf16", "f32", True, shape, True, pad, shift)
        run_gemm(b, rows, cols, group, False, "f32", "bf16", False, shape, True, pad, shift)


@pytest.mark.parametrize("group,affine,st,out", list(itertools.product((32, 64, 128), (False, True), ("bf16", "f32"), ("bf16", "f32"))))
def test_gemm_values(group, affine, st, out):
    for b, rows, cols in ((1, 300, 4100), (16, 129, 2000), (40, 200, 777), (130, 260, 1500)):
        run_gemm(b, rows, cols, group, affine, st, out, bias=True)


@pytest.mark.parametrize("shape", SHAPES)
def test_gemm_shapes_values(shape):
    for b, group, affine in ((3, 128, False), (70, 32, True), (260, 64, True)):
        run_gemm(b, 270, 2200, group, affine, "bf16", "f32", shape=shape)


@pytest.mark.parametrize("b,rows,cols,group,affine", [(1, 14336, 4096, 128, False), (16, 4096, 14336, 64, True), (77, 1000, 4100, 32, True),
                                                      (256, 2048, 4096, 128, False), (1024, 768, 2049, 64, False), (2, 64, 28672, 32, True)])
def test_gemm_full_sizes(b, rows, cols, group, affine):
    _say(f"full size {b} x {rows} x {cols}")
    run_gemm(b, rows, cols, group, affine, "bf16", "bf16")
    run_gemm(b, rows, cols, group, affine, "f32", "f32", whole=True)


def test_gemm_drawn_sizes():
    rng = random.Random(4)
    spread = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    for i in range(40):
        b, rows, cols = spread(1, 700), spread(1, 900), spread(1, 3000)
        _say(f"drawn {i}: {b} x {rows} x {cols}")
        run_gemm(b, rows, cols, rng.choice((32, 64, 128)), rng.random() < 0.5, rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")),
                 rng.random() < 0.5, 0, True, rng.choice((0, 0, 1, 8)), rng.choice((0, 0, 3, 8)), seed=i)


@pytest.mark.parametrize("b,rows,cols,group", [(1, 1, (1 << 21) + 5, 32), (2, 3, (1 << 21) + 40, 128)])
def test_gemm_rows_past_32_bit_offsets(b, rows, cols, group):
    _say(f"rows past 32-bit offsets: {b} x {rows} x {cols}")
    run_gemm(b, rows, cols, group, True, "f32", "f32", bias=True)


@pytest.mark.parametrize("far", ["W", "X", "scale", "offset"])
def test_gemm_strides_past_32_bits(far):
    """One operand at strides whose offsets pass 32 bits (or the bound below them): the same results to the bit of whole numbers."""
    _say(f"strides past 32 bits: {far}")
    w = Weights(40, 250, 32, True, "f32", seed=3, whole=True)
    X = tokens(20, 250, 4, whole=True)
    Y, y_ok = inside(20, 40, torch.float32)
    if far == "W":
        wide = torch.empty_strided((40, 128), (1 << 27, 1), dtype=torch.uint8, device=DEV)[:, :125]  # whole 16-byte words
        wide.copy_(w.W)
        w.W = wide
    elif far == "X":
        wide = torch.empty_strided(X.shape, (1 << 27, 1), dtype=torch.bfloat16, device=DEV)
        wide.copy_(X)
        X = wide
    else:
        wide = torch.empty_strided(w.scale.shape, ((1 << 27) + 4, 1), dtype=torch.float32, device=DEV)
        wide.copy_(getattr(w, far))
        setattr(w, far, wide)
    w.run(X, Y)
    torch.cuda.synchronize()
    assert np.array_equal(f64(Y), w.ref(f64(X))[0]) and y_ok()


def test_gemm_infinities_stay_in_their_token():
    for shape in SHAPES:  # 520 columns: rows on 16-byte boundaries
        for affine, b in itertools.product((False, True), (4, 16, 40)):
            w = Weights(48, 520, 64, affine, "bf16", 3)
            X = tokens(b, 520, 4)
            Y = torch.empty(b, 48, device=DEV)
            if not takes(w, X, Y, shape):
                continue
            clean = Y.clone()
            X[1, 13], X[2, 519], X[b - 1, 200] = float("nan"), float("inf"), float("-inf")
            w.run(X, Y, shape)
            bad = torch.zeros(b, dtype=torch.bool, device=DEV)
            bad[[1, 2, b - 1]] = True
            assert torch.equal(Y[~bad], clean[~bad]) and not torch.isfinite(Y[bad]).any(), f"shape {shape} affine {affine}"


def test_gemm_nan_scales_show_in_their_row_alone():
    w = Weights(40, 300, 64, True, "bf16", 3)
    X = tokens(5, 300, 4)
    Y, Z = torch.empty(5, 40, device=DEV), torch.empty(5, 40, device=DEV)
    w.run(X, Y)
    w.scale[2, 17], w.offset[4, 30] = float("nan"), float("nan")
    w.run(X, Z)
    keep = [i for i in range(40) if i not in (17, 30)]
    assert torch.equal(Y[:, keep], Z[:, keep]) and torch.isnan(Z[:, [17, 30]]).all()


def test_gemm_repeats_to_the_bit_and_rows_do_not_see_each_other():
    w = Weights(333, 1304, 32, True, "f32", 8)
    for shape, b in itertools.product(SHAPES, (3, 11, 37)):
        X = tokens(b, 1304, 9)
        Y, Z = torch.empty(b, 333, device=DEV), torch.empty(b, 333, device=DEV)
        if not takes(w, X, Y, shape):
            continue
        for _ in range(3):
            w.run(X, Z, shape)
            assert torch.equal(Y, Z), shape
        X2 = X.clone()
        X2[1:] = 0
        w.run(X2, Z, shape)
        assert torch.equal(Y[0], Z[0]) and not Z[1:].any(), shape


@pytest.mark.parametrize("rows,cols,x,pad,shift", [
    (1, 1, "f32", 0, 0), (3, 5, "bf16", 1, 1), (37, 1001, "f32", 0, 0), (64, 4096, "bf16", 0, 0), (5, 14336, "bf16", 8, 0),
    (2, 40000, "f32", 3, 1), (1000, 64, "bf16", 0, 0), (300, 513, "bf16", 7, 3), (70, 127, "f32", 0, 2), (129, 2049, "bf16", 0, 0)])
@pytest.mark.parametrize("group,affine,st", list(itertools.product((32, 64, 128), (False, True), ("bf16", "f32"))))
def test_quantize_and_back(rows, cols, x, pad, shift, group, affine, st):
    X = rand(rows, cols, DT[x], 3, pad, shift)
    X[:, cols // 2] *= 3
    Q, q_ok = packed_inside(rows, cols, pad % 3)
    n = o4.groups(cols, group)
    s, s_ok = inside(n, rows, DT[st], pad)
    m, m_ok = inside(n, rows, DT[st], 2 * pad, shift) if affine else (None, lambda: True)
    uw.uw_i4_quantize(X, Q, s, m, group)
    q, sn, mn = o4.quantize(f64(X).astype(np.float32), group, affine, st == "bf16")
    what = f"{rows}x{cols} {x} group={group} affine={affine} st={st}"
    assert np.array_equal(f64(s), sn), what
    assert m is None or np.array_equal(f64(m), mn), what
    got = Q.cpu().numpy()
    assert np.array_equal(got, o4.pack(q)), f"{what}: {(o4.unpack(got, cols) != q).sum()} integers differ"
    for out in ("f32", "bf16"):
        Y, y_ok = inside(rows, cols, DT[out], pad, shift)
        uw.uw_i4_dequantize(Q, s, Y, m, group)
        v = o4.dequantize_f32(q, sn, mn, group).astype(np.float64)
        assert np.array_equal(f64(Y), v if out == "f32" else o8.to_bf16(v)), what
        assert y_ok()
    assert q_ok() and s_ok() and m_ok()


@pytest.mark.parametrize("group,affine,st", list(itertools.product((32, 128), (False, True), ("bf16", "f32"))))
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_quantize_special_groups(group, affine, st, x):
    """Zeros, one loud value, ties, the ends of the range, denormal steps, infinities and NaN."""
    cols = 200
    X = torch.randn(16, cols, generator=torch.Generator().manual_seed(3))
    X[0] = 0
    X[1] *= 1e-30
    X[2] = 0
    X[2, -1] = 3.0
    X[3, cols // 2] = 1e15
    X[4, 0] = float("inf")
    X[5, -1] = float("nan")
    X[6] = float("-inf")
    X[7] = -0.0
    X[8] = 1e-40
    X[9] = torch.arange(cols) % 15 - 7.0  # whole steps and none between
    X[10] = (torch.arange(cols) % 29 - 14.0) / 2  # ties
    X[11] = 3.38e38 * (1 - 2.0 * (torch.arange(cols) % 2))  # the span is past the fp32 range
    X[12] *= 1e-37
    X[13] *= 1e37
    X[14] = 0.7  # nothing but one value
    X[15] = 2.0 ** -126 * (torch.arange(cols) % 16)
    X = X.to(DT[x]).to(DEV)
    Q, _ = packed_inside(16, cols)
    n = o4.groups(cols, group)
    s = torch.empty(n, 16, dtype=DT[st], device=DEV)
    m = torch.empty_like(s) if affine else None
    uw.uw_i4_quantize(X, Q, s, m, group)
    q, sn, mn = o4.quantize(f64(X).astype(np.float32), group, affine, st == "bf16")
    assert np.array_equal(f64(s), sn, equal_nan=True)
    assert m is None or np.array_equal(f64(m), mn, equal_nan=True)
    got = o4.unpack(Q.cpu().numpy(), cols)
    assert np.array_equal(got, q), np.argwhere(got != q)[:5].tolist()


def test_quantize_more_rows_than_a_launch_holds():
    rows = (1 << 24) + 5
    X = torch.randn(rows, 8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).bfloat16()
    Q = torch.zeros(rows, 16, dtype=torch.uint8, device=DEV)[:, :4]
    s = torch.zeros(1, rows, device=DEV)
    uw.uw_i4_quantize(X, Q, s, group=32)
    Y = torch.empty(rows, 8, device=DEV)
    uw.uw_i4_dequantize(Q, s, Y, group=32)
    for at in (slice(0, 7), slice((1 << 24) - 9, rows)):
        q, sn, _ = o4.quantize(f64(X[at]).astype(np.float32), 32, False, False)
        assert np.array_equal(Q[at].cpu().numpy(), o4.pack(q)) and np.array_equal(f64(s[:, at]), sn)
        assert np.array_equal(f64(Y[at]), o4.dequantize_f32(q, sn, None, 32))


class Block:
    """A decoder block's MLP in 4 bits between two joins, with outputs allocated once."""

    def __init__(self, b, cols, hid, seed=1, group=128, affine=False):
        g = torch.Generator().manual_seed(seed)
        mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.gu = uw.Int4Matrix.from_weights((0.05 * mk(2 * hid, cols)).bfloat16().to(DEV), group, affine)
        self.down = uw.Int4Matrix.from_weights((0.05 * mk(cols, hid)).bfloat16().to(DEV), group, affine, torch.float32)
        self.x, self.r = mk(b, cols).bfloat16().to(DEV), mk(b, cols).bfloat16().to(DEV)
        self.gains = [(1 + 0.2 * mk(cols)).bfloat16().to(DEV) for _ in range(4)]
        self.gate = (0.5 + 0.2 * mk(cols)).bfloat16().to(DEV)
        new = lambda n: torch.empty(b, n, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.h, self.n, self.GU, self.a, self.z, self.h2, self.y = new(cols), new(cols), new(2 * hid), new(hid), new(cols), new(cols), new(cols)
        self.hid = hid

    def run(self, stream=None):
        p1, g1, p2, g2 = self.gains
        uw.uw_block_norm(self.x, self.r, p1, self.gate, self.h, g1, self.n, eps=EPS, stream=stream)
        self.gu.gemm(self.n, self.GU, stream=stream)
        uw.uw_silu_mul(self.GU[:, : self.hid], self.GU[:, self.hid:], self.a, stream=stream)
        self.down.gemm(self.a, self.z, stream=stream)
        uw.uw_block_norm(self.z, self.h, p2, self.gate, self.h2, g2, self.y, eps=EPS, stream=stream)


@pytest.mark.parametrize("b,cols,hid,group,affine", [(1, 512, 1024, 128, False), (16, 640, 1000, 32, True), (70, 256, 515, 64, False)])
def test_block_against_the_oracle(b, cols, hid, group, affine):
    m = Block(b, cols, hid, 2, group, affine)
    m.run()
    torch.cuda.synchronize()
    p1, g1, p2, g2 = (f64(g) for g in m.gains)
    bf = torch.bfloat16

    def close(got, ref, part, what):  # the join: 32 u of its terms, then bf16
        lim = 32 * U * (np.abs(part) + np.abs(ref)) + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7)
        assert (np.abs(f64(got) - ref) <= lim).all(), what

    h, part = o4.join(f64(m.x), f64(m.r), True, p1, EPS, f64(m.gate), 1.0, 1.0)
    close(m.h, h, part, "h")
    check(m.n, o8.rmsnorm(f64(m.h), g1, EPS), 32 * U, bf, "norm")
    for w, X, Y in ((m.gu, m.n, m.GU), (m.down, m.a, m.z)):
        q = o4.unpack(w.q.cpu().numpy(), w.cols)
        ref, mass = o4.gemm(q, f64(w.scale), None if w.offset is None else f64(w.offset), w.group, f64(X))
        lim = 2 * U * (2 * w.cols + w.scale.shape[0] + 20) * mass + (2.0 ** -8 + 2 * U) * np.abs(ref)
        assert (np.abs(f64(Y) - ref) <= lim).all()
    got = f64(m.GU)
    check(m.a, o8.silu_mul(got[:, :hid], got[:, hid:]), 8 * U, bf, "silu", 2.0 ** -118 * np.abs(got).max())
    h, part = o4.join(f64(m.z), f64(m.h), True, p2, EPS, f64(m.gate), 1.0, 1.0)
    close(m.h2, h, part, "h2")
    check(m.y, o8.rmsnorm(f64(m.h2), g2, EPS), 32 * U, bf, "y")


def test_block_in_a_graph_replayed():
    m, other = Block(3, 512, 1024), Block(40, 256, 640, seed=5, group=32, affine=True)
    m.run()
    other.run()
    torch.cuda.synchronize()
    inputs = [(torch.randn_like(m.x), torch.randn_like(m.r)) for _ in range(4)]
    want = []
    for x, r in inputs:
        m.x.copy_(x)
        m.r.copy_(r)
        m.run()
        want.append((m.y.clone(), m.h2.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=side):
        m.run()
    with torch.cuda.graph(g2, stream=side):
        other.run()
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
        assert torch.equal(m.y, y) and torch.equal(m.h2, h) and torch.equal(other.y, y2)


def test_block_on_two_streams_at_once():
    a, b = Block(4, 512, 2048, seed=1), Block(33, 512, 1024, seed=2, group=64, affine=True)
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


def test_int4_from_compressed_weights():
    w = workloads.weights("gate", rows=768, cols=1024, seed=12)
    m = uw.CompressedMatrix.from_weights(w, device="cuda:0")
    q4 = uw.Int4Matrix.from_compressed(m, group=64)
    q, s, _ = o4.quantize(products.bf16_to_f32(w.numpy().view(np.uint16)), 64, False, True)
    assert np.array_equal(q4.q.cpu().numpy(), o4.pack(q)) and np.array_equal(f64(q4.scale), s)
    p4 = uw.Int4Matrix.from_compressed(m.transcode_palette(), group=64, affine=True, scale_dtype=torch.float32)
    X = rand(4, 1024, torch.bfloat16, 3, loud=False)
    lossless = m.gemm(X.contiguous())
    for four in (q4, p4):
        # half a step of (largest of 64) / 7 off at most, uniform: 0.1 of the weights' size in the mean
        assert torch.linalg.norm(lossless - four.gemm(X)) <= 0.15 * torch.linalg.norm(lossless)
        assert torch.equal(four.gemv(X[1]), four.gemm(X[1:2])[0])
        assert four.dequantize().shape == (768, 1024)
    m.close()


def test_matrix_of_packed_weights_and_slices():
    """Weights as other programs keep them: unsigned nibbles with scales and zero points; rows and columns sliced."""
    rng = np.random.default_rng(5)
    rows, cols, group = 96, 256, 64
    u, z = rng.integers(0, 16, (rows, cols)), rng.integers(0, 16, (cols // group, rows))
    s = (2.0 ** rng.integers(-1, 2, z.shape)).astype(np.float32)
    words = np.zeros((rows, cols // 8), np.int64)
    for e in range(8):
        words |= u[:, e::8] << (4 * e)
    Q = torch.from_numpy(words.astype(np.uint32).view(np.int32)).to(DEV).view(torch.uint8)
    m = uw.Int4Matrix(Q, torch.from_numpy(s).to(DEV), torch.from_numpy((s * (8 - z)).astype(np.float32)).to(DEV), group=group)
    X = tokens(3, cols, 6, whole=True)
    want = f64(X) @ (o4.spread(s, cols, group) * (u - o4.spread(z, cols, group))).T
    assert np.array_equal(f64(m.gemm(X)), want)
    # rows 32 .. 64, and columns 64 .. 192 of them
    part = uw.Int4Matrix(Q[32:64, 32:96], m.scale[1:3, 32:64], m.offset[1:3, 32:64], group=group)
    got = f64(part.gemm(X[:, 64:192]))
    want = f64(X)[:, 64:192] @ (o4.spread(s, cols, group) * (u - o4.spread(z, cols, group)))[32:64, 64:192].T
    assert np.array_equal(got, want)


def test_empty_batches_and_matrices():
    w = Weights(16, 64, 32, False, "f32")
    w.run(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 16, device=DEV))
    uw.uw_block_norm(torch.empty(0, 64, device=DEV), torch.empty(0, 64, device=DEV), Y=torch.empty(0, 64, device=DEV))


def test_refusals_name_the_operand():
    w = Weights(16, 64, 32, True, "f32")
    X, Y = tokens(4, 64, 1), torch.empty(4, 16, device=DEV)
    Q, S, M = w.W, w.scale, w.offset
    tight = torch.zeros(16 * 48 - 10, dtype=torch.uint8, device=DEV)
    for call in (
        lambda: uw.uw_i4_gemm(Q, S, X, Y, M, group=16),
        lambda: uw.uw_i4_gemm(Q, S[:1], X, Y, M, group=32),
        lambda: uw.uw_i4_gemm(Q, S, X, Y, M[:, :8], group=32),
        lambda: uw.uw_i4_gemm(Q, S, X, Y, M.bfloat16(), group=32),
        lambda: uw.uw_i4_gemm(Q, S, X, Y[:, :8], M, group=32),
        lambda: uw.uw_i4_gemm(Q, S, X[:, :60], Y, M, group=32),
        lambda: uw.uw_i4_gemm(Q, S, X, Y, M, group=32, bias=torch.zeros(8, device=DEV)),
        lambda: uw.uw_i4_gemm(Q, S, X[0], Y[0], M, group=32),
        lambda: uw.uw_i4_gemm(Q, S, X.t().contiguous().t(), Y, M, group=32),
        lambda: uw.uw_i4_gemm(Q, S.cpu(), X, Y, M, group=32),
        lambda: uw.uw_i4_gemm(torch.zeros(16, 40, dtype=torch.uint8, device=DEV)[:, :32], S, X, Y, M, group=32),  # rows off 16 bytes
        lambda: uw.uw_i4_gemm(torch.zeros(528, dtype=torch.uint8, device=DEV)[8:520].view(16, 32), S, X, Y, M, group=32),
        # 68 columns need 3 words of 16 bytes; the last row's third word is not there
        lambda: uw.uw_i4_gemm(tight.as_strided((16, 34), (48, 1)), torch.ones(3, 16, device=DEV), tokens(4, 68, 1), Y, group=32),
        lambda: uw.uw_i4_dequantize(Q, S, torch.empty(16, 70, device=DEV), M, 32),
        lambda: uw.uw_i4_quantize(torch.zeros(16, 64, device=DEV), Q[:8], S, M, 32),
        lambda: uw.uw_i4_quantize(torch.zeros(16, 64, device=DEV), Q, S[:, :8], M, 32),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: uw.uw_i4_gemm(Q, S, X.float(), Y, M, group=32),
        lambda: uw.uw_i4_gemm(Q, S.half(), X, Y, M, group=32),
        lambda: uw.uw_i4_gemm(Q.char(), S, X, Y, M, group=32),
        lambda: uw.uw_i4_gemm(Q, S, X, Y.half(), M, group=32),
        lambda: uw.uw_i4_gemm(Q, S, X, Y, M, group="g"),
        lambda: uw.uw_i4_gemm(Q, S, X, Y, M, group=32, stream="s"),
        lambda: uw.uw_i4_gemm(Q, None, X, Y, M, group=32),
        lambda: uw.uw_i4_quantize(torch.zeros(16, 64, device=DEV).half(), Q, S, M, 32),
        lambda: uw.uw_i4_dequantize(Q, S, torch.empty(16, 64, device=DEV).half(), M, 32),
    ):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(uw.UwError):
        uw.uw_i4_gemm_shaped(Q, S, X, Y, 1 << 40, M, 32)
    uw.uw_i4_gemm(Q, S, X, Y, M, group=32, stream=torch.cuda.current_stream().cuda_stream)
