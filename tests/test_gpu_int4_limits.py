"""The 4-bit product at the ends of its operands' range: the largest finite tokens, more rows than most shapes hold;
and which shapes refuse which operands.

Tolerance: that of test_gpu_int4.py for any values, 2 u (2 cols + groups + 20) of the mass.  Its count of additions holds
at any magnitude, as long as no sum passes the fp32 range: the terms and their sums are the same up to a power of two.
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import int4 as o4

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_canonical_amd as uw  # noqa: E402
from tests.test_gpu_int4 import SHAPES, WIDTHS, Weights, tokens  # noqa: E402
from tests.test_gpu_int8 import DEV, U, f64, inside  # noqa: E402

LARGEST = (2 - 2.0 ** -7) * 2.0 ** 127  # of bf16
FEW = range(1, 10)  # the shapes that hold up to 16 tokens: direct, token, stream, slices, deep slices


def run(w, X, shape):
    """The product as fp32 values checked against the oracle; False where the shape is not for so many tokens."""
    b = X.shape[0]
    Y, y_ok = inside(b, w.rows, torch.float32)
    try:
        w.run(X, Y, shape)
    except uw.UwError as e:
        assert e.status == uw.UW_ERR_UNSUPPORTED and refuses(shape, b, w.cols, X)
        return False
    ref, mass = w.ref(f64(X))
    got = f64(Y)
    what = f"shape {shape} b={b} group={w.group} affine={w.m is not None}"
    assert (np.abs(ref) < 2.0 ** 127).all(), "the results themselves are in range"
    assert np.isfinite(got).all(), f"{what}: tokens {np.argwhere(~np.isfinite(got).all(axis=1)).ravel().tolist()} are not finite"
    n = 2 * w.cols + o4.groups(w.cols, w.group) + 20
    lim = 2 * U * n * mass + 2 * U * np.abs(ref)
    assert (np.abs(got - ref) <= lim).all(), what
    assert y_ok(), what + ": wrote outside Y"
    return True


def small(w, by):
    """Scales and offsets times `by`, a power of two."""
    w.scale.mul_(by)
    w.s = f64(w.scale)
    if w.offset is not None:
        w.offset.mul_(by)
        w.m = f64(w.offset)
    return w


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("group,affine", list(itertools.product((32, 64, 128), (False, True))))
def test_large_finite_tokens(group, affine, shape):
    """Tokens whose magnitudes add up to just under 2^129 over a group."""
    cols, ran = 520, False
    w = small(Weights(48, cols, group, affine, "bf16", 3), 2.0 ** -8)
    kinds = torch.zeros(5, cols)
    kinds[0] = torch.randn(cols, generator=torch.Generator().manual_seed(4))
    kinds[1] = 1.875 * 2.0 ** 128 / group
    kinds[2, ::group], kinds[2, 3::group] = LARGEST, -LARGEST
    kinds[3, ::group], kinds[3, 5::group] = LARGEST, LARGEST
    kinds[4, 517] = -LARGEST
    for b in (1, 4, 16, 40):
        X, _ = inside(b, cols, torch.bfloat16, 8, 8)  # rows on 16-byte boundaries
        X.copy_(kinds[(torch.arange(b) + 1) % 5].bfloat16())
        ran |= run(w, X, shape)
    assert ran


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("group,affine", list(itertools.product((32, 64, 128), (False, True))))
def test_tiny_tokens(group, affine, shape):
    """Tokens down to 2^-126, whose sums are denormal in 2^-11 of their value.  There a step is 2^-149 whatever the value: each
    of the 2 cols + groups + 20 additions may lose it, times 2^11 and a scale below 1."""
    cols, ran = 520, False
    w = Weights(48, cols, group, affine, "f32", 3)
    assert w.s.max() < 1 and (w.m is None or np.abs(w.m).max() < 1)
    n = 2 * cols + o4.groups(cols, group) + 20
    for b, power in itertools.product((3, 16, 40), (-100, -112, -118, -124)):
        X, _ = inside(b, cols, torch.bfloat16, 8, 8)
        sign = torch.randn(b, cols, generator=torch.Generator().manual_seed(b)).sign()
        X.copy_((sign * (1 + torch.rand(b, cols, generator=torch.Generator().manual_seed(b))) * 2.0 ** power).bfloat16())
        Y, y_ok = inside(b, w.rows, torch.float32)
        try:
            w.run(X, Y, shape)
        except uw.UwError as e:
            assert e.status == uw.UW_ERR_UNSUPPORTED and refuses(shape, b, cols, X)
            continue
        ran = True
        ref, mass = w.ref(f64(X))
        got = f64(Y)
        over = np.abs(got - ref) > 2 * U * n * mass + 2 * U * np.abs(ref) + n * 2.0 ** -138
        assert not over.any() and y_ok(), f"shape {shape} b={b} 2^{power}: {over.sum()} of {over.size} off"
        # not merely zero: the values stand well above that
        assert power < -112 or (got != 0).all()
    assert ran


@pytest.mark.parametrize("shape", FEW)
@pytest.mark.parametrize("group,affine", list(itertools.product((32, 64, 128), (False, True))))
def test_largest_finite_tokens_of_the_shapes_for_few(group, affine, shape):
    """No finite token leaves the range in the sums of these."""
    w = small(Weights(48, 520, group, affine, "f32", 5), 2.0 ** -16)
    for b in (2, 4):
        X = torch.full((b, 520), LARGEST, device=DEV).bfloat16()
        X[1] = -X[1]
        assert run(w, X, shape) and (b != 4 or run(w, X, 0))


@pytest.mark.parametrize("group", [32, 128])
def test_more_rows_than_a_launch_of_the_token_shapes_holds(group):
    """2^28 rows: a shape that holds them is taken.  Whole numbers and powers of two: exact in fp32, whatever the order."""
    rows, cols = 1 << 28, 32
    g = torch.Generator(device=DEV).manual_seed(7)
    W = torch.randint(0, 256, (rows, 16), generator=g, dtype=torch.uint8, device=DEV)
    scale = (2.0 ** torch.randint(-1, 2, (1, rows), generator=g, device=DEV)).bfloat16()
    X = torch.randint(-4, 5, (3, cols), generator=g, device=DEV).bfloat16()
    at = torch.cat([torch.arange(64), torch.randint(0, rows - 5000, (2000,), generator=torch.Generator().manual_seed(1)),
                    torch.arange(rows - 5064, rows - 5000)])
    for n, b in ((rows, 1), (rows - 4096, 1), (rows, 3)):
        rows_at = torch.cat([at, torch.arange(n - 64, n)]).to(DEV)
        q, s = o4.unpack(W[rows_at].cpu().numpy(), cols), f64(scale[:, rows_at])
        Y = torch.full((b, n), float("nan"), device=DEV)
        uw.uw_i4_gemm(W[:n], scale[:, :n], X[:b], Y, group=group)
        assert np.array_equal(f64(Y[:, rows_at]), o4.gemm(q, s, None, group, f64(X[:b]))[0]), (n, b)
        assert not torch.isnan(Y).any()
        del Y


def refuses(shape, b, cols, X):
    """Whether a shape is not for these tokens (at strides and scales within its offsets)."""
    if shape in (2, 3):  # the token kernel
        return b > 4
    if shape == 4:  # the stream: up to 16 tokens that fit in 160 KB of LDS, with two parts of each of 8 waves
        return b > 16 or b * ((cols + 127) // 128 * 256 + 16) + 2 * 8 * ((b + 3) // 4) * 256 > 160 * 1024
    if 8 <= shape <= 15:  # rows in whole 16-byte chunks: deep slices and staged tiles
        return X.data_ptr() % 16 != 0 or (b > 1 and X.stride(0) % 8 != 0)
    return False  # the choice, direct, slices, staged tiles through registers


def check_refusals(b, rows, cols, group, affine, pad=0, shift=0):
    """Every shape against that rule; those that take the operands give the exact result (whole numbers)."""
    w = Weights(rows, cols, group, affine, "bf16", cols, True)
    X = tokens(b, cols, cols + 1, True, pad, shift)
    want = w.ref(f64(X))[0]
    for shape in SHAPES:
        what = f"shape {shape}: {b} x {rows} x {cols}, stride {X.stride(0)}, address % 16 = {X.data_ptr() % 16}"
        Y = torch.full((b, rows), float("nan"), device=DEV)
        try:
            w.run(X, Y, shape)
        except uw.UwError as e:
            assert e.status == uw.UW_ERR_UNSUPPORTED and refuses(shape, b, cols, X), f"{what}: refused"
            continue
        assert not refuses(shape, b, cols, X), f"{what}: not refused"
        assert np.array_equal(f64(Y), want), what


@pytest.mark.parametrize("cols", WIDTHS)
def test_shapes_that_refuse_by_width(cols):
    for (group, affine), b, rows in zip(itertools.product((32, 64, 128), (False, True)), (1, 2, 16, 17, 5, 3), (1, 15, 16, 33, 64, 70)):
        check_refusals(b, rows, cols, group, affine)
        check_refusals(b, rows, cols, group, affine, pad=-cols % 8)


@pytest.mark.parametrize("b", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129, 200, 256, 257])
def test_shapes_that_refuse_by_batch(b):
    check_refusals(b, 130, 520, 32, True)


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (8, 8), (1, 0), (3, 1), (4, 2), (0, 5), (16, 7)])
def test_shapes_that_refuse_by_alignment(pad, shift):
    for b, rows, cols, group in ((1, 40, 136, 64), (5, 100, 1001, 32), (33, 70, 300, 128), (150, 64, 129, 64)):
        check_refusals(b, rows, cols, group, True, pad, shift)


@pytest.mark.parametrize("b,cols", [(1, 65536), (2, 40960), (4, 14336), (5, 14336), (6, 14336), (11, 6656), (12, 6656), (16, 4096), (16, 4352), (16, 4608)])
def test_shapes_that_refuse_by_the_stream_s_memory(b, cols):
    check_refusals(b, 33, cols, 128, False)
