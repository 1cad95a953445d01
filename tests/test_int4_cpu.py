"""4-bit weights and the block norm without a GPU: the oracle's own pins and
the library's refusals (every bad call is turned away before any launch)."""
import numpy as np
import pytest
import torch

from oracle import int4 as o4
from oracle import int8 as o8

uw = pytest.importorskip("decode_gemv_canonical_amd")
INV, UNSUP, OK = uw.UW_ERR_INVALID, uw.UW_ERR_UNSUPPORTED, uw.UW_OK
F32, BF16, I8 = uw.UW_F32, uw.UW_BF16, uw.UW_I8
P = 1 << 20  # stands for a device address: a refused call never touches it


def test_oracle_quantize_by_hand():
    # scale 1: ties to even; the largest at 7
    q, s, m = o4.quantize(np.array([[7.0, -3.5, 2.5, 0.5, -7.0]]), 32, False, False)
    assert m is None and s.tolist() == [[1.0]] and q.tolist() == [[7, -4, 2, 0, -7]]
    # affine: -15 .. 15 in steps of 2 takes all 16 integers, middle between them at q = -0.5
    q, s, m = o4.quantize(np.arange(-15.0, 16.0, 2.0)[None], 32, True, False)
    assert s.tolist() == [[2.0]] and m.tolist() == [[1.0]] and q.tolist() == [list(range(-8, 8))]
    assert np.array_equal(o4.values(q, s, m, 32), np.arange(-15.0, 16.0, 2.0)[None])
    # zeros, and a row with a NaN
    q, s, _ = o4.quantize(np.array([[0.0, 0.0], [1.0, np.nan]]), 64, False, True)
    assert not q.any() and s[0, 0] == np.float32(2.0 ** -126) and np.isnan(s[0, 1])


def test_oracle_quantize_error_is_half_a_step():
    rng = np.random.default_rng(1)
    p = rng.standard_normal((5, 333)).astype(np.float32)
    for affine in (False, True):
        q, s, m = o4.quantize(p, 64, affine, False)
        assert (np.abs(o4.values(q, s, m, 64) - p) <= 0.5001 * o4.spread(s, 333, 64)).all()
        assert np.array_equal(o4.unpack(o4.pack(q), 333), q)


def test_oracle_gemm_is_the_product_of_the_values():
    rng = np.random.default_rng(2)
    q = rng.integers(-8, 8, (6, 70))
    s, m = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))
    x = rng.standard_normal((2, 70))
    want = np.zeros((2, 6))
    for b in range(2):
        for n in range(6):
            for k in range(70):
                want[b, n] += x[b, k] * (s[k // 32, n] * q[n, k] + m[k // 32, n])
    assert np.allclose(o4.gemm(q, s, m, 32, x)[0], want, rtol=1e-12)


def test_oracle_join_without_norm_and_gate_is_the_sum():
    x, r = np.array([[3.0, 4.0]]), np.array([[1.0, 1.0]])
    assert o4.join(x, r, False, None, 1e-5, None, 1.0, 1.0)[0].tolist() == [[4.0, 5.0]]
    h, _ = o4.join(x, r, True, np.array([2.0, 1.0]), 1e-5, np.array([0.5, 0.0]), 2.0, 0.5)
    k = 1 / np.sqrt(12.5 + float(np.float32(1e-5)))
    assert np.allclose(h, [[0.5 + 2 * 0.5 * 2 * 3 * k, 0.5]], rtol=1e-15)


def quant(**k):
    a = dict(X=P, rows=4, cols=64, ldx=64, xt=BF16, group=32, Q=P, ldq=32, scale=P, lds=4, offset=None, ldo=0, st=BF16)
    a.update(k)
    return uw.library().uw_i4_quantize(*a.values(), None)


def dequant(**k):
    a = dict(Q=P, rows=4, cols=64, ldq=32, group=32, scale=P + 4096, lds=4, offset=None, ldo=0, st=BF16, Y=P + 8192, ldy=64, yt=BF16)
    a.update(k)
    return uw.library().uw_i4_dequantize(*a.values(), None)


FORM = [{"group": 0}, {"group": 16}, {"group": 48}, {"group": 256}, {"group": -32}, {"st": I8}, {"st": 9}, {"rows": -1},
        {"cols": 0}, {"rows": 1 << 40}, {"cols": 1 << 40}, {"scale": None}, {"scale": P + 1}, {"lds": 3}, {"st": F32, "scale": P + 2},
        {"offset": P + 1, "ldo": 4}, {"offset": P + 512, "ldo": 3}, {"ldq": 31}, {"ldq": 24}, {"ldq": 16}, {"Q": None},
        {"Q": P + 8}, {"ldq": 40}]


@pytest.mark.parametrize("k", FORM + [{"X": None}, {"X": P + 1}, {"xt": I8}, {"ldx": 63}, {"xt": F32, "X": P + 2}])
def test_quantize_refuses(k):
    assert quant(**{"Q": P + 2048, "scale": P + 4096, **k}) == INV
    assert "uw_i4_quantize" in uw.uw_last_error()


@pytest.mark.parametrize("k", FORM + [{"Y": None}, {"Y": P + 8193}, {"yt": I8}, {"ldy": 63}])
def test_dequantize_refuses(k):
    assert dequant(**k) == INV
    assert "uw_i4_dequantize" in uw.uw_last_error()


def test_overlaps_are_refused():
    far = dict(X=P, Q=P + 4096, scale=P + 8192, offset=P + 12288, ldo=4)
    for k in ({"Q": P}, {"Q": P + 112}, {"scale": P + 16}, {"scale": P + 4096}, {"offset": P + 8192}, {"offset": P + 4096 + 32},
              {"offset": P + 2}):
        assert quant(**{**far, **k}) == INV and "overlaps" in uw.uw_last_error()
    for k in ({"Y": P}, {"Y": P + 4096}, {"Y": P + 4096 - 256, "yt": F32}):
        assert dequant(**k) == INV and "overlaps" in uw.uw_last_error()
    for k in ({"Y": P}, {"Y": P + 4096}, {"Y": P + 8192}, {"Y": P + 12288, "bias": P + 12288 + 16}):
        assert gemm(**k) == INV and "overlaps" in uw.uw_last_error()


def gemm(shape=None, **k):
    a = dict(W=P, rows=32, cols=64, ldw=32, group=64, scale=P + 4096, lds=32, offset=None, ldo=0, st=BF16, X=P + 8192, batch=4,
             ldx=64, bias=None, Y=P + 12288, ldy=32, yt=F32)
    a.update(k)
    if shape is None:
        return uw.library().uw_i4_gemm(*a.values(), None)
    return uw.library().uw_i4_gemm_shaped(*a.values(), shape, None)


@pytest.mark.parametrize("k", [
    {"W": None}, {"W": P + 4}, {"ldw": 33}, {"ldw": 16}, {"X": None}, {"X": P + 8193}, {"Y": None}, {"Y": P + 2}, {"yt": I8},
    {"yt": 7}, {"rows": 0}, {"batch": -1}, {"cols": 0}, {"ldx": 63}, {"ldy": 31}, {"group": 96}, {"st": I8}, {"scale": None},
    {"scale": P + 1}, {"cols": 65, "ldw": 48, "ldx": 65, "lds": 31}, {"offset": P + 3}, {"bias": P + 2}, {"batch": 1 << 40},
    {"rows": 1 << 40}, {"cols": 1 << 40},
])
def test_gemm_refuses(k):
    assert gemm(**k) == INV
    assert "uw_i4_gemm" in uw.uw_last_error()
    assert gemm(shape=1, **k) == INV


def test_gemm_shaped_refuses_unknown_shapes():
    for shape in (0, -1, uw.uw_i4_gemm_shape_count()):
        assert gemm(shape=shape) == INV


def test_gemm_refuses_more_tiles_than_a_launch_holds():
    big = dict(rows=1 << 39, batch=1 << 39, ldy=1 << 39, lds=1 << 39, group=64)
    assert gemm(**big) == UNSUP
    for shape in range(1, uw.uw_i4_gemm_shape_count()):
        assert gemm(shape=shape, **big) == UNSUP


def test_gemm_shapes_refuse_what_does_not_fit_their_offsets():
    long = dict(rows=1, batch=1, cols=1 << 21, ldw=1 << 20, ldx=1 << 21, lds=1, group=32, X=P + (1 << 24), scale=P + (1 << 26),
                Y=P + (1 << 28))
    far = dict(scale=1 << 40, lds=1 << 30, cols=128, group=32, ldw=64, ldx=128, X=1 << 38)
    for shape in range(2, uw.uw_i4_gemm_shape_count()):
        for k in (long, far, dict(ldw=1 << 22, X=1 << 38), dict(ldx=1 << 21, Y=1 << 38)):
            assert gemm(shape=shape, **k) == UNSUP, (shape, k)


def norm(**k):
    a = dict(X=P, batch=4, cols=64, ldx=64, xt=BF16, post_norm=1, post=P + 65536, pt=BF16, post_eps=1e-5, gate=P + 69632, ldg=0,
             gt=BF16, block_scale=1.0, R=P + 4096, ldr=64, rt=BF16, residual_scale=1.0, H=P + 8192, ldh=64, gain=P + 73728,
             nt=BF16, eps=1e-5, Y=P + 12288, ldy=64, yt=BF16, scale=None)
    a.update(k)
    return uw.library().uw_block_norm(*a.values(), None)


@pytest.mark.parametrize("k", [
    {"X": None}, {"R": None}, {"batch": -1}, {"cols": 0}, {"cols": 1 << 40}, {"batch": 1 << 40}, {"xt": I8}, {"rt": I8},
    {"pt": I8}, {"gt": 5}, {"nt": I8}, {"yt": 3}, {"ldx": 63}, {"ldr": 63}, {"ldh": 63}, {"ldy": 63}, {"ldg": 63},
    {"ldx": 1 << 41}, {"eps": 0.0}, {"eps": float("nan")}, {"post_eps": 0.0}, {"post_eps": float("inf")}, {"post_eps": -1.0},
    {"block_scale": float("inf")}, {"block_scale": float("nan")}, {"residual_scale": float("-inf")}, {"post_norm": 0},
    {"Y": None}, {"Y": None, "gain": None, "H": None}, {"X": P + 1}, {"R": P + 4097}, {"H": P + 1}, {"Y": P + 12289},
    {"post": P + 1}, {"gate": P + 1}, {"gain": P + 1}, {"yt": I8}, {"yt": I8, "scale": P + 2},
    {"Y": P + 8192}, {"H": P + 128}, {"Y": P + 69632}, {"H": P + 65536}, {"Y": P + 73728}, {"yt": I8, "scale": P + 4096},
    {"gate": P + 12288, "ldg": 64}, {"H": P, "Y": P}, {"xt": F32, "X": P + 2},
])
def test_block_norm_refuses(k):
    assert norm(**k) == INV
    assert "uw_block_norm" in uw.uw_last_error()


@pytest.mark.parametrize("k", [{"cols": 1 << 31, "ldx": 1 << 31, "ldr": 1 << 31, "ldh": 1 << 31, "ldy": 1 << 31},
                               {"ldx": 1 << 32}, {"ldr": 1 << 32}, {"ldg": 1 << 32}])
def test_block_norm_refuses_what_does_not_fit_its_offsets(k):
    far = dict(X=1 << 44, R=1 << 45, H=1 << 46, Y=1 << 47, post=P, gate=1 << 48, gain=P + (1 << 35))
    assert norm(**{**far, **k}) == UNSUP


def test_empty_batches_are_no_ops():
    assert norm(batch=0) == OK and gemm(batch=0) == OK and quant(rows=0) == OK and dequant(rows=0) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(1, 2)
    for call in (lambda: uw.uw_i4_quantize(x, q, s), lambda: uw.uw_i4_dequantize(q, s, x),
                 lambda: uw.uw_i4_gemm(q, s, x, torch.zeros(2, 2)), lambda: uw.uw_block_norm(x, x, Y=x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: uw.uw_i4_quantize([1], q, s), lambda: uw.uw_block_norm(x, None)):
        with pytest.raises((TypeError, ValueError)):
            call()
