"""The 8-bit activation path without a GPU: the oracle's own pins and the
library's refusals (every bad call is turned away before any launch)."""
import contextlib
import importlib.util
import os
import types

import numpy as np
import pytest
import torch

from oracle import int8 as o8

uw = pytest.importorskip("decode_gemv_canonical_amd")
INV, UNSUP, OK = uw.UW_ERR_INVALID, uw.UW_ERR_UNSUPPORTED, uw.UW_OK
F32, BF16, I8 = uw.UW_F32, uw.UW_BF16, uw.UW_I8
P = 1 << 20  # stands for a device address: a refused call never touches it


def test_oracle_quantize_by_hand():
    q, s = o8.quantize(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1, np.nan, 2, 3], [np.inf, 1, 2, 3]], np.float32))
    assert s[0] == 1.0 and q[0].tolist() == [127, -64, 0, 2]  # ties to even: -63.5, 0.5, 1.5
    assert s[1] == np.float32(2.0 ** -126) and not q[1].any()
    assert np.isnan(s[2]) and np.isnan(s[3]) and not q[2:].any()


def test_oracle_norm_and_silu_by_hand():
    h = np.array([[3.0, 4.0]])
    y = o8.rmsnorm(h, np.array([1.0, 2.0]), 1e-5)
    r = 1 / np.sqrt(12.5 + float(np.float32(1e-5)))
    assert np.allclose(y, [[3 * r, 8 * r]], rtol=1e-15)
    assert o8.silu_mul(np.array([[0.0, -800.0]]), np.array([[5.0, 1.0]])).tolist() == [[0.0, 0.0]]


def test_oracle_norm_matches_differences_of_scale():
    # y does not change when h is scaled (eps small against mean(h^2)), and the integers do not depend on the norm
    rng = np.random.default_rng(0)
    h = rng.standard_normal((3, 50))
    assert np.allclose(o8.rmsnorm(h * 64, None, 1e-12), o8.rmsnorm(h, None, 1e-12), rtol=1e-10)


def norm(**k):
    a = dict(X=P, batch=4, cols=64, ldx=64, xt=BF16, R=P, ldr=64, rt=BF16, H=P + 4096, ldh=64, gain=P, gt=BF16, eps=1e-5,
             Y=P + 8192, ldy=64, yt=BF16, scale=None)
    a.update(k)
    return uw.library().uw_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("k", [
    {"X": None}, {"Y": None}, {"batch": -1}, {"cols": 0}, {"cols": -3}, {"cols": 1 << 40}, {"batch": 1 << 40},
    {"xt": I8}, {"xt": 7}, {"rt": I8}, {"rt": 9}, {"gt": I8}, {"gt": -1}, {"yt": 3}, {"ldx": 63}, {"ldr": 63},
    {"ldh": 63}, {"ldy": 63}, {"ldx": 1 << 41}, {"eps": 0.0}, {"eps": -1e-5}, {"eps": float("nan")},
    {"eps": float("inf")}, {"R": None}, {"X": P + 1}, {"Y": P + 1}, {"R": P + 1}, {"H": P + 1}, {"gain": P + 1},
    {"yt": I8}, {"yt": I8, "scale": P + 2}, {"Y": P + 4096}, {"xt": F32, "X": P + 2},
])
def test_rmsnorm_refuses(k):
    assert norm(**k) == INV
    assert "uw_rmsnorm" in uw.uw_last_error()


def test_empty_batches_are_no_ops():
    lib = uw.library()
    assert norm(batch=0) == OK
    assert lib.uw_silu_mul(None, 64, None, 64, BF16, 0, 64, None, 64, BF16, None, None) == OK
    assert lib.uw_i8_quantize(None, 0, 64, 64, BF16, None, 64, None, None) == OK
    assert lib.uw_i8_dequantize(None, 0, 64, 64, None, None, 64, BF16, None) == OK
    assert lib.uw_i8_gemm(P, 16, 64, 64, P, None, 0, 64, None, None, None, 16, F32, None) == OK


def silu(**k):
    a = dict(G=P, ldg=64, U=P, ldu=64, xt=BF16, batch=4, cols=64, Y=P, ldy=64, yt=BF16, scale=None)
    a.update(k)
    return uw.library().uw_silu_mul(*a.values(), None)


@pytest.mark.parametrize("k", [
    {"G": None}, {"U": None}, {"Y": None}, {"xt": I8}, {"yt": 5}, {"yt": I8}, {"ldg": 60}, {"ldu": 60}, {"ldy": 60},
    {"batch": -2}, {"cols": 0}, {"G": P + 1}, {"U": P + 1},
])
def test_silu_mul_refuses(k):
    assert silu(**k) == INV


def quant(**k):
    a = dict(X=P, rows=4, cols=64, ldx=64, xt=BF16, Q=P, ldq=64, scale=P)
    a.update(k)
    return uw.library().uw_i8_quantize(*a.values(), None)


def dequant(**k):
    a = dict(Q=P, rows=4, cols=64, ldq=64, scale=P, Y=P, ldy=64, yt=BF16)
    a.update(k)
    return uw.library().uw_i8_dequantize(*a.values(), None)


@pytest.mark.parametrize("k", [{"X": None}, {"Q": None}, {"scale": None}, {"scale": P + 1}, {"xt": I8}, {"ldx": 3},
                               {"ldq": 3}, {"rows": -1}, {"cols": 0}, {"X": P + 1}])
def test_quantize_refuses(k):
    assert quant(**k) == INV


@pytest.mark.parametrize("k", [{"Y": None}, {"Q": None}, {"scale": None}, {"scale": P + 2}, {"yt": I8}, {"ldy": 3},
                               {"ldq": 3}, {"rows": -1}, {"cols": 0}, {"Y": P + 1}])
def test_dequantize_refuses(k):
    assert dequant(**k) == INV


def gemm(shape=None, ks=0, **k):
    a = dict(W=P, rows=32, cols=64, ldw=64, ws=P, X=P, batch=4, ldx=64, xs=P, bias=None, Y=P, ldy=32, yt=F32)
    a.update(k)
    if shape is None:
        return uw.library().uw_i8_gemm(*a.values(), None)
    return uw.library().uw_i8_gemm_shaped(*a.values(), shape, ks, None)


@pytest.mark.parametrize("k,want", [
    ({"W": None}, INV), ({"X": None}, INV), ({"Y": None}, INV), ({"ws": None}, INV), ({"xs": None}, INV),
    ({"ws": P + 1}, INV), ({"xs": P + 3}, INV), ({"bias": P + 2}, INV), ({"yt": I8}, INV), ({"yt": 4}, INV),
    ({"rows": 0}, INV), ({"batch": -1}, INV), ({"cols": 0}, INV), ({"ldw": 63}, INV), ({"ldx": 63}, INV),
    ({"ldy": 31}, INV), ({"Y": P + 2}, INV), ({"cols": 131072, "ldw": 131072, "ldx": 131072}, UNSUP),
    ({"cols": 1 << 40}, INV), ({"rows": 1 << 40}, INV),
])
def test_gemm_refuses(k, want):
    assert gemm(**k) == want
    assert gemm(shape=1, **k) == want


def test_gemm_shaped_refuses():
    n = uw.uw_i8_gemm_shape_count()
    assert n > 1
    for shape in (0, -1, n):
        assert gemm(shape=shape) == INV
    for ks in (-1, 9):
        assert gemm(shape=1, ks=ks) == INV
    # the last shape is a staged one: 16-byte aligned operands and strides only
    for k in ({"W": P + 4}, {"X": P + 8}, {"ldw": 72}, {"ldx": 65}, {"ldw": 1 << 22}):
        assert gemm(shape=n - 1, **k) == UNSUP


def test_gemm_refuses_more_tiles_than_a_launch_holds():
    big = dict(rows=1 << 39, batch=1 << 39, ldy=1 << 39)
    assert gemm(**big) == UNSUP
    assert gemm(W=P + 1, **big) == UNSUP
    for shape in range(1, uw.uw_i8_gemm_shape_count()):
        assert gemm(shape=shape, **big) == UNSUP


def test_binding_refuses_host_tensors():
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError):
        uw.uw_rmsnorm(x, None, x)
    with pytest.raises(ValueError):
        uw.uw_silu_mul(x, x, x)
    with pytest.raises(ValueError):
        uw.uw_i8_quantize(x, q, s)
    with pytest.raises(ValueError):
        uw.uw_i8_dequantize(q, s, x)
    with pytest.raises(ValueError):
        uw.uw_i8_gemm(q, s, q, s, torch.zeros(2, 2))
    with pytest.raises(ValueError):
        uw.Int8Matrix(q, s)


# -- overlaps ------------------------------------------------------------------
# norm() above: 4 rows of 64 bf16, X and R at P, H at P + 4096, Y at P + 8192

@pytest.mark.parametrize("k", [
    {"H": P, "ldh": 72}, {"H": P, "rt": F32, "R": P + 8192, "Y": P + 65536},   # in place with another stride or type
    {"H": P + 2}, {"H": P + 128}, {"H": P - 128},                              # one element, one row on
    {"R": P + 65536, "Y": P, "ldy": 65}, {"R": P + 65536, "Y": P, "yt": F32}, {"Y": P + 64}, {"Y": P - 4, "yt": F32},
    {"Y": P + 4096 + 510}, {"Y": P + 4096 - 510},                              # the last or first element of H
    {"R": P + 65536, "Y": P + 65536, "yt": I8, "scale": P + 16384},            # integers over the residual
    {"yt": I8, "scale": P + 8}, {"yt": I8, "scale": P + 8192 + 252}, {"yt": I8, "scale": P + 4096},
    {"gain": P + 8192 + 384, "Y": P + 8192}, {"gain": P + 4096}, {"H": None, "gain": P + 8192},
])
def test_rmsnorm_refuses_overlaps(k):
    assert norm(**k) == INV
    assert "overlap" in uw.uw_last_error()


@pytest.mark.parametrize("k", [
    {"Y": P + 2}, {"Y": P, "ldy": 66}, {"Y": P, "yt": F32}, {"Y": P, "yt": I8, "scale": P + 8192},
    {"U": P + 4096, "Y": P + 4096 - 510}, {"Y": P + 4096, "yt": I8, "scale": P + 4096 + 252}, {"G": P + 2, "Y": P},
    {"ldg": 128, "ldu": 128, "U": P + 128, "Y": P + 64, "ldy": 128},           # half of each half
    {"Y": P + 4096, "yt": I8, "scale": P},
])
def test_silu_mul_refuses_overlaps(k):
    assert silu(**k) == INV
    assert "overlap" in uw.uw_last_error()


@pytest.mark.parametrize("k", [{"scale": P + 8192}, {"Q": P + 8192}, {"Q": P + 511, "scale": P + 8192},
                               {"Q": P + 8192, "scale": P + 8192 + 255}])
def test_quantize_refuses_overlaps(k):
    k = {name: at if name != "scale" else at // 4 * 4 for name, at in k.items()}
    assert quant(**k) == INV
    assert "overlap" in uw.uw_last_error()


@pytest.mark.parametrize("k", [{}, {"Y": P + 254}, {"Q": P + 4096, "Y": P + 14}, {"Q": P + 4096, "Y": P - 510}])
def test_dequantize_refuses_overlaps(k):
    assert dequant(**k) == INV
    assert "overlap" in uw.uw_last_error()


@pytest.mark.parametrize("k", [{}, {"W": P + 8192, "ws": P + 8192, "xs": P + 8192},
                               {"X": P + 8192, "ws": P + 8192, "xs": P + 8192, "Y": P + 2044},
                               {"W": P + 8192, "X": P + 16384, "ws": P + 508, "xs": P + 8192},
                               {"W": P + 8192, "X": P + 16384, "ws": P + 8192, "xs": P + 508},
                               {"W": P + 8192, "X": P + 16384, "ws": P + 8192, "xs": P + 8192, "bias": P - 124}])
def test_gemm_refuses_overlaps(k):
    for shape in (None, 1):
        assert gemm(shape=shape, **k) == INV
        assert "overlap" in uw.uw_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that are not refused would run on these addresses")
def test_overlaps_are_refused_exactly():
    """Against the sets of bytes: refused where two rows share one, and only there (in place, element for element, aside)."""
    rng = np.random.default_rng(7)
    seen = {True: 0, False: 0}
    for _ in range(20000):
        n, cols = int(rng.integers(1, 6)), int(rng.integers(1, 20))
        ldg = cols + int(rng.integers(0, 40))
        ldy = ldg if rng.random() < 0.5 else cols + int(rng.integers(0, 40))
        at = int(rng.integers(-160, 160))
        xt, yt = (BF16, F32)[rng.integers(2)], (BF16, F32)[rng.integers(2)]
        xs, ys = (2 if xt == BF16 else 4), (2 if yt == BF16 else 4)
        G, Y = P, P + 4 * at
        x_bytes = {r * ldg * xs + e for r in range(n) for e in range(cols * xs)}
        y_bytes = {4 * at + r * ldy * ys + e for r in range(n) for e in range(cols * ys)}
        twin = G == Y and xt == yt and (ldg == ldy or n == 1)
        want = bool(x_bytes & y_bytes) and not twin
        rc = uw.library().uw_silu_mul(G, ldg, G, ldg, xt, n, cols, Y, ldy, yt, None, None)
        assert (rc == INV) == want, (n, cols, ldg, ldy, at, xt, yt)
        seen[want] += 1
    assert min(seen.values()) > 3000


# -- outputs of calls on another stream ---------------------------------------------

class FakeStreams:
    """torch's streams and allocations, recorded: which stream each torch.empty was made under."""

    def __init__(self, monkeypatch):
        self.stack, self.made = [1], []
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.stream(self.stack[-1]))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: self.stream(0))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: self.stream(raw))
        monkeypatch.setattr(torch.cuda, "stream", self.under)
        monkeypatch.setattr(torch, "empty", self.empty)

    def stream(self, raw):
        return types.SimpleNamespace(cuda_stream=raw)

    @contextlib.contextmanager
    def under(self, s):
        self.stack.append(s.cuda_stream)
        yield
        self.stack.pop()

    def empty(self, *shape, dtype=None, device=None):
        self.made.append(self.stack[-1])
        return types.SimpleNamespace(stride=lambda d: 64, data_ptr=lambda: P, numel=lambda: 64, element_size=lambda: 1)


CALLS = {
    "Int8Matrix.gemm": lambda m, s: m.gemm(types.SimpleNamespace(shape=(4, 64), device="cuda"), None, stream=s),
    "Int8Matrix.dequantize": lambda m, s: m.dequantize(stream=s),
    "CompressedMatrix.gemm": lambda m, s: m.gemm(types.SimpleNamespace(shape=(4, 64), device="cuda"), stream=s),
    "CompressedMatrix.gemv": lambda m, s: m.gemv(types.SimpleNamespace(shape=(64,), device="cuda"), stream=s),
    "CompressedMatrix.decompress": lambda m, s: m.decompress(stream=s),
    "CompressedMatrix.autotune": lambda m, s: m.autotune(4, stream=s),
    "CompressedMatrix.transcode_palette": lambda m, s: m.transcode_palette(attach=False, stream=s),
    "PaletteMatrix.gemm": lambda m, s: m.gemm(types.SimpleNamespace(shape=(4, 64), device="cuda"), stream=s),
    "PaletteMatrix.gemv": lambda m, s: m.gemv(types.SimpleNamespace(shape=(64,), device="cuda"), stream=s),
    "PaletteMatrix.decompress": lambda m, s: m.decompress(stream=s),
}


@pytest.mark.parametrize("call", CALLS)
def test_outputs_are_allocated_under_the_stream_that_writes_them(call, monkeypatch):
    mod = uw.uw
    fake = FakeStreams(monkeypatch)
    for name in ("uw_i8_gemm", "uw_i8_dequantize", "uw_gemm_fused", "uw_gemv_fused", "uw_decompress", "uw_autotune",
                 "uw_palette_transcode", "uw_palette_gemm", "uw_palette_gemv",
                 "uw_palette_decompress", "uw_workspace_size", "uw_autotune_scratch_size", "uw_palette_transcode_size"):
        monkeypatch.setattr(mod, name, lambda *a, **k: 256)
    monkeypatch.setattr(mod, "uw_palette_create_transcoded", lambda *a: None)  # a handle that nothing has to destroy
    cls = getattr(mod, call.split(".")[0])
    m = cls.__new__(cls)
    where = types.SimpleNamespace(device="cuda")
    m.q = m.scale = m.d_blob = m.d_buf = where
    m.rows, m.cols, m.handle, m.info = 32, 64, None, {"n_raw_groups": 0}
    for stream, want in ((None, 1), (fake.stream(1), 1), (fake.stream(7), 7), (9, 9), (0, 0)):
        fake.made.clear()
        CALLS[call](m, stream)
        assert fake.made == [want], f"stream {stream}: made under {fake.made}"
        assert fake.stack == [1]
    with pytest.raises(TypeError):
        CALLS[call](m, "s")


# -- the build -------------------------------------------------------------------------

@pytest.mark.parametrize("with_torch", [True, False])
def test_library_builds_without_torch(with_torch, tmp_path, monkeypatch, capsys):
    """libuw.so needs hipcc and g++ alone; only the Python binding's C++ side needs torch."""
    path = os.path.join(os.path.dirname(uw.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("_uw_build_test", path)
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    made = []

    def run(cmd, verbose):
        made.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(b, "_run", run)
    for name, at in (("BUILD", "o"), ("LIBDIR", "lib"), ("LIB", "lib/libuw.so"), ("TORCH_LIB", "lib/_uw_torch.so")):
        monkeypatch.setattr(b, name, str(tmp_path / at))
    if not with_torch:
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    b.build()
    assert os.path.exists(tmp_path / "lib" / "libuw.so")
    assert os.path.exists(tmp_path / "lib" / "_uw_torch.so") == with_torch
    assert any("torch" in a for c in made for a in c if a.startswith("-l")) == with_torch
    assert ("torch" in capsys.readouterr().err) != with_torch
    assert sorted(os.listdir(tmp_path / "lib")) == (["_uw_torch.so", "libuw.so"] if with_torch else ["libuw.so"])


# -- widths ------------------------------------------------------------------------------

@pytest.mark.parametrize("cols", [1 << 36, (1 << 39) + 1])
def test_rows_wider_than_a_launch(cols):
    """silu's plain outputs and dequantize spread a row over a launch's fewer than 2^32 threads."""
    Y = 1 << 45
    for yt in (BF16, F32):
        assert silu(batch=1, cols=cols, yt=yt, Y=Y) == UNSUP
        assert dequant(rows=1, cols=cols, yt=yt, Y=Y, scale=1 << 44) == UNSUP
    assert "wider" in uw.uw_last_error()
