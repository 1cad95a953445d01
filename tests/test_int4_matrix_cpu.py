"""Int4Matrix without a GPU: it refuses tokens and outputs of another width than its own before anything else.  (An odd
width and the even one above it have the same packed rows and groups, so the operators cannot tell them apart.)"""
import pytest
import torch

uw = pytest.importorskip("decode_gemv_canonical_amd")


def matrix(rows, cols, group, affine=False):
    groups = (cols + group - 1) // group
    scale = torch.ones(groups, rows)
    return uw.Int4Matrix(torch.zeros(rows, (cols + 1) // 2, dtype=torch.uint8), scale, scale.clone() if affine else None, cols, group)


@pytest.mark.parametrize("cols,other", [(1000, 999), (1001, 1002), (999, 1000), (1002, 1001), (64, 63), (1000, 1128), (1, 2)])
@pytest.mark.parametrize("affine", [False, True])
def test_other_widths_are_refused(cols, other, affine):
    m = matrix(16, cols, 64, affine)
    x = torch.zeros(3, other, dtype=torch.bfloat16)
    for call in (lambda: m.gemm(x, torch.zeros(3, 16)), lambda: m.gemm(x), lambda: m.gemv(x[0], torch.zeros(16)), lambda: m.gemv(x[0])):
        with pytest.raises(ValueError, match=f"{cols} columns"):
            call()
    with pytest.raises(ValueError, match=f"\\(16, {cols}\\)"):
        m.dequantize(torch.zeros(16, other))
    with pytest.raises(ValueError, match=f"\\(16, {cols}\\)"):
        m.dequantize(torch.zeros(15, cols))


def test_tokens_of_other_ranks_are_refused():
    m = matrix(16, 64, 64)
    for call in (lambda: m.gemm(torch.zeros(64)), lambda: m.gemm(torch.zeros(2, 3, 64)), lambda: m.gemv(torch.zeros(1, 64)),
                 lambda: m.gemv(torch.zeros(()))):
        with pytest.raises(ValueError, match="64 columns"):
            call()
    for call in (lambda: m.gemm([1.0] * 64), lambda: m.gemv(None), lambda: m.dequantize(7)):
        with pytest.raises(TypeError):
            call()


def test_the_right_width_reaches_the_binding():
    m = matrix(16, 1001, 64)
    for call in (lambda: m.gemm(torch.zeros(2, 1001, dtype=torch.bfloat16), torch.zeros(2, 16)),
                 lambda: m.gemv(torch.zeros(1001, dtype=torch.bfloat16), torch.zeros(16)), lambda: m.dequantize(torch.zeros(16, 1001))):
        with pytest.raises(ValueError, match="CUDA"):  # host tensors
            call()
