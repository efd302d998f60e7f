"""What the vocabulary losses' plans hold in the workspace (no GPU needed)."""

import itertools

import pytest

import dense_fp32_gemm_04_gb300 as sg

MB = 1 << 20


def _operand_bytes(T, V, D, two_parts):
    """FP32 operands as parts in rows of whole 128-byte lines: H and W as two float16 parts, H as bfloat16 ones, factors."""
    rows = (D + 63) // 64 * 64 * 2
    return (2 * (T + V) + (2 if two_parts else 3) * T) * rows + 4 * (T + V) + 2048


@pytest.mark.parametrize("T,V,D", [(512, 32768, 256), (2048, 32768, 2048), (4096, 131072, 1024), (8192, 32768, 2048),
                                   (20000, 50021, 515), (300, 300000, 64)])
@pytest.mark.parametrize("mode", [sg.MATH_FP32, sg.MATH_TF32])
def test_dz_of_a_piece_stays_within_its_limit(lib, T, V, D, mode):
    """All parts of dZ that are alive take 512 MB at most: one piece, or two of several; operands and dH's sums beside it."""
    p = sg.vocab_plan(T, V, D, dtype=sg.DTYPE_F32, grad=True, math_mode=mode)
    two = mode == sg.MATH_TF32
    column = T * 2 * ((2 if two else 3) + 2)  # bfloat16 parts for dW, float16 ones for dH
    blocks = (p.piece + 255) // 256 * 256
    dz = min(p.pieces, 2) * blocks * column
    assert dz <= 512 * MB
    assert p.workspace_bytes > dz + _operand_bytes(T, V, D, two)  # dH's sums are the rest
    if p.pieces > 1:  # no more pieces than that takes
        assert V * column > 512 * MB and (V / (p.pieces - 1) + 256) * column > 256 * MB


def test_bfloat16_pieces(lib):
    for T, V in itertools.product((300, 4096, 30000), (32768, 131072)):
        p = sg.vocab_plan(T, V, 1024, grad=True)
        assert min(p.pieces, 2) * T * p.piece * 2 <= 512 * MB
        assert p.pieces == 1 or (V / (p.pieces - 1) + 256) * T * 2 > 256 * MB
