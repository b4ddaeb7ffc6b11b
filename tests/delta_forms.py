"""Shapes that the launchers of the gated delta rule and of the 8-bit product send to each of their kernels, with the
kernel that each one is for; and how near FP32 results of the delta rule have to be."""

# kind, batch, length, key heads, value heads, dk, dv, columns beside q, k, v in their matrix; the block: teams of
# four warps, or single warps
CHAINS = [
    (("bf16", 2, 150, 32, 64, 128, 128, 0), "8 warps"),   # as many heads as an ordinary training pass has
    (("bf16", 2, 129, 32, 64, 72, 120, 0), "8 warps"),    # columns behind dk and dv in stages that come by bulk copies
    (("bf16", 2, 130, 64, 64, 93, 77, 0), "8 warps"),     # no row but the first aligned
    (("bf16", 1, 100, 50, 150, 64, 300, 8), "8 warps"),   # few columns for the last block
    (("bf16", 1, 70, 32, 128, 60, 125, 3), "8 warps"),
    (("f16", 2, 150, 64, 64, 128, 128, 0), "4 warps"),
    (("f16", 2, 65, 32, 64, 104, 120, 16), "4 warps"),
    (("f16", 1, 130, 64, 128, 127, 113, 1), "8 warps"),
    (("f16", 2, 66, 32, 64, 64, 120, 8), "8 warps"),
    (("f16", 2, 128, 64, 64, 64, 64, 0), "4 warps"),
    (("f16", 2, 70, 64, 64, 99, 61, 1), "4 warps"),
    (("f32", 2, 150, 64, 64, 128, 128, 0), "8 warps"),
    (("f32", 2, 65, 32, 64, 104, 120, 8), "8 warps"),
    (("f32", 1, 130, 64, 128, 93, 121, 1), "8 warps"),
    (("f32", 1, 66, 64, 128, 61, 124, 2), "8 warps"),
    (("f32", 2, 129, 64, 64, 60, 64, 4), "4 warps"),
    (("f32", 1, 70, 128, 128, 128, 50, 0), "4 warps"),
    (("bf16", 8, 66, 30, 60, 64, 64, 0), "4 warps"),      # two blocks on an SM
    (("bf16", 2, 130, 15, 30, 128, 64, 0), "2 teams"),
    (("bf16", 2, 130, 15, 30, 64, 64, 0), "2 teams"),
    (("bf16", 2, 70, 30, 30, 50, 50, 3), "2 teams"),
    (("bf16", 2, 128, 64, 64, 64, 64, 0), "4 warps"),
    (("bf16", 2, 70, 32, 64, 50, 61, 3), "4 warps"),
    (("f16", 2, 130, 30, 30, 64, 64, 0), "2 teams"),
    (("f32", 2, 130, 15, 30, 60, 64, 0), "2 teams"),
    (("f32", 1, 190, 2, 4, 128, 128, 0), "1 teams"),
]
# the same for packed sequences between these rows
CUTS = [3, 3, 131, 132, 259, 300]
PACKED = [("bf16", 15, 30, 128, 128), ("bf16", 30, 30, 93, 77), ("f32", 15, 30, 128, 128), ("f16", 30, 30, 100, 116)]

# tokens, features, depth, elements beside y's rows; the kernel, its columns and the blocks that share a tile
PRODUCTS = [
    ((4001, 2056, 1043, 0), "gemm_q8_rows_kernel 256 1"),   # more tiles than SMs, the last of few columns or tokens
    ((16384, 512, 1100, 8), "gemm_q8_rows_kernel 256 1"),
    ((1000, 2008, 640, 0), "gemm_q8_rows_kernel 128 1"),
    ((2311, 2008, 208, 8), "gemm_q8_rows_kernel 128 1"),
    ((20000, 8, 130, 0), "gemm_q8_rows_kernel 128 1"),
    ((4485, 1301, 300, 0), "gemm_q8_kernel 128 1"),         # rows that do not take 16 bytes at once
    ((1001, 2001, 640, 1), "gemm_q8_kernel 128 1"),
    ((2500, 2048, 256, 1), "gemm_q8_kernel 64 1"),
    ((20000, 3, 130, 0), "gemm_q8_kernel 64 1"),
    ((65, 4456, 9099, 0), "gemm_q8_kernel 128 4"),
    ((1335, 506, 2578, 1), "gemm_q8_kernel 128 2"),
    ((300, 257, 2000, 2), "gemm_q8_kernel 64 8"),
    ((40, 39901, 1200, 1), "gemm_q8_kernel 64 1"),          # more tiles than SMs
    ((17, 1000, 1040, 0), "gemm_q8_kernel 32 4"),
    ((16, 30000, 96, 1), "gemm_q8_kernel 16 1"),
]


def allowed(length, backward=False):
    """Relative error in the Frobenius norm of what the delta rule returns in FP32. Every operand of a matrix product
    is within 2^-18 of itself and the two operands' last terms' product is left out, 2^-18 too: a product of terms
    whose norm is the result's is off by three of them at most, about one as their errors are independent. A chunk's results go
    through six products one after another (K S, the inverse, U, the mixing matrix's two, the state's update)
    and an FP32 sum each, less than 8 in all, and chunks add up; gradients come through the forward and the
    backward chain."""
    chunks = -(-length // 64)
    return 2.0 ** -18 * 8 * chunks * (2 if backward else 1)
