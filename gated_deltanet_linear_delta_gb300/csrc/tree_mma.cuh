// tree_mma.cuh -- what the tensor-core kernels of the gated delta rule over trees share: m16n8k16 products of bf16
// (mma.sync), their operands from shared memory, and fp32 values split into bf16 terms.
#pragma once

#include "tc_ops.cuh"
#include "tree.cuh"

namespace gdn {

// ---- products ----------------------------------------------------------------------
// Lane (g = lane / 4, c = lane % 4): D and C hold rows g and g + 8, columns 2 c and 2 c + 1, as {g 2c, g 2c+1, g+8 2c,
// g+8 2c+1}; A the same of both halves of its 16 columns; B rows 2 c .. and 2 c + 8 .. of column g.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four 8 x 8 matrices whose rows are 16 bytes at the lanes' addresses (lanes 0..7 the first's, 8..15 the second's, ..)
__device__ __forceinline__ void load_matrices(uint32_t (&x)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}
// A pair of fp32 as bf16, and what that leaves of them
__device__ __forceinline__ uint32_t split2(float &x, float &y) {
    const uint32_t h = tc::bf2_bits(__floats2bfloat162_rn(x, y));
    x -= __uint_as_float(h << 16);
    y -= __uint_as_float(h & 0xffff0000u);
    return h;
}

// ---- layouts in shared memory: where the 16 bytes `ch` of row r lie (as the tensor maps' swizzles put them) ----
// rows of DK bf16, in blocks of 64 columns of ROWS rows; the 8 rows of a matrix lie in different banks
template <int DK, int ROWS>
__device__ __forceinline__ uint32_t row_piece(int r, int ch) {
    if (DK >= 64) return (uint32_t)((ch >> 3) * (ROWS * 128) + r * 128 + (((ch ^ r) & 7) << 4));
    return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
}
// 32 columns of a state, rows of 128 bytes: 32 bytes of 4 rows 2 apart lie in different banks
__device__ __forceinline__ uint32_t state_piece(int r, int ch) { return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)); }
// block (i, j <= i) of 16 x 16 coefficients, 64 bytes a row (fp32, or two bf16 terms each); rows spread as above
__device__ __forceinline__ uint32_t coef_block(int i, int j) { return (uint32_t)((i * (i + 1) / 2 + j) * 1024); }
__device__ __forceinline__ uint32_t coef_piece(int r, int ch) { return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)); }

}  // namespace gdn
