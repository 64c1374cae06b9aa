// f8_quant.hip -- quantisation to 8-bit floating point with a power-of-two
// scale for each block of 128.
//
// For a block with largest finite size t = f 2^p (f in [1/2, 1)), the scale is
// 2^e with the least e such that t <= 2^e * top, top = 0.875 * 2^P the format's
// largest value (P = 9 for E4M3, 16 for E5M2): e = p - P, plus 1 where
// f > 0.875. x * 2^-e is exact, so the rounding to 8 bits is the only one.
//
// Bound by memory. A workgroup holds 128 x 128 values in registers, 8 rows x 8
// columns a thread: a row's block lies in 16 lanes (its largest value is four
// exchanges away), a column's in 16 lane groups (two exchanges and one trip
// through LDS). So x is read once for both directions. The transposed bytes go
// through LDS, 8 rows of a column at a time, so that both results are written
// in whole 128-byte lines. 11008 x 4096 from F32, both ways: 58 us, 4.7 TB/s, the
// rate of a large copy; 3 x 1000 x 1111: 9.9 us, a single round of 216 workgroups
// that wait for their loads once and for LDS twice.
#include "grad_internal.h"

namespace sm {
namespace {

constexpr int kWave = 64;

// e + 127 of a block from the bits of its largest finite size.
template <bool E5M2>
__device__ __forceinline__ int scale_byte(uint32_t top) {
    // top = 1.m * 2^(field - 127) = f 2^p with p = field - 126; f > 0.875 where 1.m > 1.75
    const int e = (int)(top >> 23) - 126 - (E5M2 ? 16 : 9) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return top == 0 ? kF8Zero : (e < -127 ? 0 : e + 127);
}

// 2^(127 - byte): what values are multiplied by.
__device__ __forceinline__ float inverse_scale(int byte) {
    // byte <= 247 (the largest fp32 value), so the exponent field 254 - byte is positive
    return __uint_as_float((uint32_t)(254 - byte) << 23);
}

template <bool E5M2>
__device__ __forceinline__ uint32_t to_f8x4(float a, float b, float c, float d) {
    int r = 0;
    if (E5M2) {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    }
    return (uint32_t)r;
}

__device__ __forceinline__ uint32_t finite_size(float v) {  // bits of |v|, 0 for NaN and infinities
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b >= 0x7f800000u ? 0u : b;
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Thread (wave w, lane l): rows 8 (4 w + l / 16) + 0..7 of the tile, columns
// 8 (l % 16) + 0..7.
template <bool BF16, bool E5M2, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void f8_quant_kernel(F8Quant f) {
    __shared__ uint32_t col_top[COLS ? 4 : 1][COLS ? 128 : 1];
    __shared__ __attribute__((aligned(16))) uint2 tile[COLS ? 128 * 16 : 1];  // [column][8 rows], swizzled
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int rg = wave * 4 + lane / 16, cg = lane % 16;
    const int64_t ct = blockIdx.x % f.col_tiles;
    const int64_t rt = blockIdx.x / f.col_tiles % f.row_tiles;
    const int64_t batch = blockIdx.x / f.col_tiles / f.row_tiles;
    const int64_t r0 = rt * 128 + rg * 8, c0 = ct * 128 + cg * 8;
    [[maybe_unused]] const bool whole = (ct + 1) * 128 <= f.cols && (rt + 1) * 128 <= f.rows;
    float v[8][8];
    // BF16: all of a thread's loads before any is unpacked (3001 x 5003 both ways
    // 25.3 -> 21.7 us). F32: each where it is used, since behind the last column its
    // twice as many registers cost more to move (3 x 1000 x 1111 10.2 us, 12.5 us the
    // other way; 11008 x 4096 the same).
    if constexpr (BF16) {
        Raw<BF16, 8> raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // rows past the last one: that one again, then zeros
            const int64_t row = r0 + i < f.rows ? r0 + i : f.rows - 1;
            raw[i] = load_raw<BF16, 8>(f.x, (batch * f.rows + row) * f.cols, (int)c0, (int)f.cols);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            unpack(raw[i], r0 + i < f.rows ? (int)c0 : (int)f.cols + 7, (int)f.cols, v[i], whole);
    } else {
        const int have = (int)(f.cols - c0 < 0 ? 0 : f.cols - c0 < 8 ? f.cols - c0 : 8);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            load_n<BF16>(f.x, (batch * f.rows + r0 + i) * f.cols + c0, r0 + i < f.rows ? have : 0, v[i]);
    }
    uint32_t top[8] = {};  // of the thread's columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t row_top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = finite_size(v[i][j]);
            row_top = umax(row_top, b);
            top[j] = umax(top[j], b);
        }
        if (ROWS) {
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) row_top = umax(row_top, __shfl_xor(row_top, d));
            if (r0 + i < f.rows) {
                const int byte = scale_byte<E5M2>(row_top);
                const float s = inverse_scale(byte);
                const int64_t row = batch * f.rows + r0 + i;
                *reinterpret_cast<uint2 *>(f.q + row * f.pitch + c0) =
                    make_uint2(to_f8x4<E5M2>(v[i][0] * s, v[i][1] * s, v[i][2] * s, v[i][3] * s),
                               to_f8x4<E5M2>(v[i][4] * s, v[i][5] * s, v[i][6] * s, v[i][7] * s));
                uint8_t *out = f.q_scale + row * f.scale_pitch + ct;
                if (cg == 0) *out = (uint8_t)byte;
                // padding behind the row's last block
                if (ct == f.col_tiles - 1 && cg > 0 && ct + cg < f.scale_pitch) out[cg] = kF8Zero;
            }
        }
    }
    if (COLS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top[j] = umax(top[j], __shfl_xor(top[j], 16));
            top[j] = umax(top[j], __shfl_xor(top[j], 32));
        }
        if (lane < 16)
#pragma unroll
            for (int j = 0; j < 8; ++j) col_top[wave][cg * 8 + j] = top[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = cg * 8 + j;
            const uint32_t t = umax(umax(col_top[0][c], col_top[1][c]), umax(col_top[2][c], col_top[3][c]));
            const int byte = scale_byte<E5M2>(t);
            const float s = inverse_scale(byte);
            // the column group rotates the rows' places, so that 16 lanes write to 16 places of a bank row
            tile[c * 16 + (rg ^ cg)] =
                make_uint2(to_f8x4<E5M2>(v[0][j] * s, v[1][j] * s, v[2][j] * s, v[3][j] * s),
                           to_f8x4<E5M2>(v[4][j] * s, v[5][j] * s, v[6][j] * s, v[7][j] * s));
            if (rg == j && c0 + j < f.cols) {  // one row group for each column
                uint8_t *out = f.qt_scale + (batch * f.cols + c0 + j) * f.tscale_pitch + rt;
                *out = (uint8_t)byte;
                if (rt == f.row_tiles - 1)
                    for (int i = 1; rt + i < f.tscale_pitch; ++i) out[i] = kF8Zero;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = i * 32 + threadIdx.x / 8, p = threadIdx.x % 8 * 2;  // 16 rows of a column
            if (ct * 128 + c < f.cols) {
                const uint2 lo = tile[c * 16 + (p ^ (c / 8))], hi = tile[c * 16 + ((p + 1) ^ (c / 8))];
                *reinterpret_cast<uint4 *>(f.qt + (batch * f.cols + ct * 128 + c) * f.tpitch + rt * 128 + p * 8) =
                    make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
}

template <bool BF16, bool E5M2>
void launch(const F8Quant &f, hipStream_t s) {
    const dim3 grid((unsigned)(f.batch * f.row_tiles * f.col_tiles));
    if (f.q && f.qt)
        f8_quant_kernel<BF16, E5M2, true, true><<<grid, 256, 0, s>>>(f);
    else if (f.q)
        f8_quant_kernel<BF16, E5M2, true, false><<<grid, 256, 0, s>>>(f);
    else
        f8_quant_kernel<BF16, E5M2, false, true><<<grid, 256, 0, s>>>(f);
}

}  // namespace

void launch_f8_quant(const F8Quant &f, hipStream_t s) {
    if (f.bf16)
        f.e5m2 ? launch<true, true>(f, s) : launch<true, false>(f, s);
    else
        f.e5m2 ? launch<false, true>(f, s) : launch<false, false>(f, s);
}

}  // namespace sm
