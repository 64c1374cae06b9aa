// linear_loss.hip -- softmax cross entropy of an output layer, and its
// gradients, on the gfx950 matrix cores.
//
//   l[t][v] = scale x[t].w[v],  lse[t] = log sum_v exp l[t][v],  loss[t] = lse[t] - l[t][target]
//   g[t][v] = scale dloss[t] (exp(l[t][v] - lse[t]) - [v = target]),  dx = g w,  dw_m = g_m^T x_m
//
// The logits are not kept. Forward, each tile of them becomes one running
// maximum and one sum of exponentials a row and half a tile's columns, which are
// joined afterwards (where they have few tiles and long rows, the tiles' sums over parts of
// k go through memory, up to 512 MB of them). Backward, the logits of a piece of the vocabulary are computed
// again and stored as g, from which that piece's dw and its share of dx are two
// more products; then the next piece overwrites it.
//
// Everything is a product of BF16 operands on v_mfma_f32_32x32x16_bf16 with
// fp32 sums. An fp32 operand is taken apart into BF16 planes, h + m + l, each the
// rounding of what the ones before it left: three planes hold its 24 bits. A
// product of planes is a longer sum: the pairs (h h), (h m), (m h), (m m),
// (h l), (l h) leave out parts below 2^-22 of the operands' product (6e-9 of a sum of
// random ones). Six BF16 products run at 2.6 times the rate of fp32's own matrix
// instruction. Logits and fp32 results take all planes of their operands. For a BF16
// result g is rounded to one plane, an error as large as that of the result's own
// rounding, and an fp32 operand that meets it is held in two. g is stored in fp32
// where a result is, and its planes are made in registers: it is read once for all of
// them. x and w are laid out as planes by a pass of their own where they are not BF16
// rows of whole vectors.
//
// The products are computed as b a^T: the instruction's rows are out's columns,
// so that a lane's accumulators hold four consecutive columns of one row of out,
// and a row of logits lies in two lanes.
//
// Bound by the matrix pipe, and at full load by the card's power, which lowers its
// clock to 1.7 GHz of 2.4. 8192 tokens of 32000 x 4096 in BF16: logits and their sums 1.63 to 1.73 ms,
// g 1.69, dw 1.60, dx 1.51 (1.24 to 1.43 PFLOP/s of 2.1 TFLOP each, matrix cores busy for 62 to 76 % of
// the cycles; a large library product without any of the epilogues takes 1.55). With fewer slices a
// tile, or g in fp32, results and barriers show: 4096 x 50257 x 768 forward 284 us (1.11 PFLOP/s, busy
// for 49 %), eight workers' products 35 to 53 %. One token of
// 32000 x 768 takes 18 us, 49 MB at 3.4 TB/s in the kernel and a second one that joins.
// Where a product has few tiles, its k is split and a pass adds the parts.
#include "loss_tiles.h"

namespace sm {
namespace {

// ---------------------------------------------------------------------------
// Around the products
// ---------------------------------------------------------------------------
// BF16 planes of a matrix, rows padded to whole vectors with zeros; rows without
// a target are zeros where targets are given (what such a token holds, NaN too,
// reaches no gradient), and what g needs of each row is written beside them.
template <bool BF16>
__global__ __launch_bounds__(256) void loss_planes_kernel(LossPlanes f) {
    const int64_t vectors = f.pitch / 8, total = f.rows * vectors;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / vectors, c = (i - row * vectors) * 8;
        int have = left(f.cols, c);
        if (f.targets) {
            const int64_t t = f.targets64 ? static_cast<const int64_t *>(f.targets)[row]
                                          : static_cast<const int32_t *>(f.targets)[row];
            const bool there = t >= 0 && t < f.vocab;
            if (!there) have = 0;
            if (c == 0) {
                f.row_target[row] = there ? (int32_t)t : -1;
                f.row_base[row] = there ? f.lse[row] * kLog2E : 0.0f;
                f.row_d[row] = there ? f.scale * f.dloss[row] : 0.0f;
            }
        }
        float v[8];
        load_n<BF16>(f.in, row * f.cols + c, have, v);
        for (int p = 0; p < f.planes; ++p) {
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = to_bf16x2(v[2 * j], v[2 * j + 1]);
                // a value near the largest rounds to an infinity: its first plane is cut instead
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t bits = __float_as_uint(v[2 * j + h]);
                    const uint32_t mine = h ? w[j] >> 16 : w[j] & 0xffffu;
                    if ((mine & 0x7fffu) == 0x7f80u && (bits & 0x7fffffffu) < 0x7f800000u)
                        w[j] = h ? (w[j] & 0xffffu) | (bits & 0xffff0000u) : (w[j] & 0xffff0000u) | bits >> 16;
                    const float left_over = v[2 * j + h] - __uint_as_float(h ? w[j] & 0xffff0000u : w[j] << 16);
                    // infinities and NaN leave nothing
                    v[2 * j + h] = (bits & 0x7fffffffu) < 0x7f800000u ? left_over : 0.0f;
                }
            }
            *reinterpret_cast<u32x4 *>(f.out[p] + row * f.pitch + c) = w;
        }
    }
}

// Logits whose sums over k came in parts, added in order: a wave takes kLossBlock
// columns of a row, four a lane. Forward it leaves their maximum and sum, backward g.
template <bool GRAD, bool WIDE>
__global__ __launch_bounds__(256) void loss_parts_kernel(LossTile f) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t blocks = (f.n + kLossBlock - 1) / kLossBlock, part = f.m * f.out_pitch;
    for (int64_t i = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; i < f.m * blocks; i += (int64_t)gridDim.x * 4) {
        const int64_t row = i / blocks, block = i - row * blocks, col = block * kLossBlock + lane * 4;
        const int have = left(f.n, col) < 4 ? left(f.n, col) : 4;
        f32x4 l = {};
        if (have > 0) {
            const float *p = static_cast<const float *>(f.out) + row * f.out_pitch + col;
            for (int s = 0; s < f.splits; s += 8) {  // loads before sums
                f32x4 q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    q[j] = *reinterpret_cast<const f32x4 *>(p + (s + j < f.splits ? s + j : s) * part);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (s + j < f.splits) l += q[j];
            }
            // (of a token whose lse is no number, g is none either)
            if (f.plain_a && (!GRAD || fabsf(static_cast<const float *>(f.rows[1])[row]) < INFINITY))
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < have && l[j] != l[j]) l[j] = plain_logit(f, row, col + j);
        }
        const int32_t t = *reinterpret_cast<const int32_t *>(static_cast<const char *>(f.rows[0]) + row * f.row_step);
        const uint32_t at = (uint32_t)t - (uint32_t)(f.vocab0 + col);  // the target's place among the four
        if constexpr (GRAD) {
            const float base = static_cast<const float *>(f.rows[1])[row], d = static_cast<const float *>(f.rows[2])[row];
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = __builtin_amdgcn_exp2f(fmaf(l[j], f.factor, -base));
                v[j] = j < have && t >= 0 ? d * (at == (uint32_t)j ? p - 1.0f : p) : 0.0f;
            }
            if constexpr (WIDE)
                *reinterpret_cast<f32x4 *>(static_cast<float *>(f.g) + row * f.g_pitch + col) = f32x4{v[0], v[1], v[2], v[3]};
            else
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(f.g) + row * f.g_pitch + col) =
                    u32x2{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
        } else {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                l[j] = j < have ? l[j] * f.factor : -INFINITY;
                top = fmaxf(top, l[j]);
                // the low half of a target of 64 bits, as in the tiles
                if (at == (uint32_t)j && j < have) f.target[row] = l[j];
            }
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += __builtin_amdgcn_exp2f(l[j] - base);
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) sum += __shfl_xor(sum, d);
            if (lane == 0) f.partial[block * f.m + row] = make_float2(top, sum);
        }
    }
}

// The partial maxima and sums of f.group rows (a power of 2, up to 64): 1024 / group
// threads of a row take every so manieth block of columns, eight at a time, and
// are joined in a tree, with what earlier pieces of the vocabulary left.
__global__ __launch_bounds__(1024) void loss_join_kernel(LossJoin f) {
    __shared__ float2 lds[1024];
    const int slots = 1024 / f.group, slot = threadIdx.x / f.group;
    const int64_t row = (int64_t)blockIdx.x * f.group + threadIdx.x % f.group;
    const bool there = row < f.rows;
    float top = -INFINITY, sum = 0.0f;
    auto add = [&](float2 p) {
        const float m = fmaxf(top, p.x);
        // a sum of nothing stays one, whatever its maximum stands for
        sum = (sum == 0.0f ? 0.0f : sum * __builtin_amdgcn_exp2f(top - m)) +
              (p.y == 0.0f ? 0.0f : p.y * __builtin_amdgcn_exp2f(p.x - m));
        top = m;
    };
    if (there)
        for (int64_t b = slot; b < f.blocks; b += 8 * slots) {
            float2 p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = b + i * slots < f.blocks ? f.partial[(b + i * slots) * f.rows + row] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) add(p[i]);
        }
    for (int d = slots / 2; d > 0; d >>= 1) {
        lds[threadIdx.x] = make_float2(top, sum);
        __syncthreads();
        if (slot < d) add(lds[threadIdx.x + d * f.group]);
        __syncthreads();
    }
    if (slot || !there) return;
    if (!f.first) add(f.state[row]);
    if (!f.last) {
        f.state[row] = make_float2(top, sum);
        return;
    }
    const float lse2 = top + log2f(sum);
    if (f.lse) f.lse[row] = lse2 * kLn2;
    const int64_t t = f.targets64 ? static_cast<const int64_t *>(f.targets)[row] : static_cast<const int32_t *>(f.targets)[row];
    if (f.loss) f.loss[row] = t >= 0 && t < f.vocab ? (lse2 - f.target[row]) * kLn2 : 0.0f;
}

// out = the parts' sum, in order, and what `prev` holds; 4 entries a thread at a time.
__global__ __launch_bounds__(256) void loss_sums_kernel(LossSums f) {
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < f.total; at += (int64_t)gridDim.x * 1024) {
        const int have = (int)(f.total - at < 4 ? f.total - at : 4);
        float v[4] = {}, prev[4];
        if (f.prev_bf16)
            load_n<true>(f.prev, at, f.prev ? have : 0, prev);
        else
            load_n<false>(f.prev, at, f.prev ? have : 0, prev);
        for (int s = 0; s < f.splits; s += 8) {  // loads before sums
            float p[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) load_n<false>(f.partial, (s + i < f.splits ? s + i : s) * f.pitch + at, have, p[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (s + i < f.splits)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] += p[i][j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += prev[j];
        if (f.out_bf16)
            store_n<true>(f.out, at, have, v);
        else
            store_n<false>(f.out, at, have, v);
    }
}

}  // namespace

void launch_loss_planes(const LossPlanes &f, hipStream_t s) {
    const int64_t blocks = (f.rows * (f.pitch / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (f.bf16)
        loss_planes_kernel<true><<<grid, 256, 0, s>>>(f);
    else
        loss_planes_kernel<false><<<grid, 256, 0, s>>>(f);
}

void launch_loss_logits(const LossTile &f, bool grad, hipStream_t s) {
    if (f.splits > 1)
        launch_tiles<kRows16, kRows16, kValues, true>(f, s);
    else if (!grad)
        f.plain_a ? launch_tiles<kRows16, kRows16, kPlanesLse, true>(f, s) : launch_tiles<kRows16, kRows16, kLse, true>(f, s);
    else if (f.plain_a)
        f.g32 ? launch_tiles<kRows16, kRows16, kPlanesGrad, true>(f, s) : launch_tiles<kRows16, kRows16, kPlanesGrad, false>(f, s);
    else
        f.g32 ? launch_tiles<kRows16, kRows16, kGrad, true>(f, s) : launch_tiles<kRows16, kRows16, kGrad, false>(f, s);
}

void launch_loss_parts(const LossTile &f, bool grad, hipStream_t s) {
    const int64_t waves = f.m * ((f.n + kLossBlock - 1) / kLossBlock), blocks = (waves + 3) / 4;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (!grad)
        loss_parts_kernel<false, true><<<grid, 256, 0, s>>>(f);
    else if (f.g32)
        loss_parts_kernel<true, true><<<grid, 256, 0, s>>>(f);
    else
        loss_parts_kernel<true, false><<<grid, 256, 0, s>>>(f);
}

void launch_loss_join(LossJoin f, hipStream_t s) {
    // as few rows a workgroup as leave 256 of them
    for (f.group = 64; f.group > 1 && f.rows <= f.group / 2 * 256; f.group /= 2) {}
    loss_join_kernel<<<dim3((unsigned)((f.rows + f.group - 1) / f.group)), 1024, 0, s>>>(f);
}

void launch_loss_sums(const LossSums &f, hipStream_t s) {
    const int64_t blocks = (f.total + 1023) / 1024;
    loss_sums_kernel<<<dim3((unsigned)(blocks < 65536 ? blocks : 65536)), 256, 0, s>>>(f);
}

}  // namespace sm
