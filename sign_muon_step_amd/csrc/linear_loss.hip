// linear_loss.hip -- softmax cross entropy of an output layer, and its
// gradients, on the gfx950 matrix cores.
//
//   l[t][v] = scale x[t].w[v],  lse[t] = log sum_v exp l[t][v],  loss[t] = lse[t] - l[t][target]
//   g[t][v] = scale dloss[t] (exp(l[t][v] - lse[t]) - [v = target]),  dx = g w,  dw_m = g_m^T x_m
//
// No logit leaves the chip. Forward, each tile of logits becomes one running
// maximum and one sum of exponentials a row and 128 columns, which are joined
// afterwards. Backward, the logits of a piece of the vocabulary are computed
// again and stored as g, from which that piece's dw and its share of dx are two
// more products; then the next piece overwrites it.
//
// Everything is a product of BF16 operands on v_mfma_f32_32x32x16_bf16 with
// fp32 sums. An fp32 operand is taken apart into BF16 planes, h + m + l, each the
// rounding of what the ones before it left: three planes hold its 24 bits. A
// product of planes is a longer sum: the pairs (h h), (h m), (m h), (m m),
// (h l), (l h) leave out parts below 2^-22 of the operands' product (6e-9 of a sum of
// random ones). Six BF16 products run at 2.6 times the rate of fp32's own matrix
// instruction. Logits take all planes of their operands. g and the operands of dx
// and dw take two planes, and the pairs (h h), (h m), (m h), where the result is
// fp32, which is off by up to 2^-16 of each factor (3e-6 of a sum of random
// products; an exponential of an fp32 logit of 16 is off by 1e-6 itself), and one
// plane where the result is BF16, whose own rounding is as large.
//
// The products are computed as b a^T: the instruction's rows are out's columns,
// so that a lane's accumulators hold four consecutive columns of one row of out,
// and a row of logits lies in two lanes.
#include "grad_internal.h"

namespace sm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kTile = kLossTile, kWaves = 4, kSlice = kLossSlice;
constexpr int kOperand = kTile * kSlice * 2, kStage = 2 * kOperand, kStages = 2;  // bytes of LDS
constexpr int kLoads = kOperand / 1024 / kWaves;  // per wave, slice and operand
constexpr int kBlocks = 4;                        // 32 x 32 blocks of a wave, each way

// ---------------------------------------------------------------------------
// Operands
// ---------------------------------------------------------------------------
// A slice of an operand lies in LDS as it does in memory:
//  - rows of 64 k (TRANS = false: k runs along memory's rows), 128 bytes, whose
//    16-byte chunks are XOR-swizzled so that 16 consecutive rows' reads fall on all banks;
//  - 64 rows of 256 columns (TRANS = true: memory's rows are k), 512 bytes, read
//    by the instruction that transposes 4 x 16 values on the way; its 32-byte
//    segments are XOR-swizzled by the row, so that 4 rows' reads fall on all banks.
template <bool TRANS>
struct Operand {
    uint32_t at[kLoads];  // of a lane's loads from the slice's start
    int chunk;            // TRANS = false: of the lane's loads, along k

    __device__ __forceinline__ void start(int64_t pitch, int wave, int lane) {
        chunk = (lane & 7) ^ ((wave * 4 + lane / 16) & 7);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (TRANS) {
                const int row = (i * kWaves + wave) * 2 + lane / 32;
                at[i] = (uint32_t)(row * pitch + (((lane & 31) ^ ((row & 3) << 2)) << 4));
            } else {
                const int row = (i * kWaves + wave) * 8 + lane / 8;
                at[i] = (uint32_t)(row * pitch + (chunk << 4));
            }
        }
    }
    // The loads of slice `ks` of a plane: `first` and `have` are the tile's first
    // row (TRANS: column) of the operand and the rows of it that exist, k the
    // operand's whole length. What lies outside is zero; TRANS: columns past the
    // last one hold what follows in memory, and end in results that are not kept.
    __device__ __forceinline__ void load(const uint16_t *plane, int64_t pitch, int64_t first, int64_t have, int64_t k,
                                         int64_t ks, uint32_t to) const {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(plane);
        const int64_t k0 = ks * kSlice;
        u32x4 buffer;
        uint32_t past = 0;
        if (TRANS) {
            const int64_t rows = k - k0 < kSlice ? k - k0 : kSlice;
            buffer = make_buffer(p + k0 * pitch + first * 2, rows * pitch - first * 2);
        } else {
            buffer = make_buffer(p + first * pitch + k0 * 2, have * pitch - k0 * 2);
            past = k0 + chunk * 8 < k ? 0u : kOutside;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load16_lds(to + (uint32_t)(i * kWaves * 1024), at[i] | past, buffer);
    }
    // Block i of the wave's 128 rows from w0 on, 16 k from 16 s on, of a slice in LDS.
    static __device__ __forceinline__ bf16x8 read(const char *slice, int w0, int i, int s, int lane) {
        if (TRANS) {
            const int l = lane & 15, g = lane >> 4;
            const int k = 16 * s + 8 * (g >> 1) + l / 4;  // and 4 more
            const int chunk = w0 / 8 + i * 4 + (g & 1) * 2 + (l & 3) / 2;
            const char *p = slice + k * (kTile * 2) + ((chunk ^ ((l / 4) << 2)) << 4) + (l & 1) * 8;
            typedef __attribute__((address_space(3))) i16x4 *Lds;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * kTile * 2));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        const int row = w0 + i * 32 + (lane & 31), chunk = 2 * s + (lane >> 5);
        return *reinterpret_cast<const bf16x8 *>(slice + row * (kSlice * 2) + ((chunk ^ ((row >> 1) & 7)) << 4));
    }
};

// A tile of one batch entry and one part of k.
struct Tile {
    int64_t row0, col0, batch;
    int split;
};

__device__ __forceinline__ Tile tile_at(const LossTile &f, int v, int total) {
    // batch and part of k, then tiles in bands of 8 rows of tiles, down the band
    // first: the tiles that run at once share operands in L2
    // (quotients come from vector code: first_lane brings them back to scalar)
    const int tm = (int)((f.m + kTile - 1) / kTile), tn = (int)((f.n + kTile - 1) / kTile);
    int t = xcd_run(v, total);
    const int per = tm * tn, unit = first_lane(t / per);
    t -= unit * per;
    const int band = first_lane(t / (8 * tn)), rows = tm - band * 8 < 8 ? tm - band * 8 : 8;
    t -= band * 8 * tn;
    const int col = first_lane(t / rows);
    Tile o;
    o.row0 = (int64_t)(band * 8 + t - col * rows) * kTile;
    o.col0 = (int64_t)col * kTile;
    const int batch = first_lane(unit / f.splits);
    o.batch = batch;
    o.split = unit - batch * f.splits;
    return o;
}

__device__ __forceinline__ int64_t target_of(const LossTile &f, int64_t row) {
    return f.targets64 ? static_cast<const int64_t *>(f.targets)[row] : static_cast<const int32_t *>(f.targets)[row];
}

// Column of value e of a lane's block n, from the wave's first on.
__device__ __forceinline__ int column(int n, int e, int lane) { return n * 32 + e / 4 * 8 + (lane >> 5) * 4 + e % 4; }

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
// A row's maximum and sum of exponentials over the wave's 128 columns, and the
// target's logit, in units of log 2.
__device__ __forceinline__ void finish_lse(const LossTile &f, const f32x16 (&acc)[kBlocks][kBlocks], int64_t row0,
                                           int64_t col0, int lane) {
    if (col0 >= f.n) return;
    const int have = (int)(f.n - col0 < 128 ? f.n - col0 : 128);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int64_t row = row0 + i * 32 + (lane & 31);
        float l[kBlocks][16], top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                l[n][e] = acc[i][n][e] * f.factor;
                if (have < 128 && column(n, e, lane) >= have) l[n][e] = -INFINITY;
                top = fmaxf(top, l[n][e]);
            }
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -INFINITY ? 0.0f : top;  // a block of minus infinities adds nothing
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum += __builtin_amdgcn_exp2f(l[n][e] - base);
        sum += __shfl_xor(sum, 32);
        const bool there = row < f.m;
        if (there && lane < 32) f.partial[(col0 / 128) * f.m + row] = make_float2(top, sum);
        const int64_t target = there ? target_of(f, row) - f.vocab0 - col0 : -1;
        const bool here = target >= 0 && target < have;
        if (__any(here)) {
#pragma unroll
            for (int n = 0; n < kBlocks; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (here && column(n, e, lane) == (int)target) f.target[row] = l[n][e];
        }
    }
}

// g, in one or two planes; zeros in columns past the vocabulary.
__device__ __forceinline__ void finish_grad(const LossTile &f, const f32x16 (&acc)[kBlocks][kBlocks], int64_t row0,
                                            int64_t col0, int lane) {
    const int have = (int)(f.n - col0 < 0 ? 0 : f.n - col0 < 128 ? f.n - col0 : 128);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int64_t row = row0 + i * 32 + (lane & 31);
        if (row >= f.m) continue;
        const int64_t target = target_of(f, row);
        const bool there = target >= 0 && target < f.vocab;
        // a token without a target has no gradient, whatever its logits are
        const float d = there ? f.scale * f.dloss[row] : 0.0f, base = f.lse[row] * kLog2E;
        const int64_t local = target - f.vocab0 - col0;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = column(n, q * 4 + j, lane);
                    const float p = __builtin_amdgcn_exp2f(fmaf(acc[i][n][q * 4 + j], f.factor, -base));
                    v[j] = there && c < have ? d * (p - (c == local ? 1.0f : 0.0f)) : 0.0f;
                }
                const int64_t at = row * f.g_pitch + col0 + column(n, q * 4, lane);
                const u32x2 h = {to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
                *reinterpret_cast<u32x2 *>(f.g[0] + at) = h;
                if (f.g[1]) {
                    const float r[4] = {v[0] - __uint_as_float(h[0] << 16), v[1] - __uint_as_float(h[0] & 0xffff0000u),
                                        v[2] - __uint_as_float(h[1] << 16), v[3] - __uint_as_float(h[1] & 0xffff0000u)};
                    *reinterpret_cast<u32x2 *>(f.g[1] + at) = u32x2{to_bf16x2(r[0], r[1]), to_bf16x2(r[2], r[3])};
                }
            }
    }
}

// A product's values, added to what `prev` holds.
__device__ __forceinline__ void finish_values(const LossTile &f, const f32x16 (&acc)[kBlocks][kBlocks], int64_t row0,
                                              int64_t col0, int64_t first, int lane) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int64_t row = row0 + i * 32 + (lane & 31);
        if (row >= f.m) continue;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t col = col0 + column(n, q * 4, lane), at = (first + row) * f.n + col;
                const int have = (int)(f.n - col < 0 ? 0 : f.n - col < 4 ? f.n - col : 4);
                float v[4], p[4];
                if (f.prev_bf16)
                    load_n<true>(f.prev, at, f.prev ? have : 0, p);
                else
                    load_n<false>(f.prev, at, f.prev ? have : 0, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = acc[i][n][q * 4 + j] + p[j];
                if (f.out_bf16)
                    store_n<true>(f.out, at, have, v);
                else
                    store_n<false>(f.out, at, have, v);
            }
    }
}

enum { kLse, kGrad, kValues };

// A workgroup takes every gridDim-th tile; four waves of 128 x 128. Slices of 64 k
// stream straight into LDS, the next one while a slice is multiplied.
template <bool TA, bool TB, int END>
__global__ __launch_bounds__(kWaves *kWave) void loss_tile_kernel(LossTile f, int total) {
    __shared__ __attribute__((aligned(1024))) char lds[kStages * kStage];
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)lds);
    const int wm = wave / 2 * 128, wn = wave % 2 * 128;
    Operand<TA> a;
    Operand<TB> b;
    a.start(f.a_pitch, wave, lane);
    b.start(f.b_pitch, wave, lane);
    const int per = (int)((f.k + kSlice - 1) / kSlice);  // slices of a pair of planes
    for (int v = blockIdx.x; v < total; v += gridDim.x) {
        const Tile t = tile_at(f, v, total);
        const int begin = t.split * f.chunk;
        const int end = begin + f.chunk < f.pairs * per ? begin + f.chunk : f.pairs * per;
        const int64_t have_a = f.m - t.row0 < kTile ? f.m - t.row0 : kTile;
        const int64_t have_b = f.n - t.col0 < kTile ? f.n - t.col0 : kTile;
        auto load = [&](int c) {
            const int pair = first_lane(c / per), ks = c - pair * per;
            const uint32_t to = lds0 + (uint32_t)(c % kStages * kStage + wave * 1024);
            const char *pa = reinterpret_cast<const char *>(f.a[f.plane_a[pair]]) + t.batch * f.a_batch;
            const char *pb = reinterpret_cast<const char *>(f.b[f.plane_b[pair]]) + t.batch * f.b_batch;
            a.load(reinterpret_cast<const uint16_t *>(pa), f.a_pitch, t.row0, have_a, f.k, ks, to);
            b.load(reinterpret_cast<const uint16_t *>(pb), f.b_pitch, t.col0, have_b, f.k, ks, to + kOperand);
        };
        f32x16 acc[kBlocks][kBlocks];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int n = 0; n < kBlocks; ++n) acc[i][n] = zeros();
        load(begin);
        for (int c = begin; c < end; ++c) {
            wait_loads<0>();
            barrier();  // slice c is there, and every wave is done with slice c - 1
            if (c + 1 < end) load(c + 1);
            const char *slice = lds + c % kStages * kStage;
#pragma unroll
            for (int s = 0; s < kSlice / 16; ++s) {
                bf16x8 fa[kBlocks], fb[kBlocks];
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) fa[i] = Operand<TA>::read(slice, wm, i, s, lane);
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) fb[i] = Operand<TB>::read(slice + kOperand, wn, i, s, lane);
#pragma unroll
                for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                    for (int n = 0; n < kBlocks; ++n)
                        acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[n], fa[i], acc[i][n], 0, 0, 0);
            }
        }
        barrier();  // every wave is done with the last slice before the next tile's first is loaded
        if constexpr (END == kLse)
            finish_lse(f, acc, t.row0 + wm, t.col0 + wn, lane);
        else if constexpr (END == kGrad)
            finish_grad(f, acc, t.row0 + wm, t.col0 + wn, lane);
        else
            finish_values(f, acc, t.row0 + wm, t.col0 + wn, f.out_batch * (t.split * (int64_t)f.batch + t.batch), lane);
    }
}

// ---------------------------------------------------------------------------
// Around the products
// ---------------------------------------------------------------------------
// BF16 planes of a matrix, rows padded to whole vectors with zeros; rows without
// a target are zeros where targets are given (what such a token holds, NaN too,
// reaches no gradient).
template <bool BF16>
__global__ __launch_bounds__(256) void loss_planes_kernel(LossPlanes f) {
    const int64_t vectors = f.pitch / 8, total = f.rows * vectors;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / vectors, c = (i - row * vectors) * 8;
        int have = left(f.cols, c);
        if (f.targets) {
            const int64_t t = f.targets64 ? static_cast<const int64_t *>(f.targets)[row]
                                          : static_cast<const int32_t *>(f.targets)[row];
            if (t < 0 || t >= f.vocab) have = 0;
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

// The partial maxima and sums of 64 rows: 16 waves take every 16th block of
// columns, and the first joins them, with what earlier pieces of the vocabulary
// left.
__global__ __launch_bounds__(1024) void loss_join_kernel(LossJoin f) {
    __shared__ float2 lds[16][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t row = (int64_t)blockIdx.x * kWave + lane;
    float top = -INFINITY, sum = 0.0f;
    auto add = [&](float2 p) {
        const float m = fmaxf(top, p.x);
        // a sum of nothing stays one, whatever its maximum stands for
        sum = (sum == 0.0f ? 0.0f : sum * __builtin_amdgcn_exp2f(top - m)) +
              (p.y == 0.0f ? 0.0f : p.y * __builtin_amdgcn_exp2f(p.x - m));
        top = m;
    };
    if (row < f.rows)
        for (int64_t b = wave; b < f.blocks; b += 16) add(f.partial[b * f.rows + row]);
    lds[wave][lane] = make_float2(top, sum);
    __syncthreads();
    if (wave || row >= f.rows) return;
    for (int w = 1; w < 16; ++w) add(lds[w][lane]);
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

// out = the parts' sums, in order, added to what `prev` holds; 4 entries a thread.
__global__ __launch_bounds__(256) void loss_sums_kernel(LossSums f) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= f.total) return;
    const int have = (int)(f.total - at < 4 ? f.total - at : 4);
    float v[4];
    load_n<false>(f.prev, at, f.prev ? have : 0, v);
    for (int s = 0; s < f.splits; ++s) {
        float p[4];
        load_n<false>(f.partial, s * f.total + at, have, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += p[j];
    }
    if (f.out_bf16)
        store_n<true>(f.out, at, have, v);
    else
        store_n<false>(f.out, at, have, v);
}

template <bool TA, bool TB, int END>
void launch_tiles(const LossTile &f, hipStream_t s) {
    const int64_t tiles = (f.m + kTile - 1) / kTile * ((f.n + kTile - 1) / kTile) * f.batch * f.splits;
    const int total = (int)tiles, most = device_cus() / 8 * 8;
    loss_tile_kernel<TA, TB, END><<<dim3((unsigned)(total < most ? total : most)), kWaves * kWave, 0, s>>>(f, total);
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
    grad ? launch_tiles<false, false, kGrad>(f, s) : launch_tiles<false, false, kLse>(f, s);
}

void launch_loss_join(const LossJoin &f, hipStream_t s) {
    loss_join_kernel<<<dim3((unsigned)((f.rows + kWave - 1) / kWave)), 1024, 0, s>>>(f);
}

void launch_loss_dx(const LossTile &f, hipStream_t s) { launch_tiles<false, true, kValues>(f, s); }
void launch_loss_dw(const LossTile &f, hipStream_t s) { launch_tiles<true, true, kValues>(f, s); }

void launch_loss_sums(const LossSums &f, hipStream_t s) {
    loss_sums_kernel<<<dim3((unsigned)((f.total + 1023) / 1024)), 256, 0, s>>>(f);
}

}  // namespace sm
