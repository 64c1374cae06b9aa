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
#include <type_traits>

#include "grad_internal.h"

namespace sm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kWaves = 4, kSlice = kLossSlice, kStages = 2;

// ---------------------------------------------------------------------------
// Operands
// ---------------------------------------------------------------------------
// A slice of an operand lies in LDS as it does in memory:
//  - rows of 64 k (TRANS = false: k runs along memory's rows), 128 bytes, whose
//    16-byte chunks are XOR-swizzled so that 16 consecutive rows' reads fall on all banks;
//  - 64 rows of TILE columns (TRANS = true: memory's rows are k), read by the
//    instruction that transposes 4 x 16 values on the way; its 32-byte segments are
//    XOR-swizzled by the row, so that 4 rows' reads fall on all banks.
template <bool TRANS, int TILE>
struct Operand {
    static constexpr int kBytes = TILE * kSlice * 2;
    static constexpr int kLoads = kBytes / 1024 / kWaves;  // per wave and slice
    static constexpr int kRowBytes = TRANS ? TILE * 2 : kSlice * 2;
    static constexpr int kRows = 1024 / kRowBytes;         // of a load

    // A lane's place in a load: the wave's loads are kWaves * kRows rows apart, and the swizzle is the same in all.
    static __device__ __forceinline__ int row(int wave, int lane) { return wave * kRows + lane / (kWave / kRows); }
    static __device__ __forceinline__ int chunk(int wave, int lane) {
        const int r = row(wave, lane), c = lane & (kRowBytes / 16 - 1);
        return TRANS ? c ^ ((r & 3) << 2) : c ^ ((r >> 1) & 7);
    }
    // Block i of the wave's rows from w0 on, 16 k from 16 s on, of a slice in LDS.
    static __device__ __forceinline__ bf16x8 read(const char *slice, int w0, int i, int s, int lane) {
        if (TRANS) {
            const int l = lane & 15, g = lane >> 4;
            const int k = 16 * s + 8 * (g >> 1) + l / 4;  // and 4 more
            const int c = w0 / 8 + i * 4 + (g & 1) * 2 + (l & 3) / 2;
            const char *p = slice + k * kRowBytes + ((c ^ ((l / 4) << 2)) << 4) + (l & 1) * 8;
            typedef __attribute__((address_space(3))) i16x4 *Lds;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * kRowBytes));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        const int row = w0 + i * 32 + (lane & 31), c = 2 * s + (lane >> 5);
        return *reinterpret_cast<const bf16x8 *>(slice + row * kRowBytes + ((c ^ ((row >> 1) & 7)) << 4));
    }
};

// A tile of one batch entry and one part of k.
struct Tile {
    int64_t row0, col0, batch;
    int split;
};

template <int TILE>
__device__ __forceinline__ Tile tile_at(const LossTile &f, int v, int total) {
    // batch and part of k, then tiles in bands of 8 rows of tiles, down the band
    // first: the tiles that run at once share operands in L2
    // (quotients come from vector code: first_lane brings them back to scalar)
    const int tm = (int)((f.m + TILE - 1) / TILE), tn = (int)((f.n + TILE - 1) / TILE);
    int t = xcd_run(v, total);
    const int per = tm * tn, unit = first_lane(t / per);
    t -= unit * per;
    const int band = first_lane(t / (8 * tn)), rows = tm - band * 8 < 8 ? tm - band * 8 : 8;
    t -= band * 8 * tn;
    const int col = first_lane(t / rows);
    Tile o;
    o.row0 = (int64_t)(band * 8 + t - col * rows) * TILE;
    o.col0 = (int64_t)col * TILE;
    const int batch = first_lane(unit / f.splits);
    o.batch = batch;
    o.split = unit - batch * f.splits;
    return o;
}

// The slices of a workgroup's tiles, one after the other, on their way into LDS:
// the pairs of planes of a tile, and the slices of k of a pair. A lane's offsets
// stay; a slice is a buffer's start and length. What lies outside an operand, and
// slices past the last tile's, lie beyond the length and give zeros. TRANS: columns
// past the last one hold what follows in memory, and end in results that are not
// kept.
template <bool TA, bool TB, int TILE>
struct Loader {
    using A = Operand<TA, TILE>;
    using B = Operand<TB, TILE>;
    static constexpr int kLoads = A::kLoads + B::kLoads, kStage = A::kBytes + B::kBytes;
    u32x4 buffer[2];
    uint32_t at[2], past[2], step[2];  // of the lane's first load, where the slice's k ends; between loads
    int chunk[2];
    int v, slice, end;  // the tile, the next slice to load and the end of its slices
    int per, ks, pair;  // slices of a pair of planes; the slice's place in them
    Tile t;

    __device__ __forceinline__ void start(const LossTile &f, int v_, int total, int wave, int lane) {
        chunk[0] = A::chunk(wave, lane);
        chunk[1] = B::chunk(wave, lane);
        at[0] = (uint32_t)(A::row(wave, lane) * f.a_pitch + chunk[0] * 16);
        at[1] = (uint32_t)(B::row(wave, lane) * f.b_pitch + chunk[1] * 16);
        step[0] = (uint32_t)first_lane((int)(kWaves * A::kRows * f.a_pitch));
        step[1] = (uint32_t)first_lane((int)(kWaves * B::kRows * f.b_pitch));
        per = (int)((f.k + kSlice - 1) / kSlice);
        v = v_;
        tile(f, total);
    }
    __device__ __forceinline__ void tile(const LossTile &f, int total) {
        const bool there = v < total;
        t = tile_at<TILE>(f, there ? v : 0, total);
        slice = t.split * f.chunk;
        end = slice + f.chunk < f.pairs * per ? slice + f.chunk : f.pairs * per;
        pair = first_lane(slice / per);
        ks = slice - pair * per;
        place(f, there);
    }
    // A slice's buffer, from the slice's k on, and where its k ends.
    template <bool TRANS>
    __device__ __forceinline__ void operand(int o, const uint16_t *const (&planes)[kLossPlanes], uint32_t order,
                                            int64_t batch, int64_t pitch, int64_t first, int64_t rows, int64_t k,
                                            bool there) {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(planes[order >> (2 * pair) & 3]) + batch;
        const int64_t k0 = (int64_t)ks * kSlice;
        if (TRANS) {
            const int64_t have = k - k0 < kSlice ? k - k0 : kSlice;
            buffer[o] = make_buffer(p + k0 * pitch + first * 2, there ? have * pitch - first * 2 : 0);
            past[o] = 0;
        } else {
            const int64_t have = rows - first < TILE ? rows - first : TILE;
            buffer[o] = make_buffer(p + first * pitch + k0 * 2, there ? have * pitch - k0 * 2 : 0);
            past[o] = k0 + chunk[o] * 8 < k ? 0u : kOutside;
        }
    }
    __device__ __forceinline__ void place(const LossTile &f, bool there) {
        operand<TA>(0, f.a, f.order_a, t.batch * f.a_batch, f.a_pitch, t.row0, f.m, f.k, there);
        operand<TB>(1, f.b, f.order_b, t.batch * f.b_batch, f.b_pitch, t.col0, f.n, f.k, there);
    }
    // The next slice of the same planes: the buffer's start moves on.
    template <bool TRANS>
    __device__ __forceinline__ void move(int o, int64_t pitch, int64_t k) {
        const uint32_t by = TRANS ? (uint32_t)(kSlice * pitch) : (uint32_t)(kSlice * 2);
        const int left = (int)k - ks * kSlice;  // of k
        u32x4 &b = buffer[o];
        const uint32_t lo = b[0] + by;
        b[1] += lo < by ? 1u : 0u;
        b[0] = lo;
        if (TRANS)  // rows of this slice
            b[2] -= left < kSlice ? (uint32_t)((kSlice - left) * pitch) : 0u;
        else
            b[2] -= by;
#pragma unroll
        for (int i = 0; i < 3; ++i) b[i] = (uint32_t)first_lane((int)b[i]);  // it stays in scalar registers
        if (!TRANS) past[o] = chunk[o] * 8 < left ? 0u : kOutside;
    }
    // Load i of the current slice to LDS; `to`: the wave's place in the slice's stage.
    __device__ __forceinline__ void issue(int i, uint32_t to) const {
        const int o = i < A::kLoads ? 0 : 1, r = o ? i - A::kLoads : i;
        load16_lds(to + (uint32_t)(o * A::kBytes + r * kWaves * 1024), (at[o] | past[o]) + (uint32_t)r * step[o], buffer[o]);
    }
    // On to the next slice.
    __device__ __forceinline__ void advance(const LossTile &f, int total) {
        if (++slice == end) {
            v += gridDim.x;
            tile(f, total);
        } else if (++ks == per) {
            ks = 0;
            ++pair;
            place(f, v < total);
        } else if (v < total) {
            move<TA>(0, f.a_pitch, f.k);
            move<TB>(1, f.b_pitch, f.k);
        }
    }
};

__device__ __forceinline__ int64_t target_of(const LossTile &f, int64_t row) {
    return f.targets64 ? static_cast<const int64_t *>(f.targets)[row] : static_cast<const int32_t *>(f.targets)[row];
}

// Column of value e of a lane's block n, from the wave's first on.
__device__ __forceinline__ int column(int n, int e, int lane) { return n * 32 + e / 4 * 8 + (lane >> 5) * 4 + e % 4; }

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
template <int F>
using Acc = f32x16[F][F];

// A row's maximum and sum of exponentials over the wave's columns, and the target's
// logit, in units of log 2.
template <int F>
__device__ __forceinline__ void finish_lse(const LossTile &f, Acc<F> &acc, int64_t row0, int64_t col0, int lane) {
    constexpr int kCols = F * 32;
    if (col0 < f.n) {
        const int have = (int)(f.n - col0 < kCols ? f.n - col0 : kCols);
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int64_t row = row0 + i * 32 + (lane & 31);
            const bool there = row < f.m;
            const int64_t target = (there ? target_of(f, row) : -1) - f.vocab0 - col0;
            float l[F][16], top = -INFINITY;
#pragma unroll
            for (int n = 0; n < F; ++n) {
                pin(acc[i][n]);
#pragma unroll
                for (int e = 0; e < 16; ++e) l[n][e] = acc[i][n][e] * f.factor;
            }
            if (have < kCols)
#pragma unroll
                for (int n = 0; n < F; ++n)
#pragma unroll
                    for (int e = 0; e < 16; ++e) l[n][e] = column(n, e, lane) < have ? l[n][e] : -INFINITY;
#pragma unroll
            for (int n = 0; n < F; ++n)
#pragma unroll
                for (int e = 0; e < 16; e += 2) top = fmaxf(fmaxf(l[n][e], l[n][e + 1]), top);
            top = fmaxf(top, __shfl_xor(top, 32));
            const bool here = target >= 0 && target < have;
            if (__any(here)) {
#pragma unroll
                for (int n = 0; n < F; ++n)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (here && column(n, e, lane) == (int)target) f.target[row] = l[n][e];
            }
            const float base = top == -INFINITY ? 0.0f : top;  // a block of minus infinities adds nothing
            float sum[2] = {};
#pragma unroll
            for (int n = 0; n < F; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[e & 1] += __builtin_amdgcn_exp2f(l[n][e] - base);
            sum[0] += sum[1];
            sum[0] += __shfl_xor(sum[0], 32);
            if (there && lane < 32) f.partial[(col0 / kCols) * f.m + row] = make_float2(top, sum[0]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int i = 0; i < F * F; ++i) acc[i / F][i % F] = zeros();
}

// g, in one or two planes; zeros in columns past the vocabulary.
template <int F>
__device__ __forceinline__ void finish_grad(const LossTile &f, Acc<F> &acc, int64_t row0, int64_t col0, int lane) {
    constexpr int kCols = F * 32;
    const int have = (int)(f.n - col0 < 0 ? 0 : f.n - col0 < kCols ? f.n - col0 : kCols);
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int64_t row = row0 + i * 32 + (lane & 31);
        const bool in = row < f.m;
        const int64_t target = in ? target_of(f, row) : -1;
        const bool there = target >= 0 && target < f.vocab;
        // a token without a target has no gradient, whatever its logits are
        const float d = there ? f.scale * f.dloss[row] : 0.0f, base = in ? f.lse[row] * kLog2E : 0.0f;
        const int64_t local = target - f.vocab0 - col0;
        const bool any = __any(there && local >= 0 && local < kCols);
#pragma unroll
        for (int n = 0; n < F; ++n) {
            pin(acc[i][n]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = column(n, q * 4 + j, lane);
                    const float p = __builtin_amdgcn_exp2f(fmaf(acc[i][n][q * 4 + j], f.factor, -base));
                    v[j] = there && c < have ? d * (any && c == local ? p - 1.0f : p) : 0.0f;
                }
                if (!in) continue;
                const int64_t at = row * f.g_pitch + col0 + column(n, q * 4, lane);
                const u32x2 h = {to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
                *reinterpret_cast<u32x2 *>(f.g[0] + at) = h;
                if (f.g[1]) {
                    const float r[4] = {v[0] - __uint_as_float(h[0] << 16), v[1] - __uint_as_float(h[0] & 0xffff0000u),
                                        v[2] - __uint_as_float(h[1] << 16), v[3] - __uint_as_float(h[1] & 0xffff0000u)};
                    *reinterpret_cast<u32x2 *>(f.g[1] + at) = u32x2{to_bf16x2(r[0], r[1]), to_bf16x2(r[2], r[3])};
                }
            }
            acc[i][n] = zeros();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// A product's values, added to what `prev` holds.
template <int F>
__device__ __forceinline__ void finish_values(const LossTile &f, Acc<F> &acc, int64_t row0, int64_t col0, int64_t first,
                                              int lane) {
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int64_t row = row0 + i * 32 + (lane & 31);
#pragma unroll
        for (int n = 0; n < F; ++n) {
            pin(acc[i][n]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t col = col0 + column(n, q * 4, lane), at = (first + row) * f.n + col;
                const int have = (int)(row >= f.m || f.n - col < 0 ? 0 : f.n - col < 4 ? f.n - col : 4);
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
            acc[i][n] = zeros();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

enum { kLse, kGrad, kValues };

// A workgroup takes every gridDim-th tile; four waves of half a tile each way. The
// loads run two slices ahead of the products, on into the next tile, so that a
// tile's first slices are there when the one before it is done.
template <bool TA, bool TB, int TILE, int END>
__global__ __launch_bounds__(kWaves *kWave) void loss_tile_kernel(LossTile f, int total) {
    using L = Loader<TA, TB, TILE>;
    using A = typename L::A;
    using B = typename L::B;
    constexpr int F = TILE / 64;  // 32 x 32 blocks of a wave, each way
    __shared__ __attribute__((aligned(1024))) char lds[kStages * L::kStage];
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)lds);
    const int wm = wave / 2 * (TILE / 2), wn = wave % 2 * (TILE / 2);

    L loader;
    loader.start(f, blockIdx.x, total, wave, lane);
    auto place = [&](unsigned c) {
        uint32_t to = lds0 + c % kStages * L::kStage + (uint32_t)wave * 1024u;
        // opaque: each load adds its constant to this, where the compiler would
        // keep every sum in a scalar register of its own and run out of them
        asm volatile("" : "+s"(to));
        return to;
    };
#pragma unroll 1
    for (unsigned c = 0; c < kStages; ++c) {
        const uint32_t to = place(c);
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i) loader.issue(i, to);
        loader.advance(f, total);
    }

    // The fragments of half a slice (32 k) in registers, b's F and a's F, 16 k each.
    constexpr int kReads = 4 * F, kSteps = 2 * F * F;
    bf16x8 fr[2][2][2 * F];  // [half][16 k][block]
    auto read = [&](auto h, unsigned c, int r) {  // of half h of slice c
        constexpr int H = decltype(h)::value;
        const char *stage = lds + c % kStages * L::kStage;
        const int s = r / (2 * F), i = r % (2 * F);
        fr[H][s][i] = i < F ? B::read(stage + A::kBytes, wn, i, 2 * H + s, lane) : A::read(stage, wm, i - F, 2 * H + s, lane);
    };
    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F * F; ++i) acc[i / F][i % F] = zeros();
    // The products of half a slice, from the registers, a step for each; extra(step)
    // is what else the step issues, so that the matrix pipe does not wait behind a
    // run of reads or loads.
    auto products = [&](auto h, auto extra) {
        constexpr int H = decltype(h)::value;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const int s = t / (F * F), i = t % (F * F) / F, n = t % F;
            extra(t);
            acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[H][s][n], fr[H][s][F + i], acc[i][n], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::integral_constant<int, 0> kLow{};
    constexpr std::integral_constant<int, 1> kHigh{};
    wait_loads<L::kLoads>();  // slice 0
    barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(kLow, 0, r);

    // Steps of the low half: the reads of the high half in the first half of them,
    // then at step kMeet all waves have read slice c and slice c + 1 has landed, so
    // that slice c + 2 is loaded to slice c's place from there on, and slice c + 1
    // may be read.
    constexpr int kMeet = kSteps * 5 / 8, kPerRead = kReads * 2 / kSteps, kPerLoad = L::kLoads * 2 / kSteps;
    static_assert(kPerRead * kSteps == 2 * kReads && kPerLoad * kSteps == 2 * L::kLoads, "whole steps");
    auto load_step = [&](uint32_t to, int s) {  // s: steps from kMeet on
#pragma unroll
        for (int i = s * kPerLoad; i < (s + 1) * kPerLoad; ++i)
            if (i < L::kLoads) loader.issue(i, to);
    };
    const int per = loader.per;
    unsigned c = 0;  // slices so far
#pragma unroll 1
    for (int v = blockIdx.x; v < total; v += gridDim.x) {
        const Tile t = tile_at<TILE>(f, v, total);
        const int begin = t.split * f.chunk;
        const int end = begin + f.chunk < f.pairs * per ? begin + f.chunk : f.pairs * per;
#pragma unroll 1
        for (int j = begin; j < end; ++j, ++c) {
            const uint32_t to = place(c);
            products(kLow, [&](int s) {
#pragma unroll
                for (int r = s * kPerRead; r < (s + 1) * kPerRead; ++r)
                    if (r < kReads) read(kHigh, c, r);
                if (s == kMeet) {
#pragma unroll
                    for (int r = 0; r < kReads; ++r) asm volatile("" : : "v"(fr[1][r / (2 * F)][r % (2 * F)]) : "memory");
                    wait_loads<0>();
                    barrier();
                }
                if (s >= kMeet) load_step(to, s - kMeet);
            });
            products(kHigh, [&](int s) {
#pragma unroll
                for (int r = s * kPerRead; r < (s + 1) * kPerRead; ++r)
                    if (r < kReads) read(kLow, c + 1, r);
                load_step(to, kSteps - kMeet + s);
            });
#pragma unroll
            for (int i = 0; i < F * F; ++i) pin(acc[i / F][i % F]);
            loader.advance(f, total);
        }
        if constexpr (END == kLse)
            finish_lse<F>(f, acc, t.row0 + wm, t.col0 + wn, lane);
        else if constexpr (END == kGrad)
            finish_grad<F>(f, acc, t.row0 + wm, t.col0 + wn, lane);
        else
            finish_values<F>(f, acc, t.row0 + wm, t.col0 + wn, f.out_batch * (t.split * (int64_t)f.batch + t.batch), lane);
    }
    wait_loads<0>();  // loads past the last tile write LDS too
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
    constexpr int TILE = kLossTile;
    const int64_t tiles = (f.m + TILE - 1) / TILE * ((f.n + TILE - 1) / TILE) * f.batch * f.splits;
    const int total = (int)tiles, most = device_cus() / 8 * 8;
    loss_tile_kernel<TA, TB, TILE, END><<<dim3((unsigned)(total < most ? total : most)), kWaves * kWave, 0, s>>>(f, total);
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
