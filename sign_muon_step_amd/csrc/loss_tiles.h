// loss_tiles.h -- the matrix products of the output layer's loss and its gradients
// (linear_loss.hip has the formulas): tiles fed straight into LDS, and what becomes
// of their results. Not part of the public C ABI.
#pragma once

#include <type_traits>

#include "grad_internal.h"

namespace sm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kWaves = 4;

// ---------------------------------------------------------------------------
// Operands
// ---------------------------------------------------------------------------
// A slice of an operand lies in LDS as it does in memory:
//  - kRows16, kRows32: k runs along memory's rows, and a slice has 128 bytes of each,
//    whose 16-byte chunks are XOR-swizzled so that 16 consecutive rows' reads fall on all banks;
//  - kCols16: memory's rows are k, and a slice has TILE columns of each. They are
//    read by the instruction that transposes 4 x 16 values on the way; the 32-byte
//    segments are XOR-swizzled by the row, so that 4 rows' reads fall on all banks;
//  - kCols32: the same in fp32, read value by value; each 8 rows begin 128 bytes
//    further on, so that the two halves of a wave, 8 rows apart, read other banks.
enum { kRows16, kCols16, kRows32, kCols32 };

template <int KIND, int TILE, int SLICE>
struct Operand {
    static constexpr bool kTrans = KIND == kCols16 || KIND == kCols32;
    static constexpr int kSize = KIND == kRows16 || KIND == kCols16 ? 2 : 4;
    static constexpr int kLine = (kTrans ? TILE : SLICE) * kSize;  // bytes of a row in the slice
    static constexpr int kCount = kTrans ? SLICE : TILE;           // rows
    static constexpr int kPad = KIND == kCols32 ? 128 : 0;         // bytes behind each 8 rows
    static constexpr int kBytes = kCount * kLine + kCount / 8 * kPad;
    static constexpr int kRows = 1024 / kLine;                     // of a load
    static constexpr int kLoads = kCount / kRows / kWaves;         // per wave and slice
    static_assert(kTrans || kLine == 128, "whole lines");

    // A lane's place in a load: the wave's loads are kWaves * kRows rows apart, and the swizzle is the same in all.
    static __device__ __forceinline__ int row(int wave, int lane) { return wave * kRows + lane / (kWave / kRows); }
    static __device__ __forceinline__ int chunk(int wave, int lane) {
        const int r = row(wave, lane), c = lane & (kLine / 16 - 1);
        return KIND == kCols16 ? c ^ ((r & 3) << 2) : KIND == kCols32 ? c : c ^ ((r >> 1) & 7);
    }
    // Where load i of a wave lies, from the wave's first on.
    static constexpr int place(int i) { return i * kWaves * 1024 + i * kWaves * kRows / 8 * kPad; }

    // Block i of the wave's rows from w0 on, 16 k from 16 s on, of a slice in LDS: 8 k a lane.
    static __device__ __forceinline__ bf16x8 read(const char *slice, int w0, int i, int s, int lane) {
        if constexpr (KIND == kCols16) {
            const int l = lane & 15, g = lane >> 4;
            const int k = 16 * s + 8 * (g >> 1) + l / 4;  // and 4 more
            const int c = w0 / 8 + i * 4 + (g & 1) * 2 + (l & 3) / 2;
            const char *p = slice + k * kLine + ((c ^ ((l / 4) << 2)) << 4) + (l & 1) * 8;
            typedef __attribute__((address_space(3))) i16x4 *Lds;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * kLine));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int row = w0 + i * 32 + (lane & 31), c = 2 * s + (lane >> 5);
            return *reinterpret_cast<const bf16x8 *>(slice + row * kLine + ((c ^ ((row >> 1) & 7)) << 4));
        }
    }
    // The same of an fp32 operand, the lane's first or last 4 k.
    static __device__ __forceinline__ void read(const char *slice, int w0, int i, int s, int lane, int part, float (&v)[8]) {
        const int half = lane >> 5;
        if constexpr (KIND == kCols32) {
            const char *p = slice + (2 * s + half) * (8 * kLine + kPad) + (w0 + i * 32 + (lane & 31)) * 4;
#pragma unroll
            for (int j = 4 * part; j < 4 * part + 4; ++j) v[j] = *reinterpret_cast<const float *>(p + j * kLine);
        } else {
            const int row = w0 + i * 32 + (lane & 31), c = 4 * s + 2 * half + part;
            const f32x4 q = *reinterpret_cast<const f32x4 *>(slice + row * kLine + ((c ^ ((row >> 1) & 7)) << 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * part + j] = q[j];
        }
    }
};

// A tile of one batch entry and one part of k.
struct Tile {
    int64_t row0, col0, batch;
    int split;
};

template <int TM, int TN>
__device__ __forceinline__ Tile tile_at(const LossTile &f, int v, int total) {
    // batch and part of k, then tiles in bands of 8 rows of tiles, down the band
    // first: the tiles that run at once share operands in L2
    // (quotients come from vector code: first_lane brings them back to scalar)
    const int tm = (int)((f.m + TM - 1) / TM), tn = (int)((f.n + TN - 1) / TN);
    int t = xcd_run(v, total);
    const int per = tm * tn, unit = first_lane(t / per);
    t -= unit * per;
    const int band = first_lane(t / (8 * tn)), rows = tm - band * 8 < 8 ? tm - band * 8 : 8;
    t -= band * 8 * tn;
    const int col = first_lane(t / rows);
    Tile o;
    o.row0 = (int64_t)(band * 8 + t - col * rows) * TM;
    o.col0 = (int64_t)col * TN;
    const int batch = first_lane(unit / f.splits);
    o.batch = batch;
    o.split = unit - batch * f.splits;
    return o;
}

// The slices of a workgroup's tiles, one after the other, on their way into LDS:
// the pairs of planes of a tile, and the slices of k of a pair. A lane's offsets
// stay; a slice is a buffer's start and length. What lies outside an operand, and
// slices past the last tile's, lie beyond the length and give zeros. Columns past
// the last one of an operand whose rows are k hold what follows in memory, and end
// in results that are not kept. A tile's row data (ROWS arrays of 4 bytes a row)
// come with its first slice.
template <int KA, int KB, int TM, int TN, int SLICE, int STAGES, int ROWS>
struct Loader {
    using A = Operand<KA, TM, SLICE>;
    using B = Operand<KB, TN, SLICE>;
    static constexpr int kLoads = A::kLoads + B::kLoads, kStage = A::kBytes + B::kBytes, kStages = STAGES;
    // row data lie apart, in a set for each tile whose data may still be read, or under
    // way: with one slice a tile, the tile before and those of the next three slices
    static constexpr int kRowSets = 4, kRowSet = ROWS * TM * 4, kRowData = STAGES * kStage;
    static constexpr int kBytes = kRowData + kRowSets * kRowSet;
    u32x4 buffer[2];
    uint32_t at[2], past[2], step[2];  // of the lane's first load, where the slice's k ends; between loads
    int chunk[2];
    int v, slice, end;  // the tile, the next slice to load and the end of its slices
    int per, ks, pair;  // slices of a pair of planes; the slice's place in them
    unsigned tiles;     // so far
    Tile t;

    __device__ __forceinline__ void start(const LossTile &f, int v_, int total, uint32_t lds, int wave, int lane) {
        chunk[0] = A::chunk(wave, lane);
        chunk[1] = B::chunk(wave, lane);
        at[0] = (uint32_t)(A::row(wave, lane) * f.a_pitch + chunk[0] * 16);
        at[1] = (uint32_t)(B::row(wave, lane) * f.b_pitch + chunk[1] * 16);
        step[0] = (uint32_t)first_lane((int)(kWaves * A::kRows * f.a_pitch));
        step[1] = (uint32_t)first_lane((int)(kWaves * B::kRows * f.b_pitch));
        per = (int)((f.k + SLICE - 1) / SLICE);
        v = v_;
        tiles = 0;
        tile(f, total, lds, wave, lane);
    }
    __device__ __forceinline__ void tile(const LossTile &f, int total, uint32_t lds, int wave, int lane) {
        const bool there = v < total;
        t = tile_at<TM, TN>(f, there ? v : 0, total);
        slice = t.split * f.chunk;
        end = slice + f.chunk < f.pairs * per ? slice + f.chunk : f.pairs * per;
        pair = first_lane(slice / per);
        ks = slice - pair * per;
        place(f, there);
        const int have = (int)(f.m - t.row0 < TM ? f.m - t.row0 : TM);
        if (ROWS && wave * kWave < TM)
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                load4_lds(lds + kRowData + tiles % kRowSets * kRowSet + (uint32_t)(i * TM * 4 + wave * 256),
                          (uint32_t)((wave * kWave + lane) * f.row_step),
                          make_buffer(static_cast<const uint8_t *>(f.rows[i]) + t.row0 * f.row_step,
                                      there ? have * f.row_step : 0));
        ++tiles;
    }
    // A slice's buffer, from the slice's k on, and where its k ends.
    template <class O>
    __device__ __forceinline__ void operand(int o, const void *const (&planes)[kLossPlanes], uint32_t order,
                                            int64_t batch, int64_t pitch, int64_t first, int64_t rows, int64_t k,
                                            bool there) {
        const int plane = O::kSize == 4 ? 0 : order >> (2 * pair) & 3;  // fp32 operands have one
        const uint8_t *p = static_cast<const uint8_t *>(planes[plane]) + batch;
        const int64_t k0 = (int64_t)ks * SLICE;
        if (O::kTrans) {
            const int64_t have = k - k0 < SLICE ? k - k0 : SLICE;
            buffer[o] = make_buffer(p + k0 * pitch + first * O::kSize, there ? have * pitch - first * O::kSize : 0);
            past[o] = 0;
        } else {
            const int64_t have = rows - first < O::kCount ? rows - first : O::kCount;
            buffer[o] = make_buffer(p + first * pitch + k0 * O::kSize, there ? have * pitch - k0 * O::kSize : 0);
            past[o] = k0 + chunk[o] * (16 / O::kSize) < k ? 0u : kOutside;
        }
    }
    __device__ __forceinline__ void place(const LossTile &f, bool there) {
        operand<A>(0, f.a, f.order_a, t.batch * f.a_batch, f.a_pitch, t.row0, f.m, f.k, there);
        operand<B>(1, f.b, f.order_b, t.batch * f.b_batch, f.b_pitch, t.col0, f.n, f.k, there);
    }
    // The next slice of the same planes: the buffer's start moves on.
    template <class O>
    __device__ __forceinline__ void move(int o, int64_t pitch, int64_t k) {
        const uint32_t by = O::kTrans ? (uint32_t)(SLICE * pitch) : (uint32_t)(SLICE * O::kSize);
        const int left = (int)k - ks * SLICE;  // of k
        u32x4 &b = buffer[o];
        const uint32_t lo = b[0] + by;
        b[1] += lo < by ? 1u : 0u;
        b[0] = lo;
        if (O::kTrans)  // rows of this slice
            b[2] -= left < SLICE ? (uint32_t)((SLICE - left) * pitch) : 0u;
        else
            b[2] -= by;
#pragma unroll
        for (int i = 0; i < 3; ++i) b[i] = (uint32_t)first_lane((int)b[i]);  // it stays in scalar registers
        if (!O::kTrans) past[o] = chunk[o] * (16 / O::kSize) < left ? 0u : kOutside;
    }
    // Load i of the current slice to LDS; `to`: the wave's place in the slice's stage.
    __device__ __forceinline__ void issue(int i, uint32_t to) const {
        const int o = i < A::kLoads ? 0 : 1, r = o ? i - A::kLoads : i;
        load16_lds(to + (uint32_t)(o ? A::kBytes + B::place(r) : A::place(r)), (at[o] | past[o]) + (uint32_t)r * step[o],
                   buffer[o]);
    }
    // On to the next slice.
    __device__ __forceinline__ void advance(const LossTile &f, int total, uint32_t lds, int wave, int lane) {
        if (++slice == end) {
            v += gridDim.x;
            tile(f, total, lds, wave, lane);
        } else if (++ks == per) {
            ks = 0;
            ++pair;
            place(f, v < total);
        } else if (v < total) {
            move<A>(0, f.a_pitch, f.k);
            move<B>(1, f.b_pitch, f.k);
        }
    }
};

// Column of value e of a lane's block n, from the wave's first on.
__device__ __forceinline__ int column(int n, int e, int lane) { return n * 32 + e / 4 * 8 + (lane >> 5) * 4 + e % 4; }

// ---------------------------------------------------------------------------
// Results
// ---------------------------------------------------------------------------
template <int FM, int FN>
using Acc = f32x16[FM][FN];  // 32 x 32 blocks of a wave

template <int FM, int FN>
__device__ __forceinline__ void clear(Acc<FM, FN> &acc) {
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) acc[i / FN][i % FN] = zeros();
}

// The accumulators' values, four columns of a row at a time as group(i, n, q, v)
// makes them of block (i, n), to out as BF16 or fp32 (WIDE), through a wave's part of
// LDS so that whole lines are written. out: the wave's first entry, rows of `pitch`
// entries, of which `rows` and `cols` exist.
//  kEven    rows of whole vectors: buffer stores, which drop what lies outside;
//  kAdd     the same, added to what out holds (in fp32, rounded once);
//  kUneven  plain stores.
// A tile's results are some thousand instructions that run once, so that each branch
// among them is fetched every time: what does not change during a launch is a
// parameter (with branches inside, at eight workers' 1024 tokens, 50257 x 768, dw took
// 500 us a piece of 12800, and 420 without).
enum { kEven, kAdd, kUneven };
// How the stores go through the caches: g, of which a piece is larger than they are, as
// a stream (410 -> 395 us a piece of 25000 for eight workers, and 405 -> 370 for the dx that
// reads it next); results as usual (as a stream, dw took 3 % longer).
enum { kKept = 0, kStream = 2 };
constexpr int out_lds(int bytes) { return 32 * (bytes + 16); }  // of a wave; bytes: of a row at a time
// Buffer stores of a wave and tile.
constexpr int out_stores(int blocks, bool wide, int how) { return blocks * 32 * 32 * (wide || how == kAdd ? 4 : 2) / 1024; }

template <int FM, int FN, bool WIDE, int BYTES, int HOW, int CACHE, class G>
__device__ __forceinline__ void write(Acc<FM, FN> &acc, char *mine, void *out, int64_t pitch, int rows, int cols, int lane,
                                      G &&group) {
    constexpr bool STAGE32 = WIDE || HOW == kAdd;              // the values' type in LDS
    constexpr int S = STAGE32 ? 4 : 2, E = WIDE ? 4 : 2;       // bytes of a value there and in out
    constexpr int W = 16 / S, kCols = BYTES / S, kPitch = BYTES + 16;  // values of a store, columns at a time
    constexpr int kLanes = BYTES / 16, kRows = kWave / kLanes;  // lanes of a row, rows of a store
    static_assert(kCols % 8 == 0 && FN * 32 % kCols == 0, "whole passes");
    // made anew for each tile, so that no address is kept in registers meanwhile
    asm volatile("" : "+v"(lane));
    const int r0 = lane / kLanes, c16 = lane % kLanes, row = lane & 31, half = lane >> 5;
    rows = rows < 0 ? 0 : rows < FM * 32 ? rows : FM * 32;
    cols = cols < 0 ? 0 : cols < FN * 32 ? cols : FN * 32;
    const int step = (int)pitch * E;
    char *p = static_cast<char *>(out);
    const __amdgpu_buffer_rsrc_t buffer =
        __builtin_amdgcn_make_buffer_rsrc(p, 0, rows > 0 && cols > 0 ? (rows - 1) * step + cols * E : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int n0 = 0; n0 < FN * 32; n0 += kCols) {
            // no accumulator leaves its register before its turn
#pragma unroll
            for (int n = n0 / 32; n < (n0 + kCols + 31) / 32; ++n) pin(acc[i][n]);
            const uint32_t at = n0 + c16 * W < cols ? (uint32_t)(r0 * step + (n0 + c16 * W) * E) : kOutside;
            auto offset = [&](int r) { return (int)(at + (uint32_t)((i * 32 + r * kRows) * step)); };
            [[maybe_unused]] u32x4 held[32 / kRows];
            if constexpr (HOW == kAdd)
#pragma unroll
                for (int r = 0; r < 32 / kRows; ++r) {
                    if constexpr (WIDE) {
                        held[r] = __builtin_amdgcn_raw_buffer_load_b128(buffer, offset(r), 0, 0);
                    } else {
                        const u32x2 h = __builtin_amdgcn_raw_buffer_load_b64(buffer, offset(r), 0, 0);
                        held[r] = u32x4{h[0] << 16, h[0] & 0xffff0000u, h[1] << 16, h[1] & 0xffff0000u};
                    }
                }
#pragma unroll
            for (int n = n0; n < n0 + kCols; n += 8) {
                char *to = mine + row * kPitch + (n - n0 + half * 4) * S;
                float v[4];
                group(i, n / 32, n % 32 / 8, v);
                if constexpr (STAGE32)
                    *reinterpret_cast<f32x4 *>(to) = f32x4{v[0], v[1], v[2], v[3]};
                else
                    *reinterpret_cast<u32x2 *>(to) = u32x2{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
            }
            // lanes read what others wrote (LDS accesses of a wave keep their order)
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
            auto staged = [&](int r) { return *reinterpret_cast<const u32x4 *>(mine + (r * kRows + r0) * kPitch + c16 * 16); };
            if constexpr (HOW != kUneven) {
                u32x4 v[32 / kRows];
#pragma unroll
                for (int r = 0; r < 32 / kRows; ++r) v[r] = staged(r);
#pragma unroll
                for (int r = 0; r < 32 / kRows; ++r) {
                    if constexpr (HOW == kAdd)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[r][j] = __float_as_uint(__uint_as_float(v[r][j]) + __uint_as_float(held[r][j]));
                    if constexpr (HOW == kAdd && !WIDE)
                        __builtin_amdgcn_raw_buffer_store_b64(
                            u32x2{to_bf16x2(__uint_as_float(v[r][0]), __uint_as_float(v[r][1])),
                                  to_bf16x2(__uint_as_float(v[r][2]), __uint_as_float(v[r][3]))},
                            buffer, offset(r), 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b128(v[r], buffer, offset(r), 0, CACHE);
                }
            } else {
                const int here = cols - n0;  // columns from this pass's first on
#pragma unroll 1
                for (int r = 0; r < 32 / kRows; ++r)
                    if (i * 32 + r * kRows + r0 < rows && c16 * W + W <= here)
                        *reinterpret_cast<u32x4_any *>(p + (int64_t)(i * 32 + r * kRows + r0) * step + (n0 + c16 * W) * E) =
                            staged(r);
                // the last columns of a row, one by one
                if (here > 0 && here < kCols && i * 32 + row < rows && half == 0)
#pragma unroll 1
                    for (int c = here / W * W; c < here; ++c) {
                        char *q = p + (int64_t)(i * 32 + row) * step + (n0 + c) * E;
                        const char *from = mine + row * kPitch + c * E;
                        if constexpr (WIDE)
                            *reinterpret_cast<uint32_t *>(q) = *reinterpret_cast<const uint32_t *>(from);
                        else
                            *reinterpret_cast<uint16_t *>(q) = *reinterpret_cast<const uint16_t *>(from);
                    }
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
}

// A logit (over its scale) whose products of planes add up to no number, from the operands
// themselves. An operand's planes behind the first are nought or of either sign, and an infinity of
// the other, or a product past fp32's range, comes with each of them: a vocabulary entry that the weight
// sends to minus infinity would be no number, where the sum of the operands' own products is
// minus infinity. It is for few entries: 64 masked ones of 32000 take 8192 fp32 tokens of 1024
// columns, forward and backward, from 11.9 to 22.3 ms. Where a token's sum, or its lse, is no number
// whatever its other logits are, none is made.
__device__ __forceinline__ float plain_logit(const LossTile &f, int64_t row, int64_t col) {
    double sum = 0.0;
#pragma unroll 1
    for (int64_t k = 0; k < f.k && sum == sum; k += 8) {
        const int have = left((int)f.k, (int)k);
        float a[8], b[8];
        auto load = [&](const void *p, int64_t at, bool bf16, float(&v)[8]) {
            bf16 ? load_n<true>(p, at, have, v) : load_n<false>(p, at, have, v);
        };
        load(f.plain_a, row * f.k + k, f.plain_a16, a);
        load(f.plain_b, col * f.k + k, f.plain_b16, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma((double)a[j], (double)b[j], sum);
    }
    return (float)sum;
}

// A row's maximum and sum of exponentials over the wave's columns, and the target's
// logit, in units of log 2. PLANES: an operand is in several.
template <int FM, int FN, bool PLANES>
__device__ __forceinline__ void finish_lse(const LossTile &f, Acc<FM, FN> &acc, const char *targets, int64_t row0,
                                           int64_t col0, int lane) {
    constexpr int kRows = FM * 32, kCols = FN * 32;
    const int have = (int)(f.n - col0 < 0 ? 0 : f.n - col0 < kCols ? f.n - col0 : kCols);
    const int rows = (int)(f.m - row0 < 0 ? 0 : f.m - row0 < kRows ? f.m - row0 : kRows);
    // stores that are always issued, so that their number is known: what lies outside is dropped
    const __amdgpu_buffer_rsrc_t partial =
        __builtin_amdgcn_make_buffer_rsrc(f.partial + (col0 / kCols) * f.m + row0, 0, have > 0 ? rows * 8 : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int row = i * 32 + (lane & 31);
        // the low half of a target of 64 bits: one outside the vocabulary may seem to be inside, and its
        // logit is not used
        const uint32_t at = *reinterpret_cast<const uint32_t *>(targets + row * 4) - (uint32_t)(f.vocab0 + col0);
        const int target = at < (uint32_t)have && row < rows ? (int)at : -1;
        float l[FN][16], top = -INFINITY;
#pragma unroll
        for (int n = 0; n < FN; ++n) {
            pin(acc[i][n]);
#pragma unroll
            for (int e = 0; e < 16; ++e) l[n][e] = acc[i][n][e] * f.factor;
        }
        if (have < kCols)
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) l[n][e] = column(n, e, lane) < have ? l[n][e] : -INFINITY;
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
            for (int e = 0; e < 16; e += 2) top = fmaxf(fmaxf(l[n][e], l[n][e + 1]), top);
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(target >= 0)) {
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (column(n, e, lane) == target) f.target[row0 + row] = l[n][e];
        }
        const float base = top == -INFINITY ? 0.0f : top;  // a block of minus infinities adds nothing
        float sum[2] = {};
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e & 1] += __builtin_amdgcn_exp2f(l[n][e] - base);
        sum[0] += sum[1];
        if constexpr (PLANES)
            if (__any(sum[0] != sum[0])) {  // as it stays where the operands hold NaN, or the logit is infinite
                uint64_t bad = 0;
                sum[0] = 0.0f;
                int lane1 = lane;  // made anew here, as what follows from it
                asm volatile("" : "+v"(lane1));
#pragma unroll
                for (int n = 0; n < FN; ++n) {
                    pin(acc[i][n]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float v = column(n, e, lane1) < have ? acc[i][n][e] * f.factor : -INFINITY;
                        bad |= v != v && row < rows ? 1ull << (n * 16 + e) : 0ull;
                        sum[0] += v != v ? 0.0f : __builtin_amdgcn_exp2f(v - base);
                    }
                }
                // (a sum that is no number stays none)
#pragma unroll 1
                for (; bad && sum[0] == sum[0]; bad &= bad - 1) {
                    const int at = __builtin_ctzll(bad), col = column(at / 16, at % 16, lane1);
                    const float v = plain_logit(f, row0 + row, col0 + col) * f.factor, most = fmaxf(top, v);
                    if (col == target) f.target[row0 + row] = v;
                    if (v == -INFINITY) continue;
                    sum[0] = (sum[0] == 0.0f ? 0.0f : sum[0] * __builtin_amdgcn_exp2f(top - most)) +
                             __builtin_amdgcn_exp2f(v - most);
                    top = most;
                }
                const float other = __shfl_xor(top, 32), most = fmaxf(top, other);
                sum[0] = sum[0] == 0.0f ? 0.0f : sum[0] * __builtin_amdgcn_exp2f(top - most);
                top = most;
            }
        sum[0] += __shfl_xor(sum[0], 32);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(top), __float_as_uint(sum[0])}, partial,
                                              lane < 32 ? row * 8 : (int)kOutside, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
    clear<FM, FN>(acc);
}

// g; zeros in the columns past the vocabulary that a tile has. PLANES: an operand is in several.
template <int FM, int FN, bool WIDE, bool PLANES>
__device__ __forceinline__ void finish_grad(const LossTile &f, Acc<FM, FN> &acc, char *mine, const char *data, int64_t row0,
                                            int64_t col0, int lane) {
    constexpr int kRows = FM * 32, kCols = FN * 32;
    const int have = (int)(f.n - col0 < 0 ? 0 : f.n - col0 < kCols ? f.n - col0 : kCols);
    int target[FM], limit[FM];  // of the lane's rows: the target's column, and the columns that count
    float d[FM], base[FM];
    bool any = false, whole = true;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        // the rows' targets (-1: none), lse / log 2 and scale * dloss
        const char *p = data + (i * 32 + (lane & 31)) * 4;
        const int t = *reinterpret_cast<const int *>(p);
        base[i] = *reinterpret_cast<const float *>(p + 2 * kRows * 4);
        d[i] = *reinterpret_cast<const float *>(p + 4 * kRows * 4);
        const uint32_t at = (uint32_t)t - (uint32_t)(f.vocab0 + col0);
        target[i] = t >= 0 && at < (uint32_t)have ? (int)at : -1;
        // a token without a target has no gradient, whatever its logits are
        limit[i] = t >= 0 ? have : 0;
        any |= target[i] >= 0;
        whole &= limit[i] == kCols;
    }
    auto put = [&](auto &&group) {
        write<FM, FN, WIDE, FN * 32, kEven, kStream>(acc, mine, static_cast<char *>(f.g) + (row0 * f.g_pitch + col0) * (WIDE ? 4 : 2),
                                     f.g_pitch, (int)(f.m - row0 < kRows ? f.m - row0 : kRows), kCols, lane, group);
    };
    auto exponential = [&](int i, int n, int e) {
        return __builtin_amdgcn_exp2f(fmaf(acc[i][n][e], f.factor, -base[i]));
    };
    float check = 0.0f;  // no number if one of the values is none, or infinite
    [[maybe_unused]] auto watch = [&](float v) {
        check = fmaf(v, 0.0f, check);
        asm volatile("" : "+v"(check));  // here, while v is in a register
    };
    if (__all(whole && !any))
        put([&](int i, int n, int q, float(&v)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = d[i] * exponential(i, n, q * 4 + j);
                if constexpr (PLANES) watch(v[j]);
            }
        });
    else
        put([&](int i, int n, int q, float(&v)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = column(n, q * 4 + j, lane);
                const float p = exponential(i, n, q * 4 + j);
                v[j] = c < limit[i] ? d[i] * (c == target[i] ? p - 1.0f : p) : 0.0f;
                if constexpr (PLANES) watch(v[j]);
            }
        });
    if constexpr (PLANES)
        if (__any(check != check)) {
            wait_loads<0>();  // the wave reads what it wrote
            const int rows = (int)(f.m - row0 < kRows ? f.m - row0 : kRows);
#pragma unroll 1
            for (int at = lane; at < rows * kCols; at += kWave) {
                const int row = at / kCols, col = at % kCols;
                const int t = *reinterpret_cast<const int *>(data + row * 4);
                const int64_t entry = (row0 + row) * f.g_pitch + col0 + col;
                const float b = *reinterpret_cast<const float *>(data + (row + 2 * kRows) * 4);
                const float times = *reinterpret_cast<const float *>(data + (row + 4 * kRows) * 4);
                float v = load1<!WIDE>(f.g, entry);
                // (of a token whose loss is no number, neither are its gradients)
                if (v == v || t < 0 || col >= have || (b - b) + (times - times) != 0.0f) continue;
                v = __builtin_amdgcn_exp2f(fmaf(plain_logit(f, row0 + row, col0 + col), f.factor, -b));
                if (t - f.vocab0 - col0 == col) v -= 1.0f;
                store1<!WIDE>(f.g, entry, v * times);
            }
        }
    clear<FM, FN>(acc);
}

// A product's values, added to what out holds where f.add.
template <int FM, int FN, bool WIDE, int BYTES, int HOW>
__device__ __forceinline__ void finish_values(const LossTile &f, Acc<FM, FN> &acc, char *mine, const Tile &t, int64_t row0,
                                              int64_t col0, int lane) {
    const int64_t first = (f.out_batch * (t.split * (int64_t)f.batch + t.batch) + row0) * f.out_pitch + col0;
    const int rows = (int)(f.m - row0 < FM * 32 ? f.m - row0 : FM * 32), cols = (int)(f.out_pitch - col0 < FN * 32 ? f.out_pitch - col0 : FN * 32);
    write<FM, FN, WIDE, BYTES, HOW, kKept>(acc, mine, static_cast<char *>(f.out) + first * (WIDE ? 4 : 2), f.out_pitch, rows, cols, lane,
                               [&](int i, int n, int q, float(&v)[4]) {
#pragma unroll
                                   for (int j = 0; j < 4; ++j) v[j] = acc[i][n][q * 4 + j];
                                   if (HOW != kUneven || !f.add) return;
                                   const int row = i * 32 + (lane & 31), col = column(n, q * 4, lane);
                                   const int have = row >= rows ? 0 : left(cols, col) < 4 ? left(cols, col) : 4;
                                   float p[4];
                                   load_n<!WIDE>(f.out, first + row * f.out_pitch + col, have, p);
#pragma unroll
                                   for (int j = 0; j < 4; ++j) v[j] += p[j];
                               });
    clear<FM, FN>(acc);
}

constexpr std::integral_constant<int, 0> kLow{};
constexpr std::integral_constant<int, 1> kHigh{};

// Nothing behind this runs before v is in its registers.
__device__ __forceinline__ void hold(const bf16x8 &v) { asm volatile("" : : "v"(v) : "memory"); }

// The place of slice c's loads of a wave. Opaque: each load adds its constant to
// this, where the compiler would keep every sum in a scalar register of its own and
// run out of them.
template <class L>
__device__ __forceinline__ uint32_t stage_of(uint32_t lds, unsigned c, int wave) {
    uint32_t to = lds + c % L::kStages * L::kStage + (uint32_t)wave * 1024u;
    asm volatile("" : "+s"(to));
    return to;
}

enum { kLse, kGrad, kValues, kPlanesLse, kPlanesGrad };  // kPlanes..: of an operand in several planes

// Products of BF16 operands. A workgroup takes every gridDim-th tile; four waves of
// half a tile each way. The loads run two slices ahead of the products, on into the
// next tile, so that a tile's first slices are there when the one before it is done.
// WIDE: results in fp32. HOW: of values.
template <int KA, int KB, int TM, int TN, int END, bool WIDE, int HOW>
__global__ __launch_bounds__(kWaves *kWave, TM *TN > 128 * 128 ? 1 : 2) void loss_tile_kernel(LossTile f, int total) {
    constexpr bool kIsLse = END == kLse || END == kPlanesLse, kIsGrad = END == kGrad || END == kPlanesGrad;
    constexpr int kRowArrays = kIsLse ? 1 : kIsGrad ? 3 : 0;
    using L = Loader<KA, KB, TM, TN, kLossSlice, 2, kRowArrays>;
    using A = typename L::A;
    using B = typename L::B;
    constexpr int FM = TM / 64, FN = TN / 64;
    constexpr int kOut = L::kBytes, kOutWave = kIsLse ? 0 : out_lds(FN * 32);
    __shared__ __attribute__((aligned(1024))) char lds[kOut + kWaves * kOutWave];
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)lds);
    const int wm = wave / 2 * (TM / 2), wn = wave % 2 * (TN / 2);

    L loader;
    loader.start(f, blockIdx.x, total, lds0, wave, lane);
#pragma unroll 1
    for (unsigned c = 0; c < L::kStages; ++c) {
        const uint32_t to = stage_of<L>(lds0, c, wave);
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i) loader.issue(i, to);
        loader.advance(f, total, lds0, wave, lane);
    }

    // The fragments of half a slice (32 k) in registers, b's FN and a's FM, 16 k each.
    constexpr int kBlocks = FN + FM, kReads = 2 * kBlocks, kSteps = 2 * FM * FN;
    bf16x8 fr[2][2][kBlocks];  // [half][16 k][block]
    auto read = [&](auto h, unsigned c, int r) {  // of half h of slice c
        constexpr int H = decltype(h)::value;
        const char *stage = lds + c % L::kStages * L::kStage;
        const int s = r / kBlocks, i = r % kBlocks;
        fr[H][s][i] = i < FN ? B::read(stage + A::kBytes, wn, i, 2 * H + s, lane) : A::read(stage, wm, i - FN, 2 * H + s, lane);
    };
    f32x16 acc[FM][FN];
    clear<FM, FN>(acc);
    // The products of half a slice, from the registers, a step for each; extra(step)
    // is what else the step issues, so that the matrix pipe does not wait behind a
    // run of reads or loads.
    auto products = [&](auto h, auto extra) {
        constexpr int H = decltype(h)::value;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const int s = t / (FM * FN), i = t % (FM * FN) / FN, n = t % FN;
            extra(t);
            acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[H][s][n], fr[H][s][FN + i], acc[i][n], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    wait_loads<L::kLoads>();  // slice 0
    barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(kLow, 0, r);

    // Steps of the low half: the reads of the high half, two a step, then at step
    // kMeet all waves have read slice c and slice c + 1 has landed, so that slice c + 2
    // is loaded to slice c's place from there on, a load every kSpread steps, and
    // slice c + 1 may be read. Few loads at a time: at 8192 x 32000 x 4096 the four
    // products take 7.1 ms so, 7.2 with a load every second step and 7.6 with one
    // each step.
    constexpr int kMeet = kReads / 2 + 2, kSpread = (2 * kSteps - kMeet) / L::kLoads;
    static_assert(kMeet < kSteps && kSpread > 0, "room for the reads and loads");
    auto steps = [&](auto h, unsigned c, uint32_t to, int s, int gone) {
#pragma unroll
        for (int r = 2 * s; r < 2 * s + 2; ++r)
            if (r < kReads) read(h, c, r);
        if (s + gone >= kMeet && (s + gone - kMeet) % kSpread == 0 && (s + gone - kMeet) / kSpread < L::kLoads)
            loader.issue((s + gone - kMeet) / kSpread, to);
    };
    // A tile's results are on their way to memory during the next one's first slice:
    // there, only what is older than their stores is waited for.
    constexpr int kStores = kIsLse ? FM : out_stores(FM * FN, WIDE, HOW), kBehind = kStores < 63 ? kStores : 63;
    bool behind = false;  // of buffer stores, whose number is known
    const int per = loader.per;
    unsigned c = 0;  // slices so far
    // `newer`: operations that may be under way behind the loads of slice c + 1
    auto slice = [&](auto newer) {
        const uint32_t to = stage_of<L>(lds0, c, wave);
        products(kLow, [&](int s) {
            if (s == kMeet) {
#pragma unroll
                for (int r = 0; r < kReads; ++r) hold(fr[1][r / kBlocks][r % kBlocks]);
                wait_loads<decltype(newer)::value>();
                barrier();
            }
            steps(kHigh, c, to, s, 0);
        });
        products(kHigh, [&](int s) { steps(kLow, c + 1, to, s, kSteps); });
#pragma unroll
        for (int i = 0; i < FM * FN; ++i) pin(acc[i / FN][i % FN]);
        loader.advance(f, total, lds0, wave, lane);
        ++c;
    };
    unsigned tile = 0;
#pragma unroll 1
    for (int v = blockIdx.x; v < total; v += gridDim.x, ++tile) {
        const Tile t = tile_at<TM, TN>(f, v, total);
        int j = t.split * f.chunk;
        const int end = j + f.chunk < f.pairs * per ? j + f.chunk : f.pairs * per;
        if (behind) {
            slice(std::integral_constant<int, kBehind>{});
            ++j;
        }
#pragma unroll 1
        for (; j < end; ++j) slice(kLow);
        char *mine = lds + kOut + wave * kOutWave;
        const char *data = lds + L::kRowData + tile % L::kRowSets * L::kRowSet + wm * 4;
        if constexpr (kIsLse)
            finish_lse<FM, FN, END == kPlanesLse>(f, acc, data, t.row0 + wm, t.col0 + wn, lane);
        else if constexpr (kIsGrad)
            finish_grad<FM, FN, WIDE, END == kPlanesGrad>(f, acc, mine, data, t.row0 + wm, t.col0 + wn, lane);
        else
            finish_values<FM, FN, WIDE, FN * 32, HOW>(f, acc, mine, t, t.row0 + wm, t.col0 + wn, lane);
        behind = HOW != kUneven;
    }
    wait_loads<0>();  // loads past the last tile write LDS too
}

// Products of an fp32 a, taken apart into planes in registers, and a BF16 b. PLANES:
// of a; 1 for each plane of b, or 3 for its first, 2 for its second and 1 for its third. A slice
// is 32 k: while 16 of them are multiplied, the next 16 are read and taken apart.
template <int KA, int TM, int TN, int PLANES, bool WIDE, int HOW>
__global__ __launch_bounds__(kWaves *kWave, TM *TN > 128 * 128 ? 1 : 2) void loss_wide_kernel(LossTile f, int total) {
    using L = Loader<KA, kCols16, TM, TN, kLossWideSlice, 3, 0>;
    using A = typename L::A;
    using B = typename L::B;
    constexpr int FM = TM / 64, FN = TN / 64;
    constexpr int kOut = L::kBytes, kOutBytes = FN * 16;
    __shared__ __attribute__((aligned(1024))) char lds[kOut + kWaves * out_lds(kOutBytes)];
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)lds);
    const int wm = wave / 2 * (TM / 2), wn = wave % 2 * (TN / 2);

    L loader;
    loader.start(f, blockIdx.x, total, lds0, wave, lane);
#pragma unroll 1
    for (unsigned c = 0; c < L::kStages; ++c) {
        const uint32_t to = stage_of<L>(lds0, c, wave);
#pragma unroll
        for (int i = 0; i < L::kLoads; ++i) loader.issue(i, to);
        loader.advance(f, total, lds0, wave, lane);
    }

    unsigned c = 0;  // slices so far
    float raw[FM][8];
    u32x4 plane[2][PLANES][FM];  // [half][plane][block]
    bf16x8 fb[2][FN];
    // Reads: a's blocks in two parts, then b's.
    auto read = [&](auto h, unsigned c, int r) {  // of half h of slice c
        constexpr int H = decltype(h)::value;
        const char *stage = lds + c % L::kStages * L::kStage;
        if (r < 2 * FM)
            A::read(stage, wm, r / 2, H, lane, r % 2, raw[r / 2]);
        else
            fb[H][r - 2 * FM] = B::read(stage + A::kBytes, wn, r - 2 * FM, H, lane);
    };
    constexpr int kReads = 2 * FM + FN, kParts = 4 * FM * PLANES;
    // A plane of two values of a block; what it leaves stays in their place.
    auto part = [&](auto h, int p) {
        constexpr int H = decltype(h)::value;
        const int q = p % PLANES, i = p / PLANES / 4, j = p / PLANES % 4;
        const uint32_t w = to_bf16x2(raw[i][2 * j], raw[i][2 * j + 1]);
        plane[H][q][i][j] = w;
        if (q + 1 < PLANES) {
            raw[i][2 * j] -= __uint_as_float(w << 16);
            raw[i][2 * j + 1] -= __uint_as_float(w & 0xffff0000u);
        }
    };
    f32x16 acc[FM][FN];
    clear<FM, FN>(acc);
    wait_loads<2 * L::kLoads>();  // slice 0
    barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(kLow, 0, r);
#pragma unroll
    for (int p = 0; p < kParts; ++p) part(kLow, p);

    // As above: the reads of the next 16 k first, then, at kMeet of the low half, the
    // slice's place is free for the loads of the one three on; the reads' values are
    // taken apart from kMeet on, a plane of two of them at a time.
    constexpr int kRound = FM * FN;
    auto half = [&](auto planes, auto h, auto newer, uint32_t to) {
        constexpr int N = decltype(planes)::value, H = decltype(h)::value, kSteps = N * kRound;
        constexpr int kPerRead = N == 1 ? 2 : 1, kMeet = kReads / kPerRead + (kRound > 4 ? 2 : 0);
        static_assert(kMeet < kSteps, "room for the reads");
        // the loads: from kMeet of the low half to the end of the high one
        constexpr int kRest = 2 * kSteps - kMeet, kSpread = kRest / L::kLoads > 0 ? kRest / L::kLoads : 1;
        constexpr int kPerLoad = (L::kLoads + kRest - 1) / kRest;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (s == kMeet && H == 0) {
#pragma unroll
                for (int i = 0; i < FN; ++i) hold(fb[1][i]);
#pragma unroll
                for (int i = 0; i < 8 * FM; ++i) asm volatile("" : : "v"(raw[i / 8][i % 8]) : "memory");
                wait_loads<decltype(newer)::value>();
                barrier();
            }
#pragma unroll
            for (int r = s * kPerRead; r < (s + 1) * kPerRead; ++r)
                if (r < kReads) {
                    if (H == 0)
                        read(kHigh, c, r);
                    else
                        read(kLow, c + 1, r);
                }
            const int g = s + H * kSteps - kMeet;  // steps since the loads may begin
            if (g >= 0 && g % kSpread == 0)
#pragma unroll
                for (int i = g / kSpread * kPerLoad; i < (g / kSpread + 1) * kPerLoad; ++i)
                    if (i < L::kLoads) loader.issue(i, to);
            if (s >= kMeet)
#pragma unroll
                for (int p = (s - kMeet) * kParts / (kSteps - kMeet); p < (s + 1 - kMeet) * kParts / (kSteps - kMeet); ++p) {
                    if (H == 0)
                        part(kHigh, p);
                    else
                        part(kLow, p);
                }
            const int q = s / kRound, i = s % kRound / FN, n = s % FN;
            acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[H][n], __builtin_bit_cast(bf16x8, plane[H][q][i]),
                                                                acc[i][n], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int kStores = L::kLoads + out_stores(FM * FN, WIDE, HOW), kBehind = kStores < 63 ? kStores : 63;
    bool behind = false;
    auto slice = [&](auto planes, auto newer) {
        const uint32_t to = stage_of<L>(lds0, c, wave);
        half(planes, kLow, newer, to);
        half(planes, kHigh, newer, to);
#pragma unroll
        for (int i = 0; i < FM * FN; ++i) pin(acc[i / FN][i % FN]);
        loader.advance(f, total, lds0, wave, lane);
        ++c;
    };
    const int per = loader.per;
#pragma unroll 1
    for (int v = blockIdx.x; v < total; v += gridDim.x) {
        const Tile t = tile_at<TM, TN>(f, v, total);
        int j = t.split * f.chunk;
        const int end = j + f.chunk < f.pairs * per ? j + f.chunk : f.pairs * per;
        constexpr std::integral_constant<int, L::kLoads> kNext{};  // slice c + 2's
        auto slices = [&](auto planes, int stop) {
            if (behind && j < stop) {
                slice(planes, std::integral_constant<int, kBehind>{});
                behind = false;
                ++j;
            }
#pragma unroll 1
            for (; j < stop; ++j) slice(planes, kNext);
        };
        if constexpr (PLANES == 3) {
            slices(std::integral_constant<int, 3>{}, end < per ? end : per);
            slices(std::integral_constant<int, 2>{}, end < 2 * per ? end : 2 * per);
        }
        slices(std::integral_constant<int, 1>{}, end);
        finish_values<FM, FN, WIDE, kOutBytes, HOW>(f, acc, lds + kOut + wave * out_lds(kOutBytes), t, t.row0 + wm,
                                               t.col0 + wn, lane);
        behind = HOW != kUneven;
    }
    wait_loads<0>();  // loads past the last tile write LDS too
}

int tiles_of(const LossTile &f) {
    return (int)((f.m + f.tm - 1) / f.tm * ((f.n + f.tn - 1) / f.tn) * f.batch * f.splits);
}

// One workgroup a compute unit (tiles of 128 x 128: two), a multiple of the XCDs.
dim3 grid_of(const LossTile &f) {
    const int total = tiles_of(f), most = device_cus() / 8 * 8 * (f.tm * f.tn > 128 * 128 ? 1 : 2);
    return dim3((unsigned)(total < most ? total : most));
}

template <int KA, int KB, int END, bool WIDE, int HOW = kEven>
void launch_tiles(const LossTile &f, hipStream_t s) {
    const dim3 grid = grid_of(f);
    const int total = tiles_of(f), threads = kWaves * kWave;
    if constexpr (HOW != kUneven) {
        if (f.tn == 256) {
            loss_tile_kernel<KA, KB, 256, 256, END, WIDE, HOW><<<grid, threads, 0, s>>>(f, total);
            return;
        }
        if (f.tm == 256) {
            loss_tile_kernel<KA, KB, 256, 128, END, WIDE, HOW><<<grid, threads, 0, s>>>(f, total);
            return;
        }
    }
    loss_tile_kernel<KA, KB, 128, 128, END, WIDE, HOW><<<grid, threads, 0, s>>>(f, total);
}

template <int KA, int PLANES, bool WIDE, int HOW>
void launch_wide(const LossTile &f, hipStream_t s) {
    const dim3 grid = grid_of(f);
    const int total = tiles_of(f), threads = kWaves * kWave;
    if constexpr (HOW != kUneven) {
        if (f.tm == 256) {
            loss_wide_kernel<KA, 256, 256, PLANES, WIDE, HOW><<<grid, threads, 0, s>>>(f, total);
            return;
        }
        if (f.tn == 256) {
            loss_wide_kernel<KA, 128, 256, PLANES, WIDE, HOW><<<grid, threads, 0, s>>>(f, total);
            return;
        }
    }
    loss_wide_kernel<KA, 128, 128, PLANES, WIDE, HOW><<<grid, threads, 0, s>>>(f, total);
}

}  // namespace
}  // namespace sm
