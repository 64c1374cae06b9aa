// f8_matmul.hip -- products of 8-bit floating point operands with a
// power-of-two scale for each block of 128, on the gfx950 matrix cores.
//
//   out[r][c] = sum over blocks b of 2^(ea[r][b] + eb[c][b]) sum over k in b of a[r][k] b[c][k]
//
// Two forms of the product, chosen by out's type:
//  BF16  v_mfma_scale_f32_*_f8f6f4 on the bytes themselves. It takes a scale
//        byte per lane, i.e. per row and 32 values, and applies 2^(byte - 127)
//        itself: a block's byte serves the instructions of its 128 values, and
//        no accumulator is touched in between. Before it adds in fp32 it cuts
//        the products of each 8 consecutive k below 2^-13 of the power of two
//        of the largest one (seen with one large and one small product, at
//        every distance and place): 1.4e-5 of a sum of random products, far
//        below BF16's 2^-8.
//  F32   the bytes are converted to BF16 with their scale (exact: 4 bits of
//        mantissa or less, and BF16 has fp32's exponents) and multiplied by
//        v_mfma_f32_*_bf16, which adds with fp32's accuracy at half the rate
//        (6e-9 of the same sums).
// Sums are fp32 in both.
//
// The products are computed as b a^T: the instruction's rows are out's columns,
// so that a lane's accumulators hold four consecutive columns of one row of
// out.
//
// f8_tile_kernel: a workgroup computes a TILE x TILE tile from slices of 128
// k of both operands that stream from memory straight into LDS, two slices
// deep. A slice's rows are 128 bytes: whole lines of the caches (rows of 64
// bytes, four slices deep, fetched each line twice: 650 us where this takes
// 595, at 16384 x 11008 x 4096). Their 16-byte chunks are XOR-swizzled so that
// 16 consecutive rows' reads fall on all banks.
// f8_rows_kernel: up to 64 rows of a. Bound by reading b once: no LDS on the
// way, each wave reads whole 128-byte lines of b into the instruction's
// layout, and the waves of a workgroup share k.
// f8_sums_kernel: adds the parts of k that several workgroups computed.
#include <type_traits>

#include "grad_internal.h"

namespace sm {
namespace {

constexpr int kWave = 64;
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ int first_lane(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ v8i join(u32x4 lo, u32x4 hi) {
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Nothing behind this runs before v is in its registers.
__device__ __forceinline__ void hold(const v8i &v) { asm volatile("" : : "v"(v) : "memory"); }

// 2^(byte - 127).
__device__ __forceinline__ float scale_of(int byte) { return __int_as_float(byte << 23); }

// Four bytes as BF16, scaled.
template <bool E5M2>
__device__ __forceinline__ u32x2 widen4(int bytes, float scale) {
    bf16x2 lo, hi;
    if (E5M2) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)bytes, scale, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)bytes, scale, true);
    } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)bytes, scale, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)bytes, scale, true);
    }
    return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// Bytes 8 i .. 8 i + 7 of a fragment as BF16, scaled.
template <bool E5M2>
__device__ __forceinline__ bf16x8 widen(const v8i &f, int i, float scale) {
    const u32x2 lo = widen4<E5M2>(f[2 * i], scale), hi = widen4<E5M2>(f[2 * i + 1], scale);
    return __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
}

// Four consecutive columns of out.
__device__ __forceinline__ void store_out(const F8Matmul &f, int64_t at, int have, const float (&v)[4]) {
    if (f.out_bf16)
        store_n<true>(f.out, at, have, v);
    else
        store_n<false>(f.out, at, have, v);
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
constexpr int kSliceBytes = kF8Block;  // bytes, i.e. values, of k per row and slice
constexpr int kStages = 2;

// s_waitcnt with vmcnt = N alone.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// Workgroup barrier that does not wait for the loads into LDS still in flight.
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

constexpr uint32_t kOutside = 0x80000000u;  // buffer offset beyond every extent: loads zeros

// A load of 16 (or 4) bytes a lane straight into LDS at lds + 16 (4) * lane.
// Asm without outputs, so that the compiler does not order every LDS read
// behind the loads in flight; M0 is reserved, and nothing else here reads it.
__device__ __forceinline__ void load16_lds(uint32_t lds, uint32_t offset, u32x4 buffer) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(buffer)
                 : "memory");
}
__device__ __forceinline__ void load4_lds(uint32_t lds, uint32_t offset, u32x4 buffer) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(buffer)
                 : "memory");
}

// A raw buffer over `bytes` bytes (below 2^31) from p on.
__device__ __forceinline__ u32x4 make_buffer(const uint8_t *p, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)first_lane((int)(uint32_t)a), (uint32_t)first_lane((int)((uint32_t)(a >> 32) & 0xffffu)),
                 (uint32_t)first_lane((int)bytes), 0x00020000u};
}

// LDS byte of 16-byte chunk c of a slice's row r.
__device__ __forceinline__ uint32_t slice_at(int r, int c) {
    return (uint32_t)(r * kSliceBytes + ((c ^ ((r >> 1) & 7)) << 4));
}

// One operand's rows of a tile (ROWS rows of which `valid` exist) on their way
// into LDS, by WAVES waves. base: the tile's first row at the k of slice 0. A
// lane's offset stays; the buffer's start moves by a slice (scalar work), and
// past the last slice the buffer is empty: its loads give zeros.
template <int ROWS, int WAVES>
struct Slices {
    static constexpr int kLoads = ROWS * kSliceBytes / 1024 / WAVES;  // per wave and slice
    static_assert(kLoads * WAVES * 1024 == ROWS * kSliceBytes, "whole loads");
    u32x4 buffer;
    uint32_t offset[kLoads];

    __device__ __forceinline__ void init(const uint8_t *base, int64_t pitch, int valid, int wave, int lane) {
        buffer = make_buffer(base, (valid - 1) * pitch + kSliceBytes);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = (i * WAVES + wave) * 8 + lane / 8;
            const int chunk = (lane & 7) ^ ((row >> 1) & 7);
            offset[i] = row < valid ? (uint32_t)(row * pitch + chunk * 16) : kOutside;
        }
    }
    // Load i of the current slice to `lds` (of the slice's first row).
    __device__ __forceinline__ void issue(int i, uint32_t lds, int wave) const {
        load16_lds(lds + (uint32_t)(i * WAVES + wave) * 1024u, offset[i], buffer);
    }
    // On to slice j.
    __device__ __forceinline__ void advance(int j, int slices) {
        const uint32_t lo = buffer[0] + kSliceBytes;
        buffer[1] += lo < (uint32_t)kSliceBytes ? 1u : 0u;
        buffer[0] = lo;
        if (j >= slices) buffer[2] = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) buffer[i] = (uint32_t)first_lane((int)buffer[i]);  // it stays in scalar registers
    }
};

template <int TILE> struct TileShape;
template <> struct TileShape<256> { static constexpr int kWavesM = 2, kWavesN = 2; };
template <> struct TileShape<128> { static constexpr int kWavesM = 2, kWavesN = 2; };

// Blocks go to the 8 XCDs round-robin: each XCD gets a contiguous run of tiles.
__device__ __forceinline__ int xcd_run(int b, int n) {
    const int q = n >> 3, rem = n & 7, x = b & 7, p = b >> 3;
    return x * q + (x < rem ? x : rem) + p;
}

template <int TILE, bool A5, bool B5, bool F32>
__global__ __launch_bounds__(TileShape<TILE>::kWavesM *TileShape<TILE>::kWavesN *kWave) void f8_tile_kernel(F8Matmul f) {
    using S = TileShape<TILE>;
    constexpr int kWaves = S::kWavesM * S::kWavesN;
    constexpr int FM = TILE / S::kWavesM / 32, FN = TILE / S::kWavesN / 32;  // 32 x 32 blocks of a wave
    constexpr int kOperand = TILE * kSliceBytes, kStage = 2 * kOperand;
    constexpr int kScaleLds = kStages * kStage, kScaleStage = 2 * TILE * 4;
    __shared__ __attribute__((aligned(1024))) char lds[kScaleLds + 2 * kScaleStage];
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);

    // batch and part of k, then tiles in bands of 8 rows of tiles, down the
    // band first: the tiles that run at once share operands in L2
    const int tm = (int)((f.m + TILE - 1) / TILE), tn = (int)((f.n + TILE - 1) / TILE);
    int t = xcd_run(blockIdx.x, gridDim.x);
    const int per = tm * tn, unit = t / per;
    t -= unit * per;
    const int band = t / (8 * tn), rows_left = tm - band * 8 < 8 ? tm - band * 8 : 8;
    t -= band * 8 * tn;
    const int64_t row0 = (int64_t)(band * 8 + t % rows_left) * TILE, col0 = (int64_t)(t / rows_left) * TILE;
    const int64_t batch = unit / f.splits;
    const int split = unit % f.splits;
    const int block0 = split * f.chunk;
    const int blocks = f.blocks - block0 < f.chunk ? f.blocks - block0 : f.chunk;

    const int valid_m = (int)(f.m - row0 < TILE ? f.m - row0 : TILE), valid_n = (int)(f.n - col0 < TILE ? f.n - col0 : TILE);
    Slices<TILE, kWaves> la, lb;
    la.init(f.a + batch * f.a_stride + row0 * f.pitch + (int64_t)block0 * kF8Block, f.pitch, valid_m, wave, lane);
    lb.init(f.b + batch * f.b_stride + col0 * f.pitch + (int64_t)block0 * kF8Block, f.pitch, valid_n, wave, lane);
    // scales: one dword of four blocks for each row of a, then of b, 64 rows a load
    constexpr int kScaleLoads = 2 * TILE / (kWaves * kWave);
    static_assert(kScaleLoads * kWaves * kWave == 2 * TILE, "whole scale loads");
    const int dwords = (blocks + 3) / 4;
    u32x4 sbuffer[kScaleLoads];
    uint32_t soffset[kScaleLoads];
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
        const int first = (i * kWaves + wave) * kWave;
        const bool of_b = first >= TILE;
        const int srow = first % TILE + lane, valid = of_b ? valid_n : valid_m;
        const uint8_t *base = (of_b ? f.b_scale + batch * f.bs_stride + col0 * f.scale_pitch
                                    : f.a_scale + batch * f.as_stride + row0 * f.scale_pitch) + block0;
        sbuffer[i] = make_buffer(base, (valid - 1) * f.scale_pitch + dwords * 4);
        soffset[i] = srow < valid ? (uint32_t)(srow * f.scale_pitch) : kOutside;
    }
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(
        (__attribute__((address_space(3))) char *)lds);
    auto load_scales = [&](int g) {
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i)
            load4_lds(lds0 + kScaleLds + (g & 1) * kScaleStage + (i * kWaves + wave) * 256u,
                      g < dwords && soffset[i] != kOutside ? soffset[i] + (uint32_t)g * 4 : kOutside, sbuffer[i]);
    };

    constexpr int kLoads = 2 * Slices<TILE, kWaves>::kLoads;
    auto issue = [&](int j, int i) {  // load i of slice j, the current one of both operands
        const uint32_t at = lds0 + (uint32_t)(j % kStages) * kStage;
        if (i < kLoads / 2)
            la.issue(i, at, wave);
        else
            lb.issue(i - kLoads / 2, at + kOperand, wave);
    };
    auto advance = [&](int j) {
        la.advance(j, blocks);
        lb.advance(j, blocks);
    };
    load_scales(0);
#pragma unroll
    for (int j = 0; j < kStages; ++j) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) issue(j, i);
        advance(j + 1);
    }

    // The fragments of half a slice (64 k) in registers: b's FN, then a's FM, 32
    // bytes a lane (lanes 32 on have the upper 32 k). Read r is 16 bytes of
    // fragment r / 2.
    const int wm = wave / S::kWavesN * FM * 32, wn = wave % S::kWavesN * FN * 32;
    const int row = lane & 31, half = lane >> 5;
    constexpr int kFragments = FM + FN, kReads = 2 * kFragments, kTiles = FM * FN;
    v8i fr[2][kFragments];
    auto read = [&](auto h, int j, int r) {  // of half h of slice j
        constexpr int H = decltype(h)::value;
        const char *stage = lds + j % kStages * kStage;
        const int i = r / 2, chunk = 4 * H + 2 * half + r % 2;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(i < FN ? stage + kOperand + slice_at(wn + i * 32 + row, chunk)
                                                                : stage + slice_at(wm + (i - FN) * 32 + row, chunk));
#pragma unroll
        for (int q = 0; q < 4; ++q) fr[H][i][4 * (r % 2) + q] = (int)v[q];
    };
    // The scale bytes of slice j.
    int sc[kFragments], sc_next[kFragments];
    auto read_scales = [&](int j) {
        const char *s = lds + kScaleLds + (j >> 2 & 1) * kScaleStage + (j & 3);
#pragma unroll
        for (int i = 0; i < kFragments; ++i)
            sc_next[i] = (int)*reinterpret_cast<const uint8_t *>(
                s + 4 * (i < FN ? TILE + wn + i * 32 + row : wm + (i - FN) * 32 + row));
    };
    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};

    constexpr std::integral_constant<int, 0> kLow{};
    constexpr std::integral_constant<int, 1> kHigh{};
    wait_loads<kLoads>();  // slice 0 and the first scales
    barrier();
    read_scales(0);
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(kLow, 0, r);

    // F32: 16 k of the fragments as BF16 (bytes 8 q of both lane halves), one set
    // for the products and one that is filled meanwhile: part p is four bytes of
    // fragment p / 2.
    u32x4 wide[2][F32 ? kFragments : 1];
    auto widen_part = [&](auto h, int q, int p, const int *scales) {
        constexpr int H = decltype(h)::value;
        const int i = p / 2, d = p % 2;
        const float x = scale_of(scales[i]);
        const u32x2 v = i < FN ? widen4<B5>(fr[H][i][2 * q + d], x) : widen4<A5>(fr[H][i][2 * q + d], x);
        wide[q & 1][i][2 * d] = v[0];
        wide[q & 1][i][2 * d + 1] = v[1];
    };
    if constexpr (F32)
#pragma unroll
        for (int p = 0; p < kReads; ++p) widen_part(kLow, 0, p, sc_next);

    // The products of half h of slice j, from the registers, a step for each;
    // extra(step) is what else the step issues, so that the matrix pipe does not
    // wait behind a run of reads, loads or conversions.
    auto products = [&](auto h, auto extra) {
        constexpr int H = decltype(h)::value;
        if constexpr (F32) {
            constexpr int kParts = kReads / kTiles;  // a step
#pragma unroll
            for (int t = 0; t < 4 * kTiles; ++t) {
                const int q = t / kTiles, s = t % kTiles;
                extra(t);
#pragma unroll
                for (int p = s * kParts; p < (s + 1) * kParts; ++p) {
                    if (q < 3)
                        widen_part(h, q + 1, p, sc);
                    else if (H == 0)
                        widen_part(kHigh, 0, p, sc);
                    else
                        widen_part(kLow, 0, p, sc_next);
                }
                acc[s / FN][s % FN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8, wide[q & 1][s % FN]), __builtin_bit_cast(bf16x8, wide[q & 1][FN + s / FN]),
                    acc[s / FN][s % FN], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kTiles; ++s) {
                extra(s);
                acc[s / FN][s % FN] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    fr[H][s % FN], fr[H][FN + s / FN], acc[s / FN][s % FN], B5 ? 1 : 0, A5 ? 1 : 0, 0, sc[s % FN], 0,
                    sc[FN + s / FN]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // Steps of the low half: the reads of the high half in the first half of
    // them, then at step kMeet all waves have read slice j and slice j + 1 has
    // landed, so that slice j + 2 is loaded to slice j's place from there on, two
    // (TILE 128: four) loads a step, and slice j + 1 may be read.
    constexpr int kMeet = (kTiles * 5 + 7) / 8, kPerRead = kReads * 2 / kTiles, kPerLoad = kLoads * 2 / kTiles;
    static_assert(kPerRead * kTiles == 2 * kReads && kPerLoad * kTiles == 2 * kLoads, "whole steps");
    auto load_step = [&](int j, int s) {  // s: steps from kMeet on
#pragma unroll
        for (int i = s * kPerLoad; i < (s + 1) * kPerLoad; ++i)
            if (i < kLoads) issue(j + kStages, i);
    };
    for (int j = 0; j < blocks; ++j) {
#pragma unroll
        for (int i = 0; i < kFragments; ++i) sc[i] = sc_next[i];
        if ((j & 3) == 0) load_scales((j >> 2) + 1);
        products(kLow, [&](int s) {
#pragma unroll
            for (int r = s * kPerRead; r < (s + 1) * kPerRead; ++r)
                if (r < kReads) read(kHigh, j, r);
            if (s == kMeet) {
#pragma unroll
                for (int i = 0; i < kFragments; ++i) hold(fr[1][i]);
                wait_loads<0>();
                barrier();
            }
            if (s >= kMeet) load_step(j, s - kMeet);
        });
        products(kHigh, [&](int s) {
            if (s == 0) read_scales(j + 1);
#pragma unroll
            for (int r = s * kReads / kTiles; r < (s + 1) * kReads / kTiles; ++r)
                if (r < kReads) read(kLow, j + 1, r);
            if (!F32) load_step(j, kTiles - kMeet + s);
        });
        advance(j + kStages + 1);
    }
    wait_loads<0>();  // loads past the end write LDS too
    __syncthreads();

    // 32 rows of a wave at a time through LDS, so that rows are written in
    // stretches of FN * 32 columns
    constexpr int kCols = FN * 32;
    static_assert(kWaves * 32 * (kCols * 4 + 16) <= kScaleLds, "staged rows fit");
    auto write = [&](auto narrow, void *out, int64_t first) {
        constexpr bool N = decltype(narrow)::value;  // as BF16
        constexpr int kPitch = kCols * (N ? 2 : 4) + 16;  // bytes of a staged row
        constexpr int kLanes = kCols / (N ? 8 : 4);       // 16 bytes each
        char *mine = lds + wave * 32 * kPitch;
        const int c = lane % kLanes * (N ? 8 : 4);
        const int64_t left = f.n - (col0 + wn + c);  // columns from this lane's on
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    char *at = mine + row * kPitch + (n * 32 + g * 8 + half * 4) * (N ? 2 : 4);
                    const f32x16 &v = acc[i][n];
                    if constexpr (N)
                        *reinterpret_cast<u32x2 *>(at) =
                            u32x2{to_bf16x2(v[4 * g], v[4 * g + 1]), to_bf16x2(v[4 * g + 2], v[4 * g + 3])};
                    else
                        *reinterpret_cast<f32x4 *>(at) = f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
                }
            // lanes read what others wrote (LDS accesses of a wave keep their order)
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
            u32x4 v[32 * kLanes / kWave];
#pragma unroll
            for (int r = 0; r < 32 * kLanes / kWave; ++r)
                v[r] = *reinterpret_cast<const u32x4 *>(mine + (r * (kWave / kLanes) + lane / kLanes) * kPitch + lane % kLanes * 16);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
            const int64_t to = row0 + wm + i * 32 + lane / kLanes;
            char *p = static_cast<char *>(out) + ((first + to) * f.n + col0 + wn + c) * (N ? 2 : 4);
#pragma unroll
            for (int r = 0; r < 32 * kLanes / kWave; ++r) {
                char *q = p + (int64_t)r * (kWave / kLanes) * f.n * (N ? 2 : 4);
                if (to + r * (kWave / kLanes) >= f.m) continue;
                if (left >= (N ? 8 : 4)) {
                    *reinterpret_cast<u32x4_any *>(q) = v[r];
                } else {
#pragma unroll
                    for (int j = 0; j < (N ? 8 : 4); ++j)
                        if (j < left) {
                            if constexpr (N)
                                reinterpret_cast<uint16_t *>(q)[j] = (uint16_t)(v[r][j / 2] >> (j % 2 * 16));
                            else
                                reinterpret_cast<uint32_t *>(q)[j] = v[r][j];
                        }
                }
            }
        }
    };
    if (f.splits > 1)
        write(std::false_type{}, f.partial, (split * (int64_t)f.batch + batch) * f.m);
    else
        write(std::integral_constant<bool, !F32>{}, f.out, batch * f.m);
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// 16 columns of out and up to 16 MF rows. A wave takes every waves-th group of
// four blocks of k.
template <int MF, bool A5, bool B5, bool F32>
__global__ __launch_bounds__(512) void f8_rows_kernel(F8Matmul f) {
    extern __shared__ __attribute__((aligned(16))) float sums[];  // [waves][MF][64][4]
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);
    const int tn = (int)((f.n + 15) / 16);
    const int64_t batch = blockIdx.x / tn, col0 = (int64_t)(blockIdx.x % tn) * 16;
    const int row = lane & 15, part = lane >> 4;
    // rows past the last one read the last one: their products are not written
    const int64_t col = col0 + row < f.n ? col0 + row : f.n - 1;
    const uint8_t *b = f.b + batch * f.b_stride + col * f.pitch + part * 32;
    const uint8_t *bs = f.b_scale + batch * f.bs_stride + col * f.scale_pitch;
    const uint8_t *a[MF], *as[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const int64_t r = i * 16 + row < f.m ? i * 16 + row : f.m - 1;
        a[i] = f.a + batch * f.a_stride + r * f.pitch + part * 32;
        as[i] = f.a_scale + batch * f.as_stride + r * f.scale_pitch;
    }
    f32x4 acc[MF] = {};
    const int groups = (f.blocks + 3) / 4;
    for (int g = wave; g < groups; g += f.waves) {
        const int left = f.blocks - g * 4;  // blocks of this group
        const int sb = *reinterpret_cast<const int *>(bs + g * 4);
        int sa[MF];
#pragma unroll
        for (int i = 0; i < MF; ++i) sa[i] = *reinterpret_cast<const int *>(as[i] + g * 4);
        v8i fb[4], fa[4][MF];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = (int64_t)(g * 4 + (k < left ? k : 0)) * kF8Block;
            fb[k] = join(*reinterpret_cast<const u32x4 *>(b + at), *reinterpret_cast<const u32x4 *>(b + at + 16));
#pragma unroll
            for (int i = 0; i < MF; ++i)
                fa[k][i] = join(*reinterpret_cast<const u32x4 *>(a[i] + at), *reinterpret_cast<const u32x4 *>(a[i] + at + 16));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left)
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    if constexpr (F32) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                widen<B5>(fb[k], q, scale_of(sb >> (8 * k) & 255)),
                                widen<A5>(fa[k][i], q, scale_of(sa[i] >> (8 * k) & 255)),
                                acc[i], 0, 0, 0);
                    } else {
                        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            fb[k], fa[k][i], acc[i], B5 ? 1 : 0, A5 ? 1 : 0, 0, sb >> (8 * k), 0, sa[i] >> (8 * k));
                    }
                }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i) *reinterpret_cast<f32x4 *>(sums + ((wave * MF + i) * kWave + lane) * 4) = acc[i];
    __syncthreads();
    for (int t = threadIdx.x; t < MF * kWave; t += f.waves * kWave) {
        const int l = t & (kWave - 1);
        f32x4 v = {};
        for (int w = 0; w < f.waves; ++w) v += *reinterpret_cast<const f32x4 *>(sums + (w * MF * kWave + t) * 4);
        // lane l: row l % 16 of the block's rows, columns 4 (l / 16) on
        const int64_t r = t / kWave * 16 + (l & 15), c = col0 + (l >> 4) * 4;
        const float o[4] = {v[0], v[1], v[2], v[3]};
        if (r < f.m) store_out(f, (batch * f.m + r) * f.n + c, (int)(f.n - c < 4 ? f.n - c : 4), o);
    }
}

// out = the splits' sums, in order; 4 entries a thread of the flat array.
__global__ __launch_bounds__(256) void f8_sums_kernel(F8Matmul f) {
    const int64_t total = f.batch * f.m * f.n;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= total) return;
    const int have = (int)(total - at < 4 ? total - at : 4);
    float v[4] = {};
    for (int s = 0; s < f.splits; ++s) {
        float p[4];
        load_n<false>(f.partial, s * total + at, have, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += p[j];
    }
    store_out(f, at, have, v);
}

template <bool A5, bool B5, bool F32>
void launch(const F8Matmul &f, hipStream_t s) {
    if (f.tile == 16) {
        const dim3 grid((unsigned)(f.batch * ((f.n + 15) / 16)));
        const int threads = f.waves * kWave;
        const int mf = f.m <= 16 ? 1 : f.m <= 32 ? 2 : 4;
        const size_t lds = (size_t)mf * threads * 16;
        if (mf == 1)
            f8_rows_kernel<1, A5, B5, F32><<<grid, threads, lds, s>>>(f);
        else if (mf == 2)
            f8_rows_kernel<2, A5, B5, F32><<<grid, threads, lds, s>>>(f);
        else
            f8_rows_kernel<4, A5, B5, F32><<<grid, threads, lds, s>>>(f);
        return;
    }
    const int64_t tiles = (f.m + f.tile - 1) / f.tile * ((f.n + f.tile - 1) / f.tile);
    const dim3 grid((unsigned)(tiles * f.batch * f.splits));
    if (f.tile == 256)
        f8_tile_kernel<256, A5, B5, F32><<<grid, 256, 0, s>>>(f);
    else
        f8_tile_kernel<128, A5, B5, F32><<<grid, 256, 0, s>>>(f);
}

template <bool F32>
void launch_out(const F8Matmul &f, hipStream_t s) {
    if (f.a_e5m2)
        f.b_e5m2 ? launch<true, true, F32>(f, s) : launch<true, false, F32>(f, s);
    else
        f.b_e5m2 ? launch<false, true, F32>(f, s) : launch<false, false, F32>(f, s);
}

}  // namespace

F8Plan f8_plan(int64_t batch, int64_t m, int64_t n, int64_t k) {
    const int64_t blocks = f8_pitch(k) / kF8Block, groups = (blocks + 3) / 4;
    F8Plan p{};
    p.splits = 1;
    p.chunk = (int32_t)(groups * 4);
    if (m <= 64) {
        p.tile = 16;
        const int64_t wgs = batch * ((n + 15) / 16);
        p.waves = 4;
        while (p.waves < 8 && p.waves < groups && wgs * p.waves < 2048) p.waves *= 2;
        return p;
    }
    auto tiles = [&](int64_t t) { return batch * ((m + t - 1) / t) * ((n + t - 1) / t); };
    p.tile = tiles(256) >= 192 ? 256 : 128;
    // parts of k until every compute unit has a workgroup, at least 4 blocks each
    const int64_t want = p.tile == 256 ? 256 : 512, have = tiles(p.tile);
    int64_t splits = have >= want ? 1 : want / have;
    if (splits > groups) splits = groups;
    p.chunk = (int32_t)((groups + splits - 1) / splits * 4);
    p.splits = (int32_t)((blocks + p.chunk - 1) / p.chunk);
    return p;
}

void launch_f8_matmul(const F8Matmul &f, hipStream_t s) {
    if (f.out_bf16)
        launch_out<false>(f, s);
    else
        launch_out<true>(f, s);
}

void launch_f8_sums(const F8Matmul &f, hipStream_t s) {
    const int64_t total = f.batch * f.m * f.n;
    f8_sums_kernel<<<dim3((unsigned)((total + 1023) / 1024)), 256, 0, s>>>(f);
}

}  // namespace sm
