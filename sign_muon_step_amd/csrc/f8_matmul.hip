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
//  F32   the bytes are converted to BF16 with their scale and multiplied by
//        v_mfma_f32_*_bf16, which adds with fp32's accuracy at half the rate
//        (6e-9 of the same sums). BF16 holds every value from 2^-126 to below
//        2^128 (4 bits of mantissa or less, fp32's exponents); scales from 2^120
//        on (E5M2: 2^113) can stand for more, which becomes infinite, where the
//        other form has it.
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
// f8_rows_kernel: up to 32 rows of a. Bound by reading b once: no LDS on the
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

// v is computed here, not behind a later branch.
__device__ __forceinline__ void pin(f32x16 &v) { asm volatile("" : "+a"(v)); }

// Zeros written straight to where they are kept (one zero for all of them would
// take sixteen registers of its own).
__device__ __forceinline__ f32x16 zeros() {
    float z = 0.0f;
    asm volatile("" : "+v"(z));
    return f32x16{z, z, z, z, z, z, z, z, z, z, z, z, z, z, z, z};
}

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
    asm volatile("" ::: "memory");
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

// A tile of one batch entry and one part of k.
struct Tile {
    int64_t row0, col0, batch;
    int split, block0, blocks;
};

template <int TILE> struct TileShape;
template <> struct TileShape<256> { static constexpr int kWavesM = 2, kWavesN = 2; };
template <> struct TileShape<128> { static constexpr int kWavesM = 2, kWavesN = 2; };

template <int TILE>
__device__ __forceinline__ Tile tile_at(const F8Matmul &f, int v, int total) {
    // batch and part of k, then tiles in bands of 8 rows of tiles, down the
    // band first: the tiles that run at once share operands in L2
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
    o.block0 = o.split * f.chunk;
    o.blocks = f.blocks - o.block0 < f.chunk ? f.blocks - o.block0 : f.chunk;
    return o;
}

// The slices of a workgroup's tiles, one after the other, on their way into
// LDS: both operands' rows and their scales (a row's dword of four blocks). A
// lane's offsets stay: a tile and a slice are a buffer's start and length, and
// rows past the operand's last one, like slices past the last tile's, lie
// beyond the length and give zeros.
template <int TILE, int WAVES>
struct Loader {
    static constexpr int kRowLoads = TILE * kSliceBytes / 1024 / WAVES;  // per wave, slice and operand
    static constexpr int kScaleLoads = 2 * TILE / (WAVES * kWave);
    static constexpr int kLoads = 2 * kRowLoads;
    static constexpr int kOperand = TILE * kSliceBytes, kStage = 2 * kOperand;
    // scales lie apart, a stage for each four blocks of a tile: those that a wave
    // may still read, two slices' that are there or under way, and the next one's
    static constexpr int kScales = kStages * kStage, kScaleStages = 4, kScaleStage = 2 * TILE * 4;
    static_assert(kRowLoads * WAVES * 1024 == kOperand && kScaleLoads * WAVES * kWave == 2 * TILE, "whole loads");
    u32x4 rows[2], scales[kScaleLoads];
    uint32_t row_at[kRowLoads], scale_at;
    int v, blocks, block;  // the tile, the end of its blocks and the next one to load
    unsigned group;        // groups of scales so far

    __device__ __forceinline__ void start(const F8Matmul &f, int v_, int total, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < kRowLoads; ++i) {
            const int row = (i * WAVES + wave) * 8 + lane / 8;
            row_at[i] = (uint32_t)(row * f.pitch + (((lane & 7) ^ ((row >> 1) & 7)) << 4));
        }
        static_assert(TILE == 128 || TILE % (WAVES * kWave) == 0, "a wave's scale loads are of the same rows");
        scale_at = (uint32_t)((wave * kWave % TILE + lane) * f.scale_pitch);
        v = v_;
        group = 0;
        tile(f, total, wave);
    }
    __device__ __forceinline__ void tile(const F8Matmul &f, int total, int wave) {
        const bool there = v < total;
        const Tile t = tile_at<TILE>(f, there ? v : 0, total);
        block = t.block0;
        blocks = t.block0 + t.blocks;
        const int64_t valid[2] = {f.m - t.row0 < TILE ? f.m - t.row0 : TILE, f.n - t.col0 < TILE ? f.n - t.col0 : TILE};
        const uint8_t *base[2] = {f.a + t.batch * f.a_stride + t.row0 * f.pitch,
                                  f.b + t.batch * f.b_stride + t.col0 * f.pitch};
        const uint8_t *sbase[2] = {f.a_scale + t.batch * f.as_stride + t.row0 * f.scale_pitch,
                                   f.b_scale + t.batch * f.bs_stride + t.col0 * f.scale_pitch};
#pragma unroll
        for (int o = 0; o < 2; ++o)
            rows[o] = make_buffer(base[o] + (int64_t)block * kSliceBytes,
                                  there ? (valid[o] - 1) * f.pitch + kSliceBytes : 0);
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) {
            const bool of_b = (i * WAVES + wave) * kWave >= TILE;
            scales[i] = make_buffer((of_b ? sbase[1] : sbase[0]) + block,
                                    there ? ((of_b ? valid[1] : valid[0]) - 1) * f.scale_pitch + 4 : 0);
        }
    }
    // Load i of the current slice to LDS; `to`: the wave's place in the slice's stage.
    __device__ __forceinline__ void issue(int i, uint32_t to) const {
        const int o = i / kRowLoads, r = i % kRowLoads;
        load16_lds(to + (uint32_t)(o * kOperand + r * WAVES * 1024), row_at[r], rows[o]);
    }
    // The scales of the current slice's four blocks.
    __device__ __forceinline__ void issue_scales(uint32_t lds, int wave) {
        const uint32_t to = lds + kScales + group++ % kScaleStages * kScaleStage + (uint32_t)wave * 256u;
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) load4_lds(to + (uint32_t)(i * WAVES * 256), scale_at, scales[i]);
    }
    __device__ __forceinline__ void move(u32x4 &buffer, uint32_t by) {
        const uint32_t lo = buffer[0] + by;
        buffer[1] += lo < by ? 1u : 0u;
        buffer[0] = lo;
#pragma unroll
        for (int i = 0; i < 3; ++i) buffer[i] = (uint32_t)first_lane((int)buffer[i]);  // it stays in scalar registers
    }
    // On to the next slice, and its scales where they are the first of four.
    __device__ __forceinline__ void advance(const F8Matmul &f, int total, uint32_t lds, int wave) {
        if (++block == blocks) {
            v += gridDim.x;
            tile(f, total, wave);
        } else {
            move(rows[0], kSliceBytes);
            move(rows[1], kSliceBytes);
            if (block & 3) return;
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) move(scales[i], 4);
        }
        issue_scales(lds, wave);
    }
};

// A workgroup takes every gridDim-th tile. The loads run two slices ahead of
// the products, on into the next tile, so that a tile's first slices are there
// when the one before it is done, and a tile's results are on their way to
// memory during the next one's products.
// F32: the widened form. WIDE: results in fp32 (F32, and the parts of k of BF16 results).
template <int TILE, bool A5, bool B5, bool F32, bool WIDE>
__global__ __launch_bounds__(TileShape<TILE>::kWavesM *TileShape<TILE>::kWavesN *kWave) void f8_tile_kernel(F8Matmul f,
                                                                                                         int total) {
    using S = TileShape<TILE>;
    constexpr int kWaves = S::kWavesM * S::kWavesN;
    constexpr int FM = TILE / S::kWavesM / 32, FN = TILE / S::kWavesN / 32;  // 32 x 32 blocks of a wave
    using L = Loader<TILE, kWaves>;
    constexpr int kLoads = L::kLoads;
    // results on their way: 32 rows of kOutBytes a wave
    constexpr int kOutBytes = TILE / 2, kOutPitch = kOutBytes + 16;
    constexpr int kOut = L::kScales + L::kScaleStages * L::kScaleStage;
    __shared__ __attribute__((aligned(1024))) char lds[kOut + kWaves * 32 * kOutPitch];
    const int lane = threadIdx.x & (kWave - 1), wave = first_lane(threadIdx.x / kWave);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)lds);

    L loader;
    loader.start(f, blockIdx.x, total, wave, lane);
    auto place = [&](unsigned c) {
        uint32_t to = lds0 + c % kStages * L::kStage + (uint32_t)wave * 1024u;
        // opaque: each load adds its constant to this, where the compiler would
        // keep every sum in a scalar register of its own and run out of them
        asm volatile("" : "+s"(to));
        return to;
    };
    loader.issue_scales(lds0, wave);
#pragma unroll 1
    for (unsigned c = 0; c < kStages; ++c) {
        const uint32_t to = place(c);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) loader.issue(i, to);
        loader.advance(f, total, lds0, wave);
    }

    // The fragments of half a slice (64 k) in registers: b's FN, then a's FM, 32
    // bytes a lane (lanes 32 on have the upper 32 k). Read r is 16 bytes of
    // fragment r / 2.
    const int wm = wave / S::kWavesN * FM * 32, wn = wave % S::kWavesN * FN * 32;
    const int row = lane & 31, half = lane >> 5;
    constexpr int kFragments = FM + FN, kReads = 2 * kFragments, kTiles = FM * FN;
    v8i fr[2][kFragments];
    auto read = [&](auto h, unsigned c, int r) {  // of half h of slice c
        constexpr int H = decltype(h)::value;
        const char *stage = lds + c % kStages * L::kStage;
        const int i = r / 2, chunk = 4 * H + 2 * half + r % 2;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(
            i < FN ? stage + L::kOperand + slice_at(wn + i * 32 + row, chunk) : stage + slice_at(wm + (i - FN) * 32 + row, chunk));
#pragma unroll
        for (int q = 0; q < 4; ++q) fr[H][i][4 * (r % 2) + q] = (int)v[q];
    };
    // The scale bytes of block b of a tile, in group g so far (tiles begin at
    // every fourth block of k, as the scales' dwords do).
    int sc[kFragments], sc_next[kFragments];
    auto read_scales = [&](unsigned g, int b) {
        const char *s = lds + L::kScales + g % L::kScaleStages * L::kScaleStage + (b & 3);
#pragma unroll
        for (int i = 0; i < kFragments; ++i)
            sc_next[i] = (int)*reinterpret_cast<const uint8_t *>(
                s + 4 * (i < FN ? TILE + wn + i * 32 + row : wm + (i - FN) * 32 + row));
    };
    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i / FN][i % FN] = zeros();

    constexpr std::integral_constant<int, 0> kLow{};
    constexpr std::integral_constant<int, 1> kHigh{};
    wait_loads<kLoads>();  // slice 0 and its scales
    barrier();
    Tile t = tile_at<TILE>(f, blockIdx.x, total);
    read_scales(0, 0);
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

    // The products of half a slice, from the registers, a step for each;
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
    // them, then at step kMeet all waves have read slice c and slice c + 1 has
    // landed, so that slice c + 2 is loaded to slice c's place from there on, and
    // slice c + 1 may be read.
    constexpr int kMeet = (kTiles * 5 + 7) / 8, kPerRead = kReads * 2 / kTiles;
    constexpr int kPerLoad = kLoads * 2 / kTiles;
    static_assert(kPerRead * kTiles == 2 * kReads && kPerLoad * kTiles == 2 * kLoads, "whole steps");
    auto load_step = [&](uint32_t to, int s) {  // s: steps from kMeet on
#pragma unroll
        for (int i = s * kPerLoad; i < (s + 1) * kPerLoad; ++i)
            if (i < kLoads) loader.issue(i, to);
    };

    // Results as BF16 (N) or fp32, through LDS so that whole lines are written.
    // n a multiple of the 16 bytes' columns (`even`): buffer stores, which are
    // always issued (what lies outside is dropped), so that their number is
    // known; otherwise plain stores.
    const bool even = f.n % (WIDE ? 4 : 8) == 0;
    auto write = [&](void *out, int64_t first) {
        constexpr bool N = !WIDE;
        constexpr int E = N ? 2 : 4, W = 16 / E;              // bytes of a value, values of a store
        constexpr int kCols = kOutBytes / E;                      // columns at a time
        constexpr int kLanes = kOutBytes / 16, kRows = kWave / kLanes;  // lanes of a row, rows of a store
        static_assert(kCols % 8 == 0 && FN * 32 % kCols == 0, "whole passes");
        char *mine = lds + kOut + wave * 32 * kOutPitch;
        // made anew for each tile, so that no address is kept in registers meanwhile
        int lane_ = lane;
        asm volatile("" : "+v"(lane_));
        const int r0 = lane_ / kLanes, c16 = lane_ % kLanes, row = lane_ & 31, half = lane_ >> 5;
        // the wave's part of the tile: what exists of it, and a buffer over that
        const int64_t row1 = t.row0 + wm, col1 = t.col0 + wn;
        const int rows = (int)(f.m - row1 < 0 ? 0 : f.m - row1 < FM * 32 ? f.m - row1 : FM * 32);
        const int cols = (int)(f.n - col1 < 0 ? 0 : f.n - col1 < FN * 32 ? f.n - col1 : FN * 32);
        const int pitch = (int)f.n * E;
        char *p = static_cast<char *>(out) + ((first + row1) * f.n + col1) * E;
        const __amdgpu_buffer_rsrc_t buffer =
            __builtin_amdgcn_make_buffer_rsrc(p, 0, rows > 0 && cols > 0 ? (rows - 1) * pitch + cols * E : 0, 0x00020000);
        uint32_t at[FN * 32 / kCols];  // of the lane's columns of each pass, in row r0
#pragma unroll
        for (int n0 = 0; n0 < FN * 32; n0 += kCols)
            at[n0 / kCols] = n0 + c16 * W < cols ? (uint32_t)(r0 * pitch + (n0 + c16 * W) * E) : kOutside;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int n0 = 0; n0 < FN * 32; n0 += kCols) {
                // no accumulator leaves its register before its turn
#pragma unroll
                for (int n = n0 / 32; n < (n0 + kCols + 31) / 32; ++n) pin(acc[i][n]);
#pragma unroll
                for (int n = n0; n < n0 + kCols; n += 8) {
                    char *to = mine + row * kOutPitch + (n - n0 + half * 4) * E;
                    const f32x16 &v = acc[i][n / 32];
                    const int g = n % 32 / 2;  // of the four groups of 8 columns, 4 values each
                    if constexpr (N)
                        *reinterpret_cast<u32x2 *>(to) = u32x2{to_bf16x2(v[g], v[g + 1]), to_bf16x2(v[g + 2], v[g + 3])};
                    else
                        *reinterpret_cast<f32x4 *>(to) = f32x4{v[g], v[g + 1], v[g + 2], v[g + 3]};
                }
                if (n0 + kCols == FN * 32)
#pragma unroll
                    for (int n = 0; n < FN; ++n) acc[i][n] = zeros();
                // lanes read what others wrote (LDS accesses of a wave keep their order)
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
                auto staged = [&](int r) { return *reinterpret_cast<const u32x4 *>(mine + (r * kRows + r0) * kOutPitch + c16 * 16); };
                if (even) {
                    u32x4 v[32 / kRows];
#pragma unroll
                    for (int r = 0; r < 32 / kRows; ++r) v[r] = staged(r);
#pragma unroll
                    for (int r = 0; r < 32 / kRows; ++r)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            v[r], buffer, (int)(at[n0 / kCols] + (uint32_t)((i * 32 + r * kRows) * pitch)), 0, 0);
                } else {
                    const int here = cols - n0;  // columns from this pass's first on
#pragma unroll 1
                    for (int r = 0; r < 32 / kRows; ++r)
                        if (i * 32 + r * kRows + r0 < rows && c16 * W + W <= here)
                            *reinterpret_cast<u32x4_any *>(p + (int64_t)(i * 32 + r * kRows + r0) * pitch + (n0 + c16 * W) * E) =
                                staged(r);
                    // the last columns of a row, one by one
                    if (here > 0 && here < kCols && i * 32 + row < rows && half == 0)
#pragma unroll 1
                        for (int c = here / W * W; c < here; ++c) {
                            char *q = p + (int64_t)(i * 32 + row) * pitch + (n0 + c) * E;
                            const char *from = mine + row * kOutPitch + c * E;
                            if constexpr (N)
                                *reinterpret_cast<uint16_t *>(q) = *reinterpret_cast<const uint16_t *>(from);
                            else
                                *reinterpret_cast<uint32_t *>(q) = *reinterpret_cast<const uint32_t *>(from);
                        }
                }
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    // stores of one tile and wave
    constexpr int kStores = FM * FN * 32 * 32 * (WIDE ? 4 : 2) / 1024, kBehind = kStores < 63 ? kStores : 63;
    bool behind = false;

    // Slice c, block j of tile t; `newer` operations may be under way behind the
    // loads of slice c + 1 and its scales.
    unsigned group = 0;  // of the scales of the next slice
    auto slice = [&](unsigned c, int j, auto newer) {
        const uint32_t to = place(c);
        const int next = j + 1 == t.blocks ? 0 : j + 1;
        if ((next & 3) == 0) ++group;
#pragma unroll
        for (int i = 0; i < kFragments; ++i) sc[i] = sc_next[i];
        products(kLow, [&](int s) {
#pragma unroll
            for (int r = s * kPerRead; r < (s + 1) * kPerRead; ++r)
                if (r < kReads) read(kHigh, c, r);
            if (s == kMeet) {
#pragma unroll
                for (int i = 0; i < kFragments; ++i) hold(fr[1][i]);
                wait_loads<decltype(newer)::value>();
                barrier();
            }
            if (s >= kMeet) load_step(to, s - kMeet);
        });
        products(kHigh, [&](int s) {
            if (s == 0) read_scales(group, next);
#pragma unroll
            for (int r = s * kReads / kTiles; r < (s + 1) * kReads / kTiles; ++r)
                if (r < kReads) read(kLow, c + 1, r);
            if (!F32) load_step(to, kTiles - kMeet + s);
        });
#pragma unroll
        for (int i = 0; i < kTiles; ++i) pin(acc[i / FN][i % FN]);
        loader.advance(f, total, lds0, wave);
    };
    unsigned c = 0;  // slices so far
    for (int v = blockIdx.x; v < total; v += gridDim.x) {
        int j = 0;
        if (behind) slice(c++, j++, std::integral_constant<int, kBehind>{});
#pragma unroll 1
        for (; j < t.blocks; ++j, ++c) slice(c, j, kLow);
        if constexpr (WIDE)
            write(f.splits > 1 ? f.partial : f.out, (f.splits > 1 ? t.split * (int64_t)f.batch + t.batch : t.batch) * f.m);
        else
            write(f.out, t.batch * f.m);
        behind = even;
        if (v + (int)gridDim.x < total) t = tile_at<TILE>(f, v + gridDim.x, total);
    }
    wait_loads<0>();  // loads past the last tile write LDS too
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
    // Four blocks of both operands and their scales. Blocks past the last one
    // read the group's first: their products are not taken.
    struct Group {
        v8i b[4], a[4][MF];
        int sb, sa[MF];
    };
    auto load = [&](Group &o, int g) {
        o.sb = *reinterpret_cast<const int *>(bs + g * 4);
#pragma unroll
        for (int i = 0; i < MF; ++i) o.sa[i] = *reinterpret_cast<const int *>(as[i] + g * 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = (int64_t)(g * 4 + (g * 4 + k < f.blocks ? k : 0)) * kF8Block;
            o.b[k] = join(*reinterpret_cast<const u32x4 *>(b + at), *reinterpret_cast<const u32x4 *>(b + at + 16));
#pragma unroll
            for (int i = 0; i < MF; ++i)
                o.a[k][i] = join(*reinterpret_cast<const u32x4 *>(a[i] + at), *reinterpret_cast<const u32x4 *>(a[i] + at + 16));
        }
    };
    f32x4 acc[MF] = {};
    auto products = [&](const Group &o, int g) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (g * 4 + k < f.blocks)
#pragma unroll
                for (int i = 0; i < MF; ++i) {
                    if constexpr (F32) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                widen<B5>(o.b[k], q, scale_of(o.sb >> (8 * k) & 255)),
                                widen<A5>(o.a[k][i], q, scale_of(o.sa[i] >> (8 * k) & 255)), acc[i], 0, 0, 0);
                    } else {
                        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            o.b[k], o.a[k][i], acc[i], B5 ? 1 : 0, A5 ? 1 : 0, 0, o.sb >> (8 * k), 0, o.sa[i] >> (8 * k));
                    }
                }
    };
    // the next group is on its way while one is multiplied
    const int groups = (f.blocks + 3) / 4;
    Group even, odd;
    if (wave < groups) load(even, wave);
    for (int g = wave; g < groups; g += 2 * f.waves) {
        if (g + f.waves < groups) load(odd, g + f.waves);
        products(even, g);
        if (g + f.waves >= groups) break;
        if (g + 2 * f.waves < groups) load(even, g + 2 * f.waves);
        products(odd, g + f.waves);
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
        const int mf = f.m <= 16 ? 1 : 2;
        const size_t lds = (size_t)mf * threads * 16;
        if (mf == 1)
            f8_rows_kernel<1, A5, B5, F32><<<grid, threads, lds, s>>>(f);
        else
            f8_rows_kernel<2, A5, B5, F32><<<grid, threads, lds, s>>>(f);
        return;
    }
    const int total = (int)((f.m + f.tile - 1) / f.tile * ((f.n + f.tile - 1) / f.tile)) * f.batch * f.splits;
    // one workgroup a compute unit (TILE 128: two), a multiple of the XCDs
    const int most = device_cus() / 8 * 8 * (f.tile == 256 ? 1 : 2);
    const dim3 grid((unsigned)(total < most ? total : most));
    if (f.tile == 256)
        f.splits > 1 ? f8_tile_kernel<256, A5, B5, F32, true><<<grid, 256, 0, s>>>(f, total)
                     : f8_tile_kernel<256, A5, B5, F32, F32><<<grid, 256, 0, s>>>(f, total);
    else
        f.splits > 1 ? f8_tile_kernel<128, A5, B5, F32, true><<<grid, 256, 0, s>>>(f, total)
                     : f8_tile_kernel<128, A5, B5, F32, F32><<<grid, 256, 0, s>>>(f, total);
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
    // Few rows: each tile of 16 columns reads all of a, which costs more than b from
    // about 32 rows on. Against tiles of 128 (us, BF16, n x k; 256 is never faster):
    //              8 rows       16 rows      24 rows      32 rows
    // 11008 x 4096 14.8 / 16.3  16.0 / 16.2  19.3 / 16.5  21.4 / 16.7
    // 4096 x 4096   8.8 / 12.7   8.8 / 12.8   8.7 / 13.3   9.3 / 13.5
    // 4096 x 11008 12.4 / 20.3  14.3 / 20.2  17.3 / 20.4  19.0 / 20.6
    // 2304 x 768    8.6 / 9.4    8.7 / 9.4    8.7 / 9.4    8.7 / 9.4
    // The rule goes by m alone: more than about 16 rows of a wide b (688 tiles of 16
    // columns where the device has 256 compute units) would take 15 to 22 % less in
    // tiles for a BF16 result, and the same for an F32 one (21.4 / 21.8 at 32 rows).
    if (m <= 32) {
        p.tile = 16;
        // waves that share a tile's k: 2 to 8, until each has one group of four
        // blocks or the device is full
        const int64_t wgs = batch * ((n + 15) / 16);
        p.waves = 2;
        while (p.waves < 8 && p.waves < groups && wgs * p.waves < 2048) p.waves *= 2;
        return p;
    }
    // The tile and the parts of k (whole groups of 4 blocks; the last part may be
    // shorter) of the least time by this model, in units of about half a microsecond,
    // fitted to both tiles at 8 to 11008 tiles and 6 to 64 blocks: a round of tiles
    // (one of 256 or two of 128 a compute unit) takes 3 units a block and 10 more, or 2
    // and 4 more, a group that is not full counted as a full one; adding the parts
    // takes 10 and 2 MB of partial sums written or read a unit. The compute units are
    // those of a whole MI355X, not asked for, since the workspace's size is told
    // without a device and has to be that of the same plan.
    // E.g. 8192 x 2304 x 768 to BF16: 288 tiles of 256 in two rounds, 29.3 us, 1152 of
    // 128 in three short ones, 23.7 us; 8 x 768 x 2304 x 2000 to F32: 216 tiles in one
    // round, 60 us, 864 in two, 63 us.
    double best = 0.0;
    for (const int32_t tile : {256, 128}) {
        const int64_t tiles = batch * ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
        const int64_t slots = tile == 256 ? 256 : 512;
        int32_t last = 0;
        for (int64_t splits = 1; splits <= groups && splits <= 32; ++splits) {
            const int64_t chunk = (groups + splits - 1) / splits * 4, parts = (blocks + chunk - 1) / chunk;
            if (chunk == last) continue;
            last = (int32_t)chunk;
            const double rounds = (double)((tiles * parts + slots - 1) / slots);
            double time = rounds * (tile == 256 ? 3.0 * chunk + 10.0 : 2.0 * chunk + 4.0);
            if (parts > 1) time += 10.0 + 8.0 * (double)(parts * batch) * (double)m * (double)n / 2e6;
            if (p.tile == 0 || time < best) {
                best = time;
                p.tile = tile;
                p.chunk = (int32_t)chunk;
                p.splits = (int32_t)parts;
            }
        }
    }
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
