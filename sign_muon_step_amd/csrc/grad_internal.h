// grad_internal.h -- launch descriptors and device helpers of the gradient
// operators (embedding, layer norm, 8-bit quantisation and products). Not
// part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sm {

// The calling thread's last HIP failure is kept for signmuon_strerror; returns
// the status of the launch just made.
int launch_status();

// Compute units of the current device.
int device_cus();

// ---------------------------------------------------------------------------
// Embedding.
// ---------------------------------------------------------------------------
struct Embed {
    const void *ids;
    const void *table;
    void *y;
    int64_t tokens, vocab, cols;
    float scale;
    bool id64, table_bf16, y_bf16;
};
void launch_embedding(const Embed &e, hipStream_t s);

// Tokens sorted by one workgroup in LDS; longer batches are merged from runs
// of this length.
constexpr int kSortChunk = 4096;

struct EmbedGrad {
    const void *ids;
    const void *dy;
    void *grad;
    uint64_t *keys[2];  // [workers][tokens]: id << 32 | token; the second only where tokens > kSortChunk
    float *partial;     // [workers][segments][2][cols]: a segment's first and last rows where they are
                        // shared with its neighbours
    int64_t tokens, vocab, cols;
    int32_t workers;
    int32_t seg;        // sorted tokens per segment
    int32_t segments;   // per worker
    float scale;
    bool id64, dy_bf16, grad_bf16, accumulate;
};
// Columns that one wave sums: 4 a lane.
constexpr int kEmbedCols = 256;
// Merge passes after the chunks' sorts; the sorted keys are in keys[passes & 1].
int embed_merge_passes(int64_t tokens);
int32_t embed_segment(int32_t workers, int64_t tokens, int64_t cols);
void launch_embedding_sort(const EmbedGrad &e, hipStream_t s);
void launch_embedding_merge(const EmbedGrad &e, int pass, hipStream_t s);
void launch_embedding_sums(const EmbedGrad &e, hipStream_t s);
void launch_embedding_join(const EmbedGrad &e, hipStream_t s);

// ---------------------------------------------------------------------------
// Layer norm.
// ---------------------------------------------------------------------------
struct Norm {
    const void *x;
    const float *gamma, *beta;
    void *y;
    float *mean, *rstd;
    int64_t rows, cols;
    float eps;
    bool bf16;
};
void launch_layer_norm(const Norm &n, hipStream_t s);

struct NormGrad {
    const void *dy, *x;
    const float *gamma, *mean, *rstd;
    void *dx, *dgamma, *dbeta;
    float *partial;  // [workers][parts][2][cols] sums of dy * xh and of dy; unused where parts = 1
    int64_t rows;    // per worker
    int64_t cols;
    int32_t workers;
    int32_t parts;  // blocks of rows per worker, each with a sum of its own
    bool bf16, grad_bf16;
};
int32_t norm_parts(int32_t workers, int64_t rows, int64_t cols);
void launch_layer_norm_backward(const NormGrad &n, hipStream_t s);
// Adds the parts' sums (parts > 1).
void launch_layer_norm_sums(const NormGrad &n, hipStream_t s);

// ---------------------------------------------------------------------------
// 8-bit floating point.
// ---------------------------------------------------------------------------
constexpr int kF8Block = 128;  // values per scale
constexpr int kF8Zero = 127;   // scale byte of 2^0, and of padding
inline int64_t f8_pitch(int64_t k) { return (k + kF8Block - 1) / kF8Block * kF8Block; }
inline int64_t f8_scale_pitch(int64_t k) { return (f8_pitch(k) / kF8Block + 3) / 4 * 4; }

struct F8Quant {
    const void *x;
    uint8_t *q, *q_scale, *qt, *qt_scale;  // q or qt may be null
    int64_t rows, cols;
    int64_t pitch, scale_pitch;      // of q: a row's bytes
    int64_t tpitch, tscale_pitch;    // of qt
    int32_t batch;
    int32_t row_tiles, col_tiles;    // of 128
    bool bf16, e5m2;
};
void launch_f8_quant(const F8Quant &f, hipStream_t s);

struct F8Matmul {
    const uint8_t *a, *a_scale, *b, *b_scale;
    void *out;
    float *partial;  // [splits][batch][m][n], unused where splits = 1
    int64_t m, n, pitch, scale_pitch;
    int64_t a_stride, b_stride, as_stride, bs_stride;  // bytes between batches (b's are 0 where it is shared)
    int32_t batch, blocks;     // blocks: of 128 along k
    int32_t splits, chunk;     // chunk: blocks of one split, a multiple of 4
    int32_t tile;              // rows and columns of a workgroup's tile; 16: few rows
    int32_t waves;             // tile 16: waves that share a tile's k
    bool a_e5m2, b_e5m2, out_bf16;
};
struct F8Plan {
    int32_t tile, splits, chunk, waves;
};
F8Plan f8_plan(int64_t batch, int64_t m, int64_t n, int64_t k);
void launch_f8_matmul(const F8Matmul &f, hipStream_t s);
// Adds the splits' sums (splits > 1).
void launch_f8_sums(const F8Matmul &f, hipStream_t s);

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// Vectors at any element's address: rows of an odd length start anywhere, and
// the memory pipes take vectors at any address.
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// Blocks go to the 8 XCDs round-robin: each XCD gets a contiguous run of n
// pieces of work.
__device__ __forceinline__ int xcd_run(int b, int n) {
    const int q = n >> 3, rem = n & 7, x = b & 7, p = b >> 3;
    return x * q + (x < rem ? x : rem) + p;
}

__device__ __forceinline__ float from_bf16(uint32_t h) { return __uint_as_float(h << 16); }

// Two fp32 values rounded to nearest even, as bf16 pairs (one v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if (BF16) return from_bf16(static_cast<const uint16_t *>(p)[i]);
    return static_cast<const float *>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
    if (BF16)
        static_cast<uint16_t *>(p)[i] = (uint16_t)to_bf16x2(v, v);
    else
        static_cast<float *>(p)[i] = v;
}

// N = 4 or 8 consecutive values from element i on, of which `count` exist
// (the others are 0).
template <bool BF16, int N>
__device__ __forceinline__ void load_n(const void *p, int64_t i, int count, float (&v)[N]) {
    static_assert(N == 4 || N == 8, "vector length");
    if (count >= N) {
        if (BF16) {
            const uint16_t *q = static_cast<const uint16_t *>(p) + i;
            uint32_t w[N / 2];
            if (N == 8) {
                const u32x4 t = *reinterpret_cast<const u32x4_any *>(q);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) w[j] = t[j];
            } else {
                const u32x2 t = *reinterpret_cast<const u32x2_any *>(q);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) w[j] = t[j];
            }
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        } else {
            const float *q = static_cast<const float *>(p) + i;
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const f32x4 t = *reinterpret_cast<const f32x4_any *>(q + 4 * h);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = t[j];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = j < count ? load1<BF16>(p, i + j) : 0.0f;
    }
}

template <bool BF16, int N>
__device__ __forceinline__ void store_n(void *p, int64_t i, int count, const float (&v)[N]) {
    static_assert(N == 4 || N == 8, "vector length");
    if (count >= N) {
        if (BF16) {
            uint16_t *q = static_cast<uint16_t *>(p) + i;
            uint32_t w[N / 2];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) w[j] = to_bf16x2(v[2 * j], v[2 * j + 1]);
            if constexpr (N == 8)
                *reinterpret_cast<u32x4_any *>(q) = u32x4{w[0], w[1], w[2], w[3]};
            else
                *reinterpret_cast<u32x2_any *>(q) = u32x2{w[0], w[1]};
        } else {
            float *q = static_cast<float *>(p) + i;
#pragma unroll
            for (int h = 0; h < N / 4; ++h)
                *reinterpret_cast<f32x4_any *>(q + 4 * h) = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < count) store1<BF16>(p, i + j, v[j]);
    }
}

// N values of a row from column c on, as they lie in memory. Columns past the
// row's end are not there: the vector then starts at the row's last N values,
// and unpack moves what exists to the front. So every lane loads in the same
// instruction, whatever the width, and several loads can be under way before
// the first is unpacked (a branch around each load, with the conversion inside,
// waits for one after the other).
template <bool BF16, int N>
struct Raw {
    uint32_t w[BF16 ? N / 2 : N];
};

template <bool BF16, int N>
__device__ __forceinline__ Raw<BF16, N> load_raw(const void *p, int64_t row, int c, int cols) {
    Raw<BF16, N> o;
    const char *base = static_cast<const char *>(p) + row * (BF16 ? 2 : 4);
    if (cols >= N) {
        const char *q = base + (uint32_t)(c <= cols - N ? c : cols - N) * (BF16 ? 2u : 4u);
        if constexpr (BF16 && N == 4) {
            const u32x2 t = *reinterpret_cast<const u32x2_any *>(q);
            o.w[0] = t[0];
            o.w[1] = t[1];
        } else {
#pragma unroll
            for (int h = 0; h < (BF16 ? N / 8 : N / 4); ++h) {
                const u32x4 t = *reinterpret_cast<const u32x4_any *>(q + 16 * h);
#pragma unroll
                for (int j = 0; j < 4; ++j) o.w[4 * h + j] = t[j];
            }
        }
    } else {
        // shorter than a vector: value by value, the last one again behind the end
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int at = c + j < cols ? c + j : cols - 1;
            if constexpr (BF16) {
                const uint32_t h = reinterpret_cast<const uint16_t *>(base)[at];
                o.w[j / 2] = j % 2 ? o.w[j / 2] | h << 16 : h;
            } else {
                o.w[j] = reinterpret_cast<const uint32_t *>(base)[at];
            }
        }
    }
    return o;
}

// The values, 0 past the row's end. whole: every lane's are there.
template <bool BF16, int N>
__device__ __forceinline__ void unpack(const Raw<BF16, N> &o, int c, int cols, float (&v)[N], bool whole = false) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        v[j] = BF16 ? __uint_as_float(j % 2 ? o.w[j / 2] & 0xffff0000u : o.w[j / 2] << 16)
                    : __uint_as_float(o.w[BF16 ? 0 : j]);
    if (whole) return;
    if (cols % N == 0) {
        const bool there = c < cols;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = there ? v[j] : 0.0f;
    } else if (cols >= N) {
        const int by = c - (cols - N), d = by <= 0 ? 0 : by < N ? by : N;
#pragma unroll
        for (int s = N; s >= 1; s >>= 1) {
            const bool move = d & s;
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = move ? (j + s < N ? v[j + s < N ? j + s : 0] : 0.0f) : v[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = c + j < cols ? v[j] : 0.0f;
    }
}

}  // namespace sm
