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
// Root-mean-square norm.
// ---------------------------------------------------------------------------
struct RmsNorm {
    const void *x, *residual;  // residual may be null
    const float *gamma;
    void *h, *y;               // either may be null
    uint8_t *q, *q_scale;      // both or neither
    float *rstd;               // may be null
    int64_t rows, cols;
    int64_t pitch, scale_pitch;  // of q: a row's bytes
    float eps;
    bool bf16, e5m2;
};
void launch_rms_norm(const RmsNorm &n, hipStream_t s);

struct RmsGrad {
    const void *dy, *dh, *h;  // dh may be null
    const float *gamma, *rstd;
    void *dx, *dgamma;        // either may be null
    float *partial;  // [workers][parts][cols] sums of dy * xh; unused where parts = 1
    int64_t rows;    // per worker
    int64_t cols;
    int32_t workers;
    int32_t parts;  // blocks of rows per worker, each with a sum of its own
    bool bf16, grad_bf16;
};
int32_t rms_parts(int32_t workers, int64_t rows, int64_t cols);
void launch_rms_norm_backward(const RmsGrad &n, hipStream_t s);
// Adds the parts' sums (parts > 1).
void launch_rms_norm_sums(const RmsGrad &n, hipStream_t s);

// ---------------------------------------------------------------------------
// Softmax cross entropy of an output layer.
// ---------------------------------------------------------------------------
constexpr int kLossTile = 256;      // rows and columns of the largest tile
constexpr int kLossSlice = 64;      // k of a slice in LDS
constexpr int kLossWideSlice = 32;  // the same where a is fp32
constexpr int kLossPlanes = 3, kLossPairs = 6;
inline int64_t loss_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }  // entries of a plane's row

// A matrix as BF16 planes [planes][rows][pitch].
struct LossPlanes {
    const void *in;
    uint16_t *out[kLossPlanes];
    const void *targets;  // of the rows, or null: rows without a target become zeros, and
                          // each row's target (-1: none), lse / log 2 and scale * dloss are written
    const float *lse, *dloss;
    int32_t *row_target;
    float *row_base, *row_d;
    int64_t rows, cols, pitch, vocab;
    float scale;
    int32_t planes;
    bool bf16, targets64;
};
void launch_loss_planes(const LossPlanes &f, hipStream_t s);

// The tiles of a product, and the parts of k.
struct LossTiles {
    int32_t tm, tn, splits;
};
// Tiles and workspace of the loss (logits) and of its gradients. The types are signmuon_dtype's.
struct LossPlan {
    int64_t piece, pitch;  // entries of the vocabulary at a time; of a plane's row
    LossTiles logits, dx, dw;
    bool few, g32;
    bool parts;            // of dx, summed by a launch of their own
    size_t x, w, partial, state, target, row[3], g, sum, part, total;
};
LossPlan loss_plan(int64_t tokens, int64_t vocab, int64_t cols, int x_dtype, int w_dtype);
LossPlan loss_grad_plan(int64_t workers, int64_t tokens, int64_t vocab, int64_t cols, int x_dtype, int w_dtype,
                        int grad_dtype, bool want_dw);

// A product a b^T of planes, out [m][n], sums over k and over pairs of planes.
struct LossTile {
    const void *a[kLossPlanes], *b[kLossPlanes];  // BF16; a[0] fp32 where g32 and a is g
    int64_t a_pitch, b_pitch;  // bytes of a row in memory
    int64_t a_batch, b_batch;  // bytes between batch entries
    int64_t m, n, k;
    int32_t batch, pairs;
    int32_t splits, chunk;     // chunk: slices of a split, of all pairs' slices in a row
    uint32_t order_a, order_b;  // the planes of pair i in bits 2 i on
    int32_t tm, tn;            // the tile: 256 x 256, 128 x 128, or between: 256 x 128, a fp32: 128 x 256
    int32_t planes;            // of an fp32 a: 1 or 3
    bool g32;                  // g is fp32, not BF16
    // logits
    const void *rows[3];       // 4 bytes a row, row_step bytes apart: the targets, and for g what LossPlanes writes
    int32_t row_step;
    float2 *partial;           // [columns of tn / 2][m]: maximum and sum, in units of log 2
    float *target;             // [m] logit of the target
    void *g;                   // [m][g_pitch]
    int64_t g_pitch;
    const void *plain_a, *plain_b;  // the operands that the planes were made of, where one is in several: [m][k]
    bool plain_a16, plain_b16;      // and [n][k], in BF16 or fp32
    int64_t vocab0;            // the piece's first entry
    float factor;              // scale / log 2
    // values
    void *out;
    int64_t out_batch;         // rows between batch entries, and between parts of k
    int64_t out_pitch;         // entries of a row: n, or for parts of logits more, which hold nothing
    bool out_bf16, add;        // add to what out holds (dw alone)
};
// Whether out's rows are whole vectors; where they are not, tiles are of 128 x 128.
inline bool loss_even(const LossTile &f) { return f.out_pitch % (f.out_bf16 ? 8 : 4) == 0; }
// Logits in parts of k go to out, and launch_loss_parts makes of them what the tiles make of whole ones.
void launch_loss_logits(const LossTile &f, bool grad, hipStream_t s);
constexpr int kLossBlock = 256;  // columns of a row that share a maximum and a sum there
void launch_loss_parts(const LossTile &f, bool grad, hipStream_t s);
void launch_loss_dx(const LossTile &f, hipStream_t s);
void launch_loss_dw(const LossTile &f, hipStream_t s);

struct LossJoin {
    const float2 *partial;
    float2 *state;  // [rows] between pieces of the vocabulary
    const float *target;
    const void *targets;
    float *loss, *lse;
    int64_t rows, blocks, vocab;
    int32_t group;  // rows of a workgroup
    bool first, last, targets64;
};
void launch_loss_join(LossJoin f, hipStream_t s);

struct LossSums {
    const float *partial;  // [splits], pitch entries apart
    const void *prev;      // added; null: nothing
    void *out;
    int64_t total, pitch;
    int32_t splits;
    bool prev_bf16, out_bf16;
};
void launch_loss_sums(const LossSums &f, hipStream_t s);

// ---------------------------------------------------------------------------
// Gradient norms and clipping.
// ---------------------------------------------------------------------------
constexpr int kClipUnit = 16384;   // entries of a tensor and worker that a workgroup takes,
constexpr int kClipSmallUnit = 2048;  // or, of few entries in all, these
constexpr int kClipFew = 256;      // partial sums of a worker that every workgroup may add itself
constexpr int kClipTensors = 96;   // of one launch: its descriptors are the kernel's argument

struct ClipBatch {
    const void *grad[kClipTensors];  // [workers][n]
    void *out[kClipTensors];
    int64_t n[kClipTensors];
    int32_t first[kClipTensors];     // unit of the batch that the tensor begins with
    bool bf16[kClipTensors];
    double *partial;                 // [workers][units]
    const float *factors;            // [workers], of more than kClipFew units
    float *norms;                    // [workers], written by the scaling of up to kClipFew units
    float most;
    int32_t unit;                    // entries of one
    int64_t units;                   // of a worker, all batches
    int64_t unit0;                   // that this batch begins with
    int32_t batch_units, tensors, workers;
};
void launch_clip_norm(const ClipBatch &b, hipStream_t s);
void launch_clip_scale(const ClipBatch &b, hipStream_t s);

struct ClipFinish {
    const double *partial;
    float *norms, *factors;  // [workers]
    int64_t units;
    float most;
    int32_t workers;
};
void launch_clip_finish(const ClipFinish &f, hipStream_t s);

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

constexpr int kWave = 64;

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

// ---------------------------------------------------------------------------
// Rows held by teams of lanes
// ---------------------------------------------------------------------------
// Sums over a team of TS lanes (a part of a wave, or a whole workgroup).
template <int TS>
struct Team {
    float *lds;  // TS > 64: [2][TS / 64][2]
    int parity = 0;

    __device__ __forceinline__ void sum2(float &a, float &b) {
#pragma unroll
        for (int d = 1; d < (TS < kWave ? TS : kWave); d <<= 1) {
            a += __shfl_xor(a, d);
            b += __shfl_xor(b, d);
        }
        if constexpr (TS > kWave) {
            constexpr int W = TS / kWave;
            float *at = lds + parity * 2 * W;
            parity ^= 1;  // the next sums use the other half: one barrier each
            if ((threadIdx.x & (kWave - 1)) == 0) {
                at[2 * (threadIdx.x / kWave)] = a;
                at[2 * (threadIdx.x / kWave) + 1] = b;
            }
            __syncthreads();
            a = b = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                a += at[2 * w];
                b += at[2 * w + 1];
            }
        }
    }
    __device__ __forceinline__ float sum(float a) {
#pragma unroll
        for (int d = 1; d < (TS < kWave ? TS : kWave); d <<= 1) a += __shfl_xor(a, d);
        if constexpr (TS > kWave) {
            constexpr int W = TS / kWave;
            float *at = lds + parity * 2 * W;
            parity ^= 1;
            if ((threadIdx.x & (kWave - 1)) == 0) at[threadIdx.x / kWave] = a;
            __syncthreads();
            a = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) a += at[w];
        }
        return a;
    }
};

__device__ __forceinline__ int left(int cols, int c) {  // values of a chunk at column c
    return cols - c < 0 ? 0 : cols - c < 8 ? cols - c : 8;
}

// ---------------------------------------------------------------------------
// Quantisation of a block of 128 values
// ---------------------------------------------------------------------------
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

// ---------------------------------------------------------------------------
// Tiles of matrix products, fed straight into LDS
// ---------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ int first_lane(int v) { return __builtin_amdgcn_readfirstlane(v); }

// v is computed here, not behind a later branch.
__device__ __forceinline__ void pin(f32x16 &v) { asm volatile("" : "+a"(v)); }

// Zeros written straight to where they are kept (one zero for all of them would
// take sixteen registers of its own).
__device__ __forceinline__ f32x16 zeros() {
    float z = 0.0f;
    asm volatile("" : "+v"(z));
    return f32x16{z, z, z, z, z, z, z, z, z, z, z, z, z, z, z, z};
}

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

// A load of 16 bytes a lane straight into LDS at lds + 16 * lane.
// Asm without outputs, so that the compiler does not order every LDS read
// behind the loads in flight; M0 is reserved, and nothing else here reads it.
__device__ __forceinline__ void load16_lds(uint32_t lds, uint32_t offset, u32x4 buffer) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(offset), "s"(buffer)
                 : "memory");
}
// The same of 4 bytes a lane, at lds + 4 * lane.
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

}  // namespace sm
