// rms_norm.hip -- root-mean-square norm with the residual's addition and an
// output in 8 bits, and its gradients.
//
//   h = x + r, rounded to the type it is stored in
//   rstd = 1 / sqrt(mean_c(h^2) + eps),  xh = h rstd,  y = xh g
//   t = dy g,  dx = dh + rstd (t - xh mean_c(t xh))
//   dg_m = sum of dy xh over worker m's rows
//
// All passes are bound by memory. A row is read once and held in registers by a
// team of lanes, as layer norm's. A block of 128 values that shares a scale of
// the 8-bit output lies in 16 neighbouring lanes: its largest size is four
// exchanges away, and the output costs no pass of its own. It is quantised from fp32: of 6.3 M values
// two to six lie so near the middle of two 8-bit ones that a rounding of rstd or y decides. Measured: 8192 x 768 of
// BF16 with residual to 8 bits 10.5 us a call (44 MB, 4.2 TB/s; one round of rows, so
// latency shows), the gradients of 8 x 1024 x 768 13.5 (50 MB in two launches), one token 10
// (the kernel takes 3.3, the rest is issuing the call). 8192 rows of 4096 in BF16 with residual 42 us
// (6.5 TB/s), their gradients 46 (5.8); 4096 rows of 16384, which are read again for the result and
// for dgamma, 115 and 169 (4.7 and 3.2 TB/s of what they hold).
#include "grad_internal.h"

namespace sm {
namespace {

// The value that a store in the type holds.
template <bool BF16>
__device__ __forceinline__ void round_type(float (&v)[8]) {
    if (BF16)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint32_t w = to_bf16x2(v[j], v[j + 1]);
            v[j] = __uint_as_float(w << 16);
            v[j + 1] = __uint_as_float(w & 0xffff0000u);
        }
}

// A row's columns c .. c + 7. WHOLE: rows of whole vectors, so that a lane has all
// eight or none (those without load the row's first again). Otherwise rows begin
// anywhere; keeping both in one kernel costs 163 registers and half of the waves
// where this takes 86 (8192 x 768 to 8 bits 16.2 us, now 11.6).
template <bool BF16, bool WHOLE>
__device__ __forceinline__ Raw<BF16, 8> fetch8(const void *p, int64_t row, int c, int cols) {
    if constexpr (!WHOLE) return load_raw<BF16, 8>(p, row, c, cols);
    Raw<BF16, 8> o;
    const char *q = static_cast<const char *>(p) + (row + (c < cols ? c : 0)) * (BF16 ? 2 : 4);
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
        const u32x4 t = *reinterpret_cast<const u32x4 *>(q + 16 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[4 * h + j] = t[j];
    }
    return o;
}
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void open8(const Raw<BF16, 8> &o, int c, int cols, float (&v)[8], bool whole) {
    if constexpr (!WHOLE) {
        unpack(o, c, cols, v, whole);
        return;
    }
    const bool there = c < cols;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = BF16 ? (j % 2 ? o.w[j / 2] & 0xffff0000u : o.w[j / 2] << 16) : o.w[BF16 ? 0 : j];
        v[j] = there ? __uint_as_float(w) : 0.0f;
    }
}
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void put8(void *p, int64_t row, int c, int cols, const float (&v)[8]) {
    store_n<BF16>(p, row + c, WHOLE ? (c < cols ? 8 : 0) : left(cols, c), v);
}

// Columns c .. c + 7 of an output row as 8 bits: lanes 16 i .. 16 i + 15 hold a
// block. Every lane of the block calls; columns past the row's end are padding.
template <bool E5M2>
__device__ __forceinline__ void store_f8(const RmsNorm &n, int64_t row, int64_t c, const float (&y)[8]) {
    const int have = left(n.cols, c);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = umax(top, j < have ? finite_size(y[j]) : 0u);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = umax(top, __shfl_xor(top, d));
    if (c >= n.pitch) return;
    const int byte = scale_byte<E5M2>(top);
    const float s = inverse_scale(byte);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < have ? y[j] * s : 0.0f;
    *reinterpret_cast<uint2 *>(n.q + row * n.pitch + c) =
        make_uint2(to_f8x4<E5M2>(v[0], v[1], v[2], v[3]), to_f8x4<E5M2>(v[4], v[5], v[6], v[7]));
    const int64_t block = c / kF8Block;
    const int at = (int)(c % kF8Block) / 8;
    uint8_t *out = n.q_scale + row * n.scale_pitch + block;
    if (at == 0) *out = (uint8_t)byte;
    // padding behind the row's last block
    if (c / kF8Block * kF8Block + kF8Block == n.pitch && at > 0 && block + at < n.scale_pitch) out[at] = kF8Zero;
}

enum { kNoF8 = 0, kE4M3 = 1, kE5M2 = 2 };

template <int F8>
__device__ __forceinline__ void put_f8(const RmsNorm &n, int64_t row, int64_t c, const float (&y)[8]) {
    if constexpr (F8 != kNoF8) store_f8<F8 == kE5M2>(n, row, c, y);
}

// One team per row, `teams` of the grid taking every teams-th row.
template <bool BF16, bool WHOLE, int TS, int NIT, int THREADS, int F8>
__global__ __launch_bounds__(THREADS) void rms_kernel(RmsNorm n) {
    __shared__ float lds[TS > kWave ? 4 * TS / kWave : 1];
    Team<TS> team{lds};
    const int tl = threadIdx.x % TS, cols = (int)n.cols;
    const int64_t teams = (int64_t)gridDim.x * (THREADS / TS);
    float g[NIT][8];
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int c = (i * TS + tl) * 8;
        load_n<false>(n.gamma, c, left(cols, c), g[i]);
    }
    for (int64_t row = (int64_t)blockIdx.x * (THREADS / TS) + threadIdx.x / TS; row < n.rows; row += teams) {
        Raw<BF16, 8> rx[NIT], rr[NIT];
        float v[NIT][8];
        float square = 0.0f;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            rx[i] = fetch8<BF16, WHOLE>(n.x, row * n.cols, c, cols);
            if (n.residual) rr[i] = fetch8<BF16, WHOLE>(n.residual, row * n.cols, c, cols);
        }
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            const bool whole = (i + 1) * TS * 8 <= cols;
            open8<BF16, WHOLE>(rx[i], c, cols, v[i], whole);
            if (n.residual) {
                float r[8];
                open8<BF16, WHOLE>(rr[i], c, cols, r, whole);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
                round_type<BF16>(v[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) square = fmaf(v[i][j], v[i][j], square);
        }
        const float rstd = 1.0f / sqrtf(team.sum(square) / (float)n.cols + n.eps);
        // behind the sum every lane has what it reads of the row: h may be x or the residual
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            if (n.h) put8<BF16, WHOLE>(n.h, row * n.cols, c, cols, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * g[i][j];
            if (n.y) put8<BF16, WHOLE>(n.y, row * n.cols, c, cols, v[i]);
            put_f8<F8>(n, row, c, v[i]);
        }
        if (tl == 0 && n.rstd) n.rstd[row] = rstd;
    }
}

// Rows that do not fit the registers: read once for the sum and once for the
// result. One workgroup per row; a thread reads and writes the same columns in
// both passes.
template <bool BF16, int F8>
__global__ __launch_bounds__(1024) void rms_long_kernel(RmsNorm n) {
    __shared__ float lds[64];
    Team<1024> team{lds};
    auto sum_at = [&](int64_t row, int64_t c, int have, float(&v)[8]) {
        load_n<BF16>(n.x, row * n.cols + c, have, v);
        if (!n.residual) return;
        float r[8];
        load_n<BF16>(n.residual, row * n.cols + c, have, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
        round_type<BF16>(v);
    };
    for (int64_t row = blockIdx.x; row < n.rows; row += gridDim.x) {
        float v[8], square = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            sum_at(row, c, have, v);
            if (n.h) store_n<BF16>(n.h, row * n.cols + c, have, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) square = fmaf(v[j], v[j], square);
        }
        const float rstd = 1.0f / sqrtf(team.sum(square) / (float)n.cols + n.eps);
        // whole waves, so that all lanes of a block take part in its largest size
        for (int64_t c = threadIdx.x * 8; c - (threadIdx.x % kWave) * 8 < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            float g[8];
            if (n.h)
                load_n<BF16>(n.h, row * n.cols + c, have, v);
            else
                sum_at(row, c, have, v);
            load_n<false>(n.gamma, c, have, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * g[j];
            if (n.y) store_n<BF16>(n.y, row * n.cols + c, have, v);
            put_f8<F8>(n, row, c, v);
        }
        if (threadIdx.x == 0 && n.rstd) n.rstd[row] = rstd;
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// A sum of `part`'s rows: the gradient itself where there is one part.
template <int N>
__device__ __forceinline__ void write_sum(const RmsGrad &n, int64_t worker, int64_t part, int64_t c, int have,
                                          const float (&v)[N]) {
    if (have <= 0) return;
    if (n.parts > 1)
        store_n<false>(n.partial, (worker * n.parts + part) * n.cols + c, have, v);
    else if (n.grad_bf16)
        store_n<true>(n.dgamma, worker * n.cols + c, have, v);
    else
        store_n<false>(n.dgamma, worker * n.cols + c, have, v);
}

__device__ __forceinline__ int64_t rows_per_part(const RmsGrad &n) { return (n.rows + n.parts - 1) / n.parts; }

template <bool BF16, bool WHOLE, int TS, int NIT, int THREADS>
__global__ __launch_bounds__(THREADS) void rms_grad_kernel(RmsGrad n) {
    constexpr int kTeams = THREADS / TS;
    __shared__ float sums[kTeams > 1 ? kTeams * NIT * TS * 8 : 1];  // [kTeams][NIT][TS][8]
    __shared__ float lds[TS > kWave ? 4 * TS / kWave : 1];
    Team<TS> team{lds};
    const int tl = threadIdx.x % TS, tm = threadIdx.x / TS, cols = (int)n.cols;
    const int64_t worker = blockIdx.x / n.parts, part = blockIdx.x % n.parts;
    const int64_t begin = part * rows_per_part(n);
    const int64_t end = begin + rows_per_part(n) < n.rows ? begin + rows_per_part(n) : n.rows;
    const float inv = 1.0f / (float)n.cols;
    float g[NIT][8], dg[NIT][8] = {};
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int c = (i * TS + tl) * 8;
        load_n<false>(n.gamma, c, left(cols, c), g[i]);
    }
    Raw<BF16, 8> rh[NIT], rd[NIT], rs[NIT];
    float next_rstd = 0.0f;
    auto fetch = [&](int64_t r) {
        const int64_t row = worker * n.rows + r;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            rh[i] = fetch8<BF16, WHOLE>(n.h, row * n.cols, c, cols);
            rd[i] = fetch8<BF16, WHOLE>(n.dy, row * n.cols, c, cols);
            if (n.dh) rs[i] = fetch8<BF16, WHOLE>(n.dh, row * n.cols, c, cols);
        }
        next_rstd = n.rstd[row];
    };
    // a wave has room for the next row while it works on one; for more columns other waves
    // fill the wait
    constexpr bool kAhead = TS <= kWave && BF16;
    if (kAhead && begin + tm < end) fetch(begin + tm);
    for (int64_t r = begin + tm; r < end; r += kTeams) {
        const int64_t row = worker * n.rows + r;
        if (!kAhead) fetch(r);
        float x[NIT][8], d[NIT][8], s[NIT][8];
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            const bool whole = (i + 1) * TS * 8 <= cols;
            open8<BF16, WHOLE>(rh[i], c, cols, x[i], whole);
            open8<BF16, WHOLE>(rd[i], c, cols, d[i], whole);
            if (n.dh) open8<BF16, WHOLE>(rs[i], c, cols, s[i], whole);
        }
        const float rstd = next_rstd;
        if (kAhead && r + kTeams < end) fetch(r + kTeams);
        float along = 0.0f;
#pragma unroll
        for (int i = 0; i < NIT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] *= rstd;
                dg[i][j] = fmaf(d[i][j], x[i][j], dg[i][j]);
                d[i][j] *= g[i][j];
                along = fmaf(d[i][j], x[i][j], along);
            }
        if (!n.dx) continue;
        along = team.sum(along) * inv;
        // behind the sum every lane has what it reads of the row: dx may be dy or dh
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = rstd * (d[i][j] - x[i][j] * along);
                if (n.dh) x[i][j] += s[i][j];
            }
            put8<BF16, WHOLE>(n.dx, row * n.cols, c, cols, x[i]);
        }
    }
    if (!n.dgamma) return;
    if constexpr (kTeams == 1) {
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            write_sum(n, worker, part, c, left(cols, c), dg[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NIT; ++i) store_n<false>(sums, ((tm * NIT + i) * TS + tl) * 8, 8, dg[i]);
        __syncthreads();
        for (int c = threadIdx.x * 4; c < NIT * TS * 8; c += THREADS * 4) {
            float v[4] = {};
#pragma unroll
            for (int t = 0; t < kTeams; ++t) {
                float w[4];
                load_n<false>(sums, t * NIT * TS * 8 + c, 4, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += w[j];
            }
            write_sum(n, worker, part, c, (int)(n.cols - c < 4 ? n.cols - c : 4), v);
        }
    }
}

// Rows that do not fit the registers: dx, reading the row twice.
template <bool BF16>
__global__ __launch_bounds__(1024) void rms_grad_long_kernel(RmsGrad n) {
    __shared__ float lds[64];
    Team<1024> team{lds};
    const float inv = 1.0f / (float)n.cols;
    for (int64_t row = blockIdx.x; row < n.workers * n.rows; row += gridDim.x) {
        const int64_t at = row * n.cols;
        const float rstd = n.rstd[row];
        float x[8], d[8], g[8], along = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            load_n<BF16>(n.h, at + c, have, x);
            load_n<BF16>(n.dy, at + c, have, d);
            load_n<false>(n.gamma, c, have, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) along = fmaf(d[j] * g[j], x[j] * rstd, along);
        }
        along = team.sum(along) * inv;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            float s[8];
            load_n<BF16>(n.h, at + c, have, x);
            load_n<BF16>(n.dy, at + c, have, d);
            load_n<false>(n.gamma, c, have, g);
            load_n<BF16>(n.dh, at + c, n.dh ? have : 0, s);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = rstd * (d[j] * g[j] - x[j] * rstd * along) + s[j];
            store_n<BF16>(n.dx, at + c, have, x);
        }
    }
}

// The columns' sums of such rows: one wave per 512 columns and part.
template <bool BF16>
__global__ __launch_bounds__(64) void rms_grad_columns_kernel(RmsGrad n, int blocks) {
    const int64_t c = (int64_t)(blockIdx.x % blocks) * 512 + threadIdx.x * 8;
    const int64_t part = blockIdx.x / blocks % n.parts, worker = blockIdx.x / blocks / n.parts;
    const int have = left(n.cols, c);
    const int64_t begin = part * rows_per_part(n);
    const int64_t end = begin + rows_per_part(n) < n.rows ? begin + rows_per_part(n) : n.rows;
    float dg[8] = {};
    for (int64_t r = begin; r < end; ++r) {
        const int64_t row = worker * n.rows + r;
        const float rstd = n.rstd[row];
        float x[8], d[8];
        load_n<BF16>(n.h, row * n.cols + c, have, x);
        load_n<BF16>(n.dy, row * n.cols + c, have, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[j] = fmaf(d[j], x[j] * rstd, dg[j]);
    }
    write_sum(n, worker, part, c, have, dg);
}

// 64 columns of one worker's sum: eight waves add an eighth of the parts each,
// in order, and the first adds the eight.
template <bool GB>
__global__ __launch_bounds__(512) void rms_sums_kernel(RmsGrad n, int blocks) {
    __shared__ float lds[8][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)(blockIdx.x % blocks) * kWave + lane;
    const int64_t worker = blockIdx.x / blocks;
    float total = 0.0f;
    if (c < n.cols) {
        const int each = (n.parts + 7) / 8;
        const int end = (wave + 1) * each < n.parts ? (wave + 1) * each : n.parts;
        const float *p = n.partial + worker * n.parts * n.cols + c;
#pragma unroll 8
        for (int i = wave * each; i < end; ++i) total += p[(int64_t)i * n.cols];
    }
    lds[wave][lane] = total;
    __syncthreads();
    if (wave == 0 && c < n.cols)
        store1<GB>(n.dgamma, worker * n.cols + c,
                   ((lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane])) +
                       ((lds[4][lane] + lds[5][lane]) + (lds[6][lane] + lds[7][lane])));
}

// A team's lanes, chunks a lane, and a workgroup's threads (those of one team
// where it is more than a wave: its sums meet at barriers). 16 lanes at least:
// a block of the 8-bit output.
template <int TS_, int NIT_, int THREADS_>
struct Width {
    static constexpr int TS = TS_, NIT = NIT_, THREADS = THREADS_;
    static_assert(TS <= kWave || THREADS == TS, "teams of a workgroup do not meet");
    static_assert(TS >= 16, "a block of the 8-bit output in one team");
};

// f(Width) for a row of `cols` values.
template <class F>
void by_width(int64_t cols, F &&f) {
    if (cols <= 128)
        f(Width<16, 1, 256>{});
    else if (cols <= 256)
        f(Width<32, 1, 256>{});
    else if (cols <= 512)
        f(Width<64, 1, 256>{});
    else if (cols <= 1024)
        f(Width<64, 2, 256>{});
    else if (cols <= 2048)
        f(Width<128, 2, 128>{});
    else if (cols <= 4096)
        f(Width<256, 2, 256>{});
    else
        f(Width<512, 2, 512>{});
}
constexpr int64_t kLongRow = 8192;

template <bool BF16, int F8>
void launch_rms(const RmsNorm &n, hipStream_t s) {
    if (n.cols > kLongRow) {
        rms_long_kernel<BF16, F8><<<dim3((unsigned)(n.rows < 4096 ? n.rows : 4096)), 1024, 0, s>>>(n);
        return;
    }
    auto f = [&](auto w) {
        constexpr int TS = decltype(w)::TS, NIT = decltype(w)::NIT, THREADS = decltype(w)::THREADS;
        const int64_t teams = THREADS / TS, blocks = (n.rows + teams - 1) / teams;
        const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
        if (n.cols % 8 == 0)
            rms_kernel<BF16, true, TS, NIT, THREADS, F8><<<grid, THREADS, 0, s>>>(n);
        else
            rms_kernel<BF16, false, TS, NIT, THREADS, F8><<<grid, THREADS, 0, s>>>(n);
    };
    by_width(n.cols, f);
}

template <bool BF16>
void launch_rms_type(const RmsNorm &n, hipStream_t s) {
    if (!n.q)
        launch_rms<BF16, kNoF8>(n, s);
    else if (n.e5m2)
        launch_rms<BF16, kE5M2>(n, s);
    else
        launch_rms<BF16, kE4M3>(n, s);
}

template <bool BF16>
void launch_grad(const RmsGrad &n, hipStream_t s) {
    if (n.cols > kLongRow) {
        const int64_t rows = n.workers * n.rows;
        const int blocks = (int)((n.cols + 511) / 512);
        // the columns first: dx may be dy
        if (n.dgamma)
            rms_grad_columns_kernel<BF16><<<dim3((unsigned)(n.workers * n.parts * blocks)), 64, 0, s>>>(n, blocks);
        if (n.dx) rms_grad_long_kernel<BF16><<<dim3((unsigned)(rows < 4096 ? rows : 4096)), 1024, 0, s>>>(n);
        return;
    }
    auto f = [&](auto w) {
        constexpr int TS = decltype(w)::TS, NIT = decltype(w)::NIT, THREADS = decltype(w)::THREADS;
        const dim3 grid((unsigned)(n.workers * n.parts));
        if (n.cols % 8 == 0)
            rms_grad_kernel<BF16, true, TS, NIT, THREADS><<<grid, THREADS, 0, s>>>(n);
        else
            rms_grad_kernel<BF16, false, TS, NIT, THREADS><<<grid, THREADS, 0, s>>>(n);
    };
    by_width(n.cols, f);
}

}  // namespace

void launch_rms_norm(const RmsNorm &n, hipStream_t s) {
    n.bf16 ? launch_rms_type<true>(n, s) : launch_rms_type<false>(n, s);
}

// Two rows a team at least, and at most as many waves as run at once.
int32_t rms_parts(int32_t workers, int64_t rows, int64_t cols) {
    int64_t teams = 8, waves = 4, most = 4096;
    if (cols <= kLongRow) {
        auto f = [&](auto w) {
            teams = w.THREADS / w.TS;
            waves = w.THREADS / kWave;
            most = w.NIT > 1 ? 2048 : 4096;
        };
        by_width(cols, f);
    }
    const int64_t each = most / waves / workers > 1 ? most / waves / workers : 1;
    const int64_t parts = (rows + teams * 2 - 1) / (teams * 2);
    return (int32_t)(parts < each ? parts : each);
}

void launch_rms_norm_backward(const RmsGrad &n, hipStream_t s) {
    n.bf16 ? launch_grad<true>(n, s) : launch_grad<false>(n, s);
}

void launch_rms_norm_sums(const RmsGrad &n, hipStream_t s) {
    const int blocks = (int)((n.cols + kWave - 1) / kWave);
    const dim3 grid((unsigned)(n.workers * blocks));
    if (n.grad_bf16)
        rms_sums_kernel<true><<<grid, 512, 0, s>>>(n, blocks);
    else
        rms_sums_kernel<false><<<grid, 512, 0, s>>>(n, blocks);
}

}  // namespace sm
