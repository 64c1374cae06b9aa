// layer_norm.hip -- layer norm and its gradients.
//
//   xh = (x - mean) rstd,  y = xh g + b
//   t = dy g,  dx = rstd (t - mean_c(t) - xh mean_c(t xh))
//   dg_m = sum of dy xh and db_m = sum of dy over worker m's rows
//
// Both passes are bound by memory: the forward reads x and writes y, the
// backward reads x and dy and writes dx. Each row is read once and held in
// registers by a team of lanes (8 values a lane and chunk): 8 to 64 lanes of a
// wave for up to 1024 columns, a workgroup of 128 to 512 for up to 8192; longer
// rows are read again from the caches. The variance is summed from the differences
// to the mean. Backward, BF16 with F32 sums: 16384 x 4096 85 us (4.7 TB/s of the
// least traffic, the rate of a large copy), 1 worker x 8192 x 1024 17 us, 8 workers
// x 1024 x 768 13.1 us, of which about 5 us are the launch of the second kernel and
// its pass over the partial rows.
//
// The weight's gradients are sums down the columns, over rows that many teams
// hold. A lane keeps the same columns for every row of its team and adds them
// in registers; the teams of a workgroup are added through LDS, and each
// workgroup writes one partial row, added in order by norm_sums_kernel. So the
// gradients cost no second pass over x and dy, no atomics, and have one order
// of addition on every run.
#include "grad_internal.h"

namespace sm {
namespace {

// One team per row, `teams` of the grid taking every teams-th row.
template <bool BF16, int TS, int NIT, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_kernel(Norm n) {
    __shared__ float lds[TS > kWave ? 4 * TS / kWave : 1];
    Team<TS> team{lds};
    const int tl = threadIdx.x % TS, cols = (int)n.cols;
    const int64_t teams = (int64_t)gridDim.x * (THREADS / TS);
    const float inv = 1.0f / (float)n.cols;
    float g[NIT][8], b[NIT][8];
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int c = (i * TS + tl) * 8;
        load_n<false>(n.gamma, c, left(cols, c), g[i]);
        load_n<false>(n.beta, c, n.beta ? left(cols, c) : 0, b[i]);
    }
    for (int64_t row = (int64_t)blockIdx.x * (THREADS / TS) + threadIdx.x / TS; row < n.rows; row += teams) {
        Raw<BF16, 8> raw[NIT];
        float v[NIT][8];
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < NIT; ++i) raw[i] = load_raw<BF16, 8>(n.x, row * n.cols, (i * TS + tl) * 8, cols);
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            unpack(raw[i], (i * TS + tl) * 8, cols, v[i], (i + 1) * TS * 8 <= cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) total += v[i][j];
        }
        const float mean = team.sum(total) * inv;
        float square = 0.0f;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int have = left(cols, (i * TS + tl) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] -= mean;
                if (j < have) square = fmaf(v[i][j], v[i][j], square);
            }
        }
        const float rstd = 1.0f / sqrtf(team.sum(square) * inv + n.eps);
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[i][j], b[i][j]);
            store_n<BF16>(n.y, row * n.cols + c, left(cols, c), v[i]);
        }
        if (tl == 0) {
            if (n.mean) n.mean[row] = mean;
            if (n.rstd) n.rstd[row] = rstd;
        }
    }
}

// Rows that do not fit the registers: read once for each of mean, variance and
// result. One workgroup per row.
template <bool BF16>
__global__ __launch_bounds__(1024) void norm_long_kernel(Norm n) {
    __shared__ float lds[64];
    Team<1024> team{lds};
    const float inv = 1.0f / (float)n.cols;
    for (int64_t row = blockIdx.x; row < n.rows; row += gridDim.x) {
        const int64_t at = row * n.cols;
        float v[8], total = 0.0f, square = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            load_n<BF16>(n.x, at + c, left(n.cols, c), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) total += v[j];
        }
        const float mean = team.sum(total) * inv;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            load_n<BF16>(n.x, at + c, have, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < have) square = fmaf(v[j] - mean, v[j] - mean, square);
        }
        const float rstd = 1.0f / sqrtf(team.sum(square) * inv + n.eps);
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            float g[8], b[8];
            load_n<BF16>(n.x, at + c, have, v);
            load_n<false>(n.gamma, c, have, g);
            load_n<false>(n.beta, c, n.beta ? have : 0, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = fmaf((v[j] - mean) * rstd, g[j], b[j]);
            store_n<BF16>(n.y, at + c, have, v);
        }
        if (threadIdx.x == 0) {
            if (n.mean) n.mean[row] = mean;
            if (n.rstd) n.rstd[row] = rstd;
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// A sum of `part`'s rows: the gradient itself where there is one part.
template <int N>
__device__ __forceinline__ void write_sum(const NormGrad &n, int64_t worker, int64_t part, int which, int64_t c,
                                          int have, const float (&v)[N]) {
    if (have <= 0) return;
    if (n.parts > 1) {
        store_n<false>(n.partial, ((worker * n.parts + part) * 2 + which) * n.cols + c, have, v);
        return;
    }
    void *out = which ? n.dbeta : n.dgamma;
    if (n.grad_bf16)
        store_n<true>(out, worker * n.cols + c, have, v);
    else
        store_n<false>(out, worker * n.cols + c, have, v);
}

__device__ __forceinline__ int64_t rows_per_part(const NormGrad &n) { return (n.rows + n.parts - 1) / n.parts; }

template <bool BF16, int TS, int NIT, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_grad_kernel(NormGrad n) {
    constexpr int kTeams = THREADS / TS;
    // the teams' sums of one kind, [kTeams][NIT][TS][8]
    __shared__ float sums[kTeams > 1 ? kTeams * NIT * TS * 8 : 1];
    __shared__ float lds[TS > kWave ? 4 * TS / kWave : 1];
    Team<TS> team{lds};
    const int tl = threadIdx.x % TS, tm = threadIdx.x / TS, cols = (int)n.cols;
    const int64_t worker = blockIdx.x / n.parts, part = blockIdx.x % n.parts;
    const int64_t begin = part * rows_per_part(n);
    const int64_t end = begin + rows_per_part(n) < n.rows ? begin + rows_per_part(n) : n.rows;
    const float inv = 1.0f / (float)n.cols;
    float g[NIT][8], dg[NIT][8] = {}, db[NIT][8] = {};
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int c = (i * TS + tl) * 8;
        load_n<false>(n.gamma, c, left(cols, c), g[i]);
    }
    Raw<BF16, 8> rx[NIT], rd[NIT];
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto fetch = [&](int64_t r) {
        const int64_t row = worker * n.rows + r;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            rx[i] = load_raw<BF16, 8>(n.x, row * n.cols, c, cols);
            rd[i] = load_raw<BF16, 8>(n.dy, row * n.cols, c, cols);
        }
        next_mean = n.mean[row];
        next_rstd = n.rstd[row];
    };
    // a wave with up to 1024 columns has room for the next row while it works on
    // one; for more columns other waves fill the wait
    constexpr bool kAhead = TS <= kWave && NIT <= 2;
    if (kAhead && begin + tm < end) fetch(begin + tm);
    for (int64_t r = begin + tm; r < end; r += kTeams) {
        const int64_t row = worker * n.rows + r;
        if (!kAhead) fetch(r);
        float x[NIT][8], d[NIT][8];
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
            unpack(rx[i], c, cols, x[i], (i + 1) * TS * 8 <= cols);
            unpack(rd[i], c, cols, d[i], (i + 1) * TS * 8 <= cols);
        }
        const float mean = next_mean, rstd = next_rstd;
        if (kAhead && r + kTeams < end) fetch(r + kTeams);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int have = left(cols, (i * TS + tl) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = j < have ? (x[i][j] - mean) * rstd : 0.0f;
                x[i][j] = xh;
                dg[i][j] = fmaf(d[i][j], xh, dg[i][j]);
                db[i][j] += d[i][j];
                d[i][j] *= g[i][j];
                s1 += d[i][j];
                s2 = fmaf(d[i][j], xh, s2);
            }
        }
        if (!n.dx) continue;
        team.sum2(s1, s2);
        s1 *= inv;
        s2 *= inv;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int c = (i * TS + tl) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = rstd * (d[i][j] - s1 - x[i][j] * s2);
            store_n<BF16>(n.dx, row * n.cols + c, left(cols, c), x[i]);
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!(which ? n.dbeta : n.dgamma)) continue;
        if constexpr (kTeams == 1) {
#pragma unroll
            for (int i = 0; i < NIT; ++i) {
                const int c = (i * TS + tl) * 8;
                write_sum(n, worker, part, which, c, left(cols, c), which ? db[i] : dg[i]);
            }
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NIT; ++i)
                store_n<false>(sums, ((tm * NIT + i) * TS + tl) * 8, 8, which ? db[i] : dg[i]);
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
                write_sum(n, worker, part, which, c, (int)(n.cols - c < 4 ? n.cols - c : 4), v);
            }
        }
    }
}

// Rows that do not fit the registers: dx, reading the row twice.
template <bool BF16>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(NormGrad n) {
    __shared__ float lds[64];
    Team<1024> team{lds};
    const float inv = 1.0f / (float)n.cols;
    for (int64_t row = blockIdx.x; row < n.workers * n.rows; row += gridDim.x) {
        const int64_t at = row * n.cols;
        const float mean = n.mean[row], rstd = n.rstd[row];
        float x[8], d[8], g[8], s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            load_n<BF16>(n.x, at + c, have, x);
            load_n<BF16>(n.dy, at + c, have, d);
            load_n<false>(n.gamma, c, have, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s1 = fmaf(d[j], g[j], s1);
                s2 = fmaf(d[j] * g[j], j < have ? (x[j] - mean) * rstd : 0.0f, s2);
            }
        }
        team.sum2(s1, s2);
        s1 *= inv;
        s2 *= inv;
        for (int64_t c = threadIdx.x * 8; c < n.cols; c += 8192) {
            const int have = left(n.cols, c);
            load_n<BF16>(n.x, at + c, have, x);
            load_n<BF16>(n.dy, at + c, have, d);
            load_n<false>(n.gamma, c, have, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = rstd * (d[j] * g[j] - s1 - (x[j] - mean) * rstd * s2);
            store_n<BF16>(n.dx, at + c, have, x);
        }
    }
}

// The columns' sums of such rows: one wave per 512 columns and part.
template <bool BF16>
__global__ __launch_bounds__(64) void norm_grad_columns_kernel(NormGrad n, int blocks) {
    const int64_t c = (int64_t)(blockIdx.x % blocks) * 512 + threadIdx.x * 8;
    const int64_t part = blockIdx.x / blocks % n.parts, worker = blockIdx.x / blocks / n.parts;
    const int have = left(n.cols, c);
    const int64_t begin = part * rows_per_part(n);
    const int64_t end = begin + rows_per_part(n) < n.rows ? begin + rows_per_part(n) : n.rows;
    float dg[8] = {}, db[8] = {};
    for (int64_t r = begin; r < end; ++r) {
        const int64_t row = worker * n.rows + r;
        const float mean = n.mean[row], rstd = n.rstd[row];
        float x[8], d[8];
        load_n<BF16>(n.x, row * n.cols + c, have, x);
        load_n<BF16>(n.dy, row * n.cols + c, have, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dg[j] = fmaf(d[j], (x[j] - mean) * rstd, dg[j]);
            db[j] += d[j];
        }
    }
    if (n.dgamma) write_sum(n, worker, part, 0, c, have, dg);
    if (n.dbeta) write_sum(n, worker, part, 1, c, have, db);
}

// 64 columns of one sum of one worker: eight waves add an eighth of the parts
// each, in order, and the first adds the eight.
template <bool GB>
__global__ __launch_bounds__(512) void norm_sums_kernel(NormGrad n, int blocks) {
    __shared__ float lds[8][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)(blockIdx.x % blocks) * kWave + lane;
    const int which = blockIdx.x / blocks & 1;
    const int64_t worker = blockIdx.x / blocks >> 1;
    void *out = which ? n.dbeta : n.dgamma;
    if (!out) return;
    float total = 0.0f;
    if (c < n.cols) {
        const int each = (n.parts + 7) / 8;
        const int end = (wave + 1) * each < n.parts ? (wave + 1) * each : n.parts;
        const float *p = n.partial + (worker * n.parts * 2 + which) * n.cols + c;
#pragma unroll 8
        for (int i = wave * each; i < end; ++i) total += p[(int64_t)i * 2 * n.cols];
    }
    lds[wave][lane] = total;
    __syncthreads();
    if (wave == 0 && c < n.cols)
        store1<GB>(out, worker * n.cols + c,
                   ((lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane])) +
                       ((lds[4][lane] + lds[5][lane]) + (lds[6][lane] + lds[7][lane])));
}

// A team's lanes, chunks a lane, and a workgroup's threads (those of one team
// where it is more than a wave: its sums meet at barriers).
template <int TS_, int NIT_, int THREADS_>
struct Width {
    static constexpr int TS = TS_, NIT = NIT_, THREADS = THREADS_;
    static_assert(TS <= kWave || THREADS == TS, "teams of a workgroup do not meet");
};

// f(Width) for a row of `cols` values.
template <class F>
void by_width(int64_t cols, F &&f) {
    if (cols <= 64)
        f(Width<8, 1, 256>{});
    else if (cols <= 128)
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
// Columns that a workgroup's registers hold without spilling in the backward pass:
// with four chunks a lane, 700 x 12000 takes 109 us there and 43 us reading twice. The
// forward pass, which holds less a lane, goes by the same limit: 700 x 12000 takes
// 19 us so (F32, 3.5 TB/s of the least traffic), 4096 x 16384 76 us (BF16, 3.5 TB/s).
constexpr int64_t kLongRow = 8192;

}  // namespace

void launch_layer_norm(const Norm &n, hipStream_t s) {
    if (n.cols > kLongRow) {
        const dim3 grid((unsigned)(n.rows < 4096 ? n.rows : 4096));
        if (n.bf16)
            norm_long_kernel<true><<<grid, 1024, 0, s>>>(n);
        else
            norm_long_kernel<false><<<grid, 1024, 0, s>>>(n);
        return;
    }
    auto f = [&](auto w) {
        constexpr int TS = decltype(w)::TS, NIT = decltype(w)::NIT, THREADS = decltype(w)::THREADS;
        const int64_t teams = THREADS / TS, blocks = (n.rows + teams - 1) / teams;
        const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
        if (n.bf16)
            norm_kernel<true, TS, NIT, THREADS><<<grid, THREADS, 0, s>>>(n);
        else
            norm_kernel<false, TS, NIT, THREADS><<<grid, THREADS, 0, s>>>(n);
    };
    by_width(n.cols, f);
}

// Two rows a team at least, and at most 4096 waves in all (4 on each SIMD), or 2048
// where a lane holds two chunks and its registers leave room for half as many: all
// the waves run at once, and there are fewer partial sums to join. 8 workers x 1024 x
// 768 16.2 -> 13.8 us with 2048, 8 x 4096 x 300 22.6 -> 26.3 us.
int32_t norm_parts(int32_t workers, int64_t rows, int64_t cols) {
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

void launch_layer_norm_backward(const NormGrad &n, hipStream_t s) {
    if (n.cols > kLongRow) {
        const int64_t rows = n.workers * n.rows;
        const dim3 grid((unsigned)(rows < 4096 ? rows : 4096));
        const int blocks = (int)((n.cols + 511) / 512);
        const dim3 columns((unsigned)(n.workers * n.parts * blocks));
        if (n.bf16) {
            if (n.dx) norm_grad_long_kernel<true><<<grid, 1024, 0, s>>>(n);
            if (n.dgamma || n.dbeta) norm_grad_columns_kernel<true><<<columns, 64, 0, s>>>(n, blocks);
        } else {
            if (n.dx) norm_grad_long_kernel<false><<<grid, 1024, 0, s>>>(n);
            if (n.dgamma || n.dbeta) norm_grad_columns_kernel<false><<<columns, 64, 0, s>>>(n, blocks);
        }
        return;
    }
    auto f = [&](auto w) {
        constexpr int TS = decltype(w)::TS, NIT = decltype(w)::NIT, THREADS = decltype(w)::THREADS;
        const dim3 grid((unsigned)(n.workers * n.parts));
        if (n.bf16)
            norm_grad_kernel<true, TS, NIT, THREADS><<<grid, THREADS, 0, s>>>(n);
        else
            norm_grad_kernel<false, TS, NIT, THREADS><<<grid, THREADS, 0, s>>>(n);
    };
    by_width(n.cols, f);
}

void launch_layer_norm_sums(const NormGrad &n, hipStream_t s) {
    const int blocks = (int)((n.cols + kWave - 1) / kWave);
    const dim3 grid((unsigned)(n.workers * 2 * blocks));
    if (n.grad_bf16)
        norm_sums_kernel<true><<<grid, 512, 0, s>>>(n, blocks);
    else
        norm_sums_kernel<false><<<grid, 512, 0, s>>>(n, blocks);
}

}  // namespace sm
