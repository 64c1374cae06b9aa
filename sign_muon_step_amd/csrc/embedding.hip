// embedding.hip -- embedding lookup with scaling and its gradient by sorted
// tokens.
//
// The lookup is y[t] = s W[id_t]: a copy of rows, bound by the bytes read and
// written.
//
// The gradient of worker m's table is dW_m[v] = s * sum of dy[t] over the
// tokens with id_t = v. It is bound by the stack [Mw][V][C] that the step
// reads: most rows of it are zeros. The tokens of each worker are sorted by id
// (stable), so that a row's terms are neighbours and are added in one order on
// every run, whatever the hardware does first:
//   embed_sort_kernel   chunks of 4096 tokens, each sorted by one workgroup in
//                       LDS (radix, 8 bits a pass, ranks from wave ballots)
//   embed_merge_kernel  pairs of sorted runs, each token's place from a search
//                       in the other run (only where there are several chunks)
//   embed_sums_kernel   segments of the sorted tokens, one wave for each
//                       segment and 256 columns: a row whose tokens all lie in
//                       the segment is written, the first and the last are left
//                       as partial sums where they go on in a neighbour. So the
//                       work is even whatever the ids are (one id in every
//                       place, or none twice). Further waves write the rows
//                       that no token has.
//   embed_join_kernel   adds the partial sums of each row, in their order
#include "grad_internal.h"

namespace sm {
namespace {

constexpr int kWave = 64;

// The id of token t, or vocab where it lies outside [0, vocab).
__device__ __forceinline__ uint32_t token_id(const void *ids, bool id64, int64_t t, uint32_t vocab) {
    if (id64) {
        const int64_t v = static_cast<const int64_t *>(ids)[t];
        return v >= 0 && v < (int64_t)vocab ? (uint32_t)v : vocab;
    }
    const int32_t v = static_cast<const int32_t *>(ids)[t];
    return v >= 0 && v < (int64_t)vocab ? (uint32_t)v : vocab;
}

// 2^lg lanes take one row, 8 columns each at a time.
template <bool TB, bool YB>
__global__ __launch_bounds__(256) void embed_kernel(Embed e, int lg) {
    const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
    if (t >= e.tokens) return;
    const int64_t step = (int64_t)8 << lg;
    const uint32_t id = token_id(e.ids, e.id64, t, (uint32_t)e.vocab);
    const bool there = id < (uint32_t)e.vocab;
    for (int64_t c = (int64_t)(threadIdx.x & ((1 << lg) - 1)) * 8; c < e.cols; c += step) {
        const int n = (int)(e.cols - c < 8 ? e.cols - c : 8);
        float v[8] = {};
        if (there) {
            load_n<TB>(e.table, (int64_t)id * e.cols + c, n, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= e.scale;
        }
        store_n<YB>(e.y, t * e.cols + c, n, v);
    }
}

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortRounds = kSortChunk / kSortThreads;  // keys a thread

// Keys id << 32 | token of one chunk, sorted. Wave w holds places 256 w ..
// 256 w + 255 of the current order, 64 a round, so that a key's rank among its
// digit is: those of earlier waves + those of earlier rounds of its wave +
// those of lower lanes of its round.
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(EmbedGrad e, int chunks, int bits) {
    __shared__ uint64_t keys[kSortChunk];
    __shared__ uint32_t count[kSortWaves][256];
    __shared__ uint32_t wave_total[4];
    const int worker = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int64_t first = (int64_t)chunk * kSortChunk;
    const int n = (int)(e.tokens - first < kSortChunk ? e.tokens - first : kSortChunk);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int place = wave * (kWave * kSortRounds) + lane;

    uint64_t key[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int i = place + r * kWave;
        // places past the chunk: behind every token, as their place is
        const uint32_t id =
            i < n ? token_id(e.ids, e.id64, worker * e.tokens + first + i, (uint32_t)e.vocab) : (uint32_t)e.vocab;
        key[r] = (uint64_t)id << 32 | (uint32_t)(first + i);
    }
    for (int shift = 32; shift < 32 + bits; shift += 8) {
        for (int i = threadIdx.x; i < kSortWaves * 256; i += kSortThreads) (&count[0][0])[i] = 0;
        __syncthreads();
        uint32_t rank[kSortRounds];
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            const uint32_t digit = (uint32_t)(key[r] >> shift) & 255u;
            uint64_t same = ~0ull;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const bool bit = (digit >> b) & 1u;
                const uint64_t m = __ballot(bit);
                same &= bit ? m : ~m;
            }
            const uint32_t before = __popcll(same & ((1ull << lane) - 1));
            // the wave's count of this digit so far: read by every lane, then
            // raised by the first lane of each digit (LDS accesses of a wave
            // are carried out in their order)
            volatile uint32_t *c = &count[wave][digit];
            const uint32_t had = *c;
            __builtin_amdgcn_wave_barrier();
            if (before == 0) *c = had + __popcll(same);
            __builtin_amdgcn_wave_barrier();
            rank[r] = had + before;
        }
        __syncthreads();
        // exclusive sums over digits, then waves
        uint32_t total = 0, inclusive = 0;
        if (threadIdx.x < 256) {
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = count[w][threadIdx.x];
                count[w][threadIdx.x] = total;
                total += c;
            }
            inclusive = total;
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) {
                const uint32_t up = __shfl_up(inclusive, d);
                if (lane >= d) inclusive += up;
            }
            if (lane == kWave - 1) wave_total[wave] = inclusive;
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t base = inclusive - total;
            for (int w = 0; w < wave; ++w) base += wave_total[w];
            for (int w = 0; w < kSortWaves; ++w) count[w][threadIdx.x] += base;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            keys[count[wave][(uint32_t)(key[r] >> shift) & 255u] + rank[r]] = key[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) key[r] = keys[place + r * kWave];
    }
    uint64_t *out = e.keys[0] + worker * e.tokens + first;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r)
        if (place + r * kWave < n) out[place + r * kWave] = key[r];
}

// First place in [0, n) whose key is not below `key`.
__device__ __forceinline__ int64_t lower_bound(const uint64_t *keys, int64_t n, uint64_t key) {
    int64_t lo = 0, len = n;
    while (len > 0) {
        const int64_t half = len >> 1;
        if (keys[lo + half] < key) {
            lo += half + 1;
            len -= half + 1;
        } else {
            len = half;
        }
    }
    return lo;
}

// Runs of `run` sorted keys into runs of 2 * run. Keys differ (a token is in
// one key), so a key's place is its place in its run plus the number of lower
// keys in the other.
__global__ __launch_bounds__(256) void embed_merge_kernel(const uint64_t *from, uint64_t *to, int64_t tokens,
                                                          int64_t run, int blocks) {
    const int worker = blockIdx.x / blocks;
    const int64_t i = (int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x;
    if (i >= tokens) return;
    from += worker * tokens;
    to += worker * tokens;
    const int64_t mine = i / run, pair = (mine & ~(int64_t)1) * run;
    const int64_t other = (mine ^ 1) * run;
    const uint64_t key = from[i];
    int64_t lower = 0;
    if (other < tokens) lower = lower_bound(from + other, tokens - other < run ? tokens - other : run, key);
    to[pair + (i - mine * run) + lower] = key;
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------
template <bool GB>
__device__ __forceinline__ void write_row(const EmbedGrad &e, int64_t worker, uint32_t id, int64_t c, int n,
                                          const float (&sum)[4]) {
    float v[4];
    const int64_t at = (worker * e.vocab + id) * e.cols + c;
    if (n <= 0) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e.scale * sum[j];
    if (e.accumulate) {
        float old[4];
        load_n<GB>(e.grad, at, n, old);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += old[j];
    }
    store_n<GB>(e.grad, at, n, v);
}

__device__ __forceinline__ void write_partial(const EmbedGrad &e, int64_t worker, int seg, int which, int64_t c,
                                              int n, const float (&sum)[4]) {
    if (n > 0) store_n<false>(e.partial, ((worker * e.segments + seg) * 2 + which) * e.cols + c, n, sum);
}

// Zeros in the rows of 64 ids that no token has. Rows that follow each other
// are one stretch of memory.
template <bool GB>
__device__ void zero_rows(const EmbedGrad &e, const uint64_t *keys, int64_t worker, int64_t v0, int lane) {
    const int64_t v = v0 + lane;
    bool empty = false;
    if (v < e.vocab) {
        const int64_t at = lower_bound(keys, e.tokens, (uint64_t)v << 32);
        empty = at >= e.tokens || (int64_t)(keys[at] >> 32) != v;
    }
    uint64_t mask = __ballot(empty);
    const float zero[8] = {};
    while (mask) {
        const int first = __builtin_ctzll(mask);
        const uint64_t rest = ~(mask >> first);
        const int count = rest ? __builtin_ctzll(rest) : kWave - first;  // rows of this stretch
        const int64_t at = (worker * e.vocab + v0 + first) * e.cols, len = count * e.cols;
        for (int64_t i = (int64_t)lane * 8; i < len; i += kWave * 8)
            store_n<GB>(e.grad, at + i, (int)(len - i < 8 ? len - i : 8), zero);
        mask = first + count >= kWave ? 0 : mask >> (first + count) << (first + count);
    }
}

template <bool DB, bool GB>
__global__ __launch_bounds__(256) void embed_sums_kernel(EmbedGrad e, const uint64_t *keys, int64_t sum_waves,
                                                         int64_t waves) {
    const int lane = threadIdx.x & (kWave - 1);
    int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (w >= waves) return;
    if (w >= sum_waves) {  // rows that no token has
        w -= sum_waves;
        const int64_t groups = (e.vocab + kWave - 1) / kWave;
        const int64_t worker = w / groups;
        zero_rows<GB>(e, keys + worker * e.tokens, worker, (w % groups) * kWave, lane);
        return;
    }
    const int blocks = (int)((e.cols + kEmbedCols - 1) / kEmbedCols);
    const int64_t c = (w % blocks) * kEmbedCols + lane * 4;
    const int seg = (int)(w / blocks % e.segments);
    const int64_t worker = w / blocks / e.segments;
    const int n = (int)(e.cols - c < 4 ? e.cols - c : 4);  // columns of this lane (below 1: none)
    keys += worker * e.tokens;
    const int64_t begin = (int64_t)seg * e.seg;
    const int64_t end = begin + e.seg < e.tokens ? begin + e.seg : e.tokens;
    const uint32_t before = begin > 0 ? (uint32_t)(keys[begin - 1] >> 32) : (uint32_t)e.vocab;
    const uint32_t after = end < e.tokens ? (uint32_t)(keys[end] >> 32) : (uint32_t)e.vocab;
    uint32_t cur = (uint32_t)e.vocab;  // the row being summed
    bool first = true;                 // cur is the segment's first row
    float sum[4] = {};
    const int64_t base = worker * e.tokens;
    for (int64_t g = begin; g < end; g += kWave) {
        const int have = (int)(end - g < kWave ? end - g : kWave);
        const uint64_t key = lane < have ? keys[g + lane] : (uint64_t)e.vocab << 32;
        const uint32_t key_id = (uint32_t)(key >> 32), key_at = (uint32_t)key;
        for (int i0 = 0; i0 < have; i0 += 8) {
            float v[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // eight rows in flight
                const uint32_t t = __builtin_amdgcn_readlane(key_at, i0 + i);
                const bool there = i0 + i < have && __builtin_amdgcn_readlane(key_id, i0 + i) < (uint32_t)e.vocab;
                load_n<DB>(e.dy, (base + (there ? t : 0)) * e.cols + c, there ? n : 0, v[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t id = i0 + i < have ? __builtin_amdgcn_readlane(key_id, i0 + i) : (uint32_t)e.vocab;
                if (id == (uint32_t)e.vocab) continue;  // padding is sorted behind every row
                if (id != cur) {
                    if (cur != (uint32_t)e.vocab) {
                        if (first && cur == before)
                            write_partial(e, worker, seg, 0, c, n, sum);
                        else
                            write_row<GB>(e, worker, cur, c, n, sum);
                        first = false;
                    }
                    cur = id;
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] += v[i][j];
            }
        }
    }
    if (cur == (uint32_t)e.vocab) return;
    if (first && cur == before)
        write_partial(e, worker, seg, 0, c, n, sum);
    else if (cur == after)
        write_partial(e, worker, seg, 1, c, n, sum);
    else
        write_row<GB>(e, worker, cur, c, n, sum);
}

// A row that begins in segment `seg` and goes on in the next ones: its last
// partial there, then the first partials of the segments that it reaches.
template <bool GB>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedGrad e, const uint64_t *keys, int64_t waves) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (w >= waves) return;
    const int blocks = (int)((e.cols + kEmbedCols - 1) / kEmbedCols);
    const int64_t c = (w % blocks) * kEmbedCols + lane * 4;
    const int seg = (int)(w / blocks % (e.segments - 1));
    const int64_t worker = w / blocks / (e.segments - 1);
    keys += worker * e.tokens;
    const int64_t begin = (int64_t)seg * e.seg, end = begin + e.seg;  // end < tokens: not the last segment
    const uint32_t id = (uint32_t)(keys[end - 1] >> 32);
    if (id == (uint32_t)e.vocab || (uint32_t)(keys[end] >> 32) != id) return;
    // one that began in an earlier segment is joined there
    if (begin > 0 && (uint32_t)(keys[begin - 1] >> 32) == id) return;
    const int n = (int)(e.cols - c < 4 ? e.cols - c : 4);
    if (n <= 0) return;
    // the last token of the row, and its segment
    const int64_t stop = end + lower_bound(keys + end, e.tokens - end, (uint64_t)(id + 1) << 32);
    const int last = (int)((stop - 1) / e.seg);
    const int64_t at = (worker * e.segments + seg) * 2 * e.cols + c;
    float sum[4];
    load_n<false>(e.partial, at + e.cols, n, sum);
    for (int i = 1; i <= last - seg; i += 4) {
        float v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            load_n<false>(e.partial, at + (int64_t)(i + k <= last - seg ? i + k : i) * 2 * e.cols,
                          i + k <= last - seg ? n : 0, v[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += v[k][j];
    }
    write_row<GB>(e, worker, id, c, n, sum);
}

int64_t sum_waves(const EmbedGrad &e) {
    return (int64_t)e.workers * e.segments * ((e.cols + kEmbedCols - 1) / kEmbedCols);
}

}  // namespace

void launch_embedding(const Embed &e, hipStream_t s) {
    int lg = 0;  // lanes of a row: enough for its columns, at most a wave
    while (lg < 6 && ((int64_t)8 << lg) < e.cols) ++lg;
    const int64_t rows = 256 >> lg;
    const dim3 grid((unsigned)((e.tokens + rows - 1) / rows));
    if (e.table_bf16) {
        if (e.y_bf16)
            embed_kernel<true, true><<<grid, 256, 0, s>>>(e, lg);
        else
            embed_kernel<true, false><<<grid, 256, 0, s>>>(e, lg);
    } else {
        if (e.y_bf16)
            embed_kernel<false, true><<<grid, 256, 0, s>>>(e, lg);
        else
            embed_kernel<false, false><<<grid, 256, 0, s>>>(e, lg);
    }
}

int embed_merge_passes(int64_t tokens) {
    int passes = 0;
    for (int64_t run = kSortChunk; run < tokens; run *= 2) ++passes;
    return passes;
}

// At least 16 tokens a segment, and more where that gives over 16384 waves.
int32_t embed_segment(int32_t workers, int64_t tokens, int64_t cols) {
    const int64_t blocks = (cols + kEmbedCols - 1) / kEmbedCols;
    int64_t seg = 16;
    while (seg < tokens && workers * ((tokens + seg - 1) / seg) * blocks > 16384) seg *= 2;
    return (int32_t)seg;
}

void launch_embedding_sort(const EmbedGrad &e, hipStream_t s) {
    const int chunks = (int)((e.tokens + kSortChunk - 1) / kSortChunk);
    int bits = 0;  // of the largest key, vocab (padding)
    while (bits < 32 && (e.vocab >> bits) != 0) ++bits;
    embed_sort_kernel<<<dim3((unsigned)(e.workers * chunks)), kSortThreads, 0, s>>>(e, chunks, bits);
}

void launch_embedding_merge(const EmbedGrad &e, int pass, hipStream_t s) {
    const int blocks = (int)((e.tokens + 255) / 256);
    embed_merge_kernel<<<dim3((unsigned)(e.workers * blocks)), 256, 0, s>>>(
        e.keys[pass & 1], e.keys[(pass + 1) & 1], e.tokens, (int64_t)kSortChunk << pass, blocks);
}

void launch_embedding_sums(const EmbedGrad &e, hipStream_t s) {
    const uint64_t *keys = e.keys[embed_merge_passes(e.tokens) & 1];
    const int64_t sums = sum_waves(e);
    const int64_t waves = sums + (e.accumulate ? 0 : e.workers * ((e.vocab + kWave - 1) / kWave));
    const dim3 grid((unsigned)((waves + 3) / 4));
    if (e.dy_bf16) {
        if (e.grad_bf16)
            embed_sums_kernel<true, true><<<grid, 256, 0, s>>>(e, keys, sums, waves);
        else
            embed_sums_kernel<true, false><<<grid, 256, 0, s>>>(e, keys, sums, waves);
    } else {
        if (e.grad_bf16)
            embed_sums_kernel<false, true><<<grid, 256, 0, s>>>(e, keys, sums, waves);
        else
            embed_sums_kernel<false, false><<<grid, 256, 0, s>>>(e, keys, sums, waves);
    }
}

void launch_embedding_join(const EmbedGrad &e, hipStream_t s) {
    const uint64_t *keys = e.keys[embed_merge_passes(e.tokens) & 1];
    const int64_t waves = sum_waves(e) / e.segments * (e.segments - 1);
    const dim3 grid((unsigned)((waves + 3) / 4));
    if (e.grad_bf16)
        embed_join_kernel<true><<<grid, 256, 0, s>>>(e, keys, waves);
    else
        embed_join_kernel<false><<<grid, 256, 0, s>>>(e, keys, waves);
}

}  // namespace sm
