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
//
// 8 workers x 4096 tokens, 32000 x 768, F32 from BF16: 153 us, of which 119 us are
// what the stack's zeros alone take to store; 3 x 1501 tokens, 5003 x 515: 20.5 us,
// three launches that wait for one another.
#include "grad_internal.h"

namespace sm {
namespace {

constexpr int kWave = 64;
static_assert(kSortChunk == 4 * 1024, "sorted by 1024 threads, 4 keys each");

// The id of token t, or vocab where it lies outside [0, vocab).
__device__ __forceinline__ uint32_t token_id(const void *ids, bool id64, int64_t t, uint32_t vocab) {
    if (id64) {
        const int64_t v = static_cast<const int64_t *>(ids)[t];
        return v >= 0 && v < (int64_t)vocab ? (uint32_t)v : vocab;
    }
    const int32_t v = static_cast<const int32_t *>(ids)[t];
    return v >= 0 && v < (int64_t)vocab ? (uint32_t)v : vocab;
}

// A lane's N columns of a row begin at c, or further back where they would pass the
// row's end: a value that two lanes of a wave compute is the same in both. Those in
// [from, n) are stored: none behind the end, fewer than N where the row is shorter
// than that, and none below the wave's first column, which is another wave's (adding
// to what is there, the two would each add).
struct Columns {
    int c, from, n;
};
template <int N>
__device__ __forceinline__ Columns columns(int64_t c, int64_t cols, int64_t first) {
    const int64_t at = c + N <= cols ? c : cols < N ? 0 : cols - N;
    return {(int)at, (int)(first > at ? first - at : 0), (int)(c >= cols ? 0 : cols < N ? cols : N)};
}
template <bool BF16, int N>
__device__ __forceinline__ void store_columns(void *p, int64_t row, Columns at, const float (&v)[N]) {
    if (at.from == 0 && at.n == N) {
        store_n<BF16>(p, row + at.c, N, v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j >= at.from && j < at.n) store1<BF16>(p, row + at.c + j, v[j]);
    }
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
        const Columns at = columns<8>(c, e.cols, 0);
        float v[8];
        unpack(load_raw<TB, 8>(e.table, there ? (int64_t)id * e.cols : 0, at.c, (int)e.cols), at.c, (int)e.cols, v, true);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = there ? v[j] * e.scale : 0.0f;
        store_columns<YB>(e.y, t * e.cols, at, v);
    }
}

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;

// Keys id << 32 | token of one chunk of up to 1024 R, sorted by `passes` digits
// of `width` bits (at most 8). Wave w holds places 64 R w .. of the current
// order, 64 a round, so that a key's rank among its digit is: those of earlier
// waves + those of earlier rounds of its wave + those of lower lanes of its
// round. Latency counts here (a workgroup for each worker's 4096 tokens), so a
// digit's counts of the sixteen waves are read at once and added in registers.
// Workgroups behind the sorting ones write zeros to each worker's rows from
// `beside` on, before embed_sums_kernel writes those of them that have tokens: the
// sort keeps few compute units busy, and memory not at all. 8 workers x 4096
// tokens, 32000 x 768, F32: 165 us without, 162 us with 48 MB of zeros here, 156 us
// with 96 MB, 157 to 158 us with more, up to all of them. Rows that have a token are
// then written twice; where each of them has one, the searches that are saved cost
// more: 32768 tokens, each of 32768 x 768 once, 58 us against 64 without; 8 workers x
// 4096 of 4096 43 against 48; 8 x 16384 of 20000 198 against 212.
constexpr int kZeroPiece = 32768;  // bytes of a workgroup
constexpr int64_t kZeroBeside = (int64_t)96 << 20;  // bytes of all of them

template <int R>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(EmbedGrad e, int chunks, int passes, int width,
                                                                 int64_t beside, int pieces) {
    __shared__ uint64_t keys[kSortThreads * R];
    __shared__ uint32_t count[kSortWaves][256];
    __shared__ uint32_t wave_total[4];
    const int sorting = e.workers * chunks;
    if ((int)blockIdx.x >= sorting) {
        const int b = xcd_run(blockIdx.x - sorting, gridDim.x - sorting);
        const int64_t size = e.grad_bf16 ? 2 : 4, from = (int64_t)(b % pieces) * kZeroPiece;
        const int64_t left = (e.vocab - beside) * e.cols * size - from;
        char *p = static_cast<char *>(e.grad) + ((b / pieces + 1) * e.vocab * e.cols * size - left);
        const int bytes = (int)(left < kZeroPiece ? left : kZeroPiece);
#pragma unroll
        for (int i = threadIdx.x * 16; i < kZeroPiece; i += kSortThreads * 16) {
            if (i + 16 <= bytes)
                *reinterpret_cast<u32x4_any *>(p + i) = u32x4{0, 0, 0, 0};
            else
                for (int j = i; j < bytes; j += 2) *reinterpret_cast<uint16_t *>(p + j) = 0;
        }
        return;
    }
    const int worker = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int64_t first = (int64_t)chunk * kSortChunk;
    const int n = (int)(e.tokens - first < kSortChunk ? e.tokens - first : kSortChunk);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int place = wave * (kWave * R) + lane;
    const uint32_t mask = (1u << width) - 1;

    uint64_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = place + r * kWave;
        // places past the chunk: behind every token, as their place is
        const uint32_t id =
            i < n ? token_id(e.ids, e.id64, worker * e.tokens + first + i, (uint32_t)e.vocab) : (uint32_t)e.vocab;
        key[r] = (uint64_t)id << 32 | (uint32_t)(first + i);
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = 32 + p * width;
        for (int i = threadIdx.x; i < kSortWaves * 256; i += kSortThreads) (&count[0][0])[i] = 0;
        __syncthreads();
        uint32_t rank[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t digit = (uint32_t)(key[r] >> shift) & mask;
            uint64_t same = ~0ull;
#pragma unroll
            for (int b = 0; b < 8; ++b) {  // bits past the width are 0 in every lane
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
        uint32_t own[kSortWaves], total = 0, inclusive = 0;
        if (threadIdx.x < 256) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) own[w] = count[w][threadIdx.x];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) total += own[w];
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
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (w < wave) base += wave_total[w];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                count[w][threadIdx.x] = base;
                base += own[w];
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) keys[count[wave][(uint32_t)(key[r] >> shift) & mask] + rank[r]] = key[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = keys[place + r * kWave];
    }
    uint64_t *out = e.keys[0] + worker * e.tokens + first;
#pragma unroll
    for (int r = 0; r < R; ++r)
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

// The same by a whole wave: 64 probes at a time, so two dependent loads for 4096
// keys where one lane's search takes twelve.
__device__ __forceinline__ int64_t wave_lower_bound(const uint64_t *keys, int64_t n, uint64_t key, int lane) {
    int64_t lo = 0, len = n;
    while (len > kWave) {
        const int64_t step = (len + kWave - 1) / kWave;  // probe i: the last key of its step
        const int64_t at = (lane + 1) * step - 1;
        const int64_t below = __popcll(__ballot(keys[lo + (at < len ? at : len - 1)] < key)) * step;
        if (below >= len) return lo + len;
        lo += below;
        len = len - below < step ? len - below : step;
    }
    return lo + __popcll(__ballot(lane < len && keys[lo + (lane < len ? lane : 0)] < key));
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
// The gradient of a row's columns from their sum; `old`: what is there, to add to.
template <bool GB, bool ADD>
__device__ __forceinline__ void write_row(const EmbedGrad &e, int64_t worker, uint32_t id, Columns at,
                                          const float (&sum)[4], const Raw<GB, 4> &old) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e.scale * sum[j];
    if constexpr (ADD) {
        float o[4];
        unpack(old, at.c, (int)e.cols, o, true);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += o[j];
    }
    store_columns<GB>(e.grad, (worker * e.vocab + id) * e.cols, at, v);
}

__device__ __forceinline__ void write_partial(const EmbedGrad &e, int64_t worker, int seg, int which, Columns at,
                                              const float (&sum)[4]) {
    store_columns<false>(e.partial, ((worker * e.segments + seg) * 2 + which) * e.cols, at, sum);
}

// Zeros in the rows of `rows` ids that no token has, by a workgroup (rows that
// follow each other are one stretch of memory). A workgroup writes about 12 KB
// and an XCD's workgroups follow each other in memory: 786 MB take 119 us so,
// 143 us in stretches of 96 KB (plain stores alone; 114 us at 4 KB, which has
// no room for the search).
constexpr int kMaxZeroRows = 32;
constexpr int64_t kZeroBytes = 12288;
template <bool GB>
__device__ void zero_rows(const EmbedGrad &e, const uint64_t *keys, int64_t worker, int64_t v0, int rows, int64_t most) {
    const int lane = threadIdx.x & (kWave - 1);
    // the ids that there are (each wave for itself): from the keys behind the
    // first of them, and again behind the last one seen where 64 keys do not
    // reach past the group
    const int64_t v1 = v0 + rows < most ? v0 + rows : most;
    uint32_t mask = ~0u >> (kMaxZeroRows - (int)(v1 - v0));
    for (int64_t v = v0; v < v1;) {
        const int64_t at = wave_lower_bound(keys, e.tokens, (uint64_t)v << 32, lane) + lane;
        const int64_t id = at < e.tokens ? (int64_t)(keys[at] >> 32) : e.vocab;
        uint32_t seen = id < v1 ? 1u << (int)(id - v0) : 0u;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) seen |= __shfl_xor(seen, d);
        mask &= ~seen;
        v = (int64_t)__shfl((unsigned long long)id, kWave - 1) + 1;
    }
    constexpr int W = GB ? 8 : 4;  // 16 bytes a lane, side by side
    const float zero[W] = {};
    while (mask) {
        const int first = __builtin_ctz(mask);
        const uint32_t rest = ~(mask >> first);
        const int count = rest ? __builtin_ctz(rest) : 32;  // rows of this stretch
        const int64_t at = (worker * e.vocab + v0 + first) * e.cols, len = count * e.cols;
        for (int64_t i = (int64_t)threadIdx.x * W; i < len; i += 256 * W)
            store_n<GB>(e.grad, at + i, (int)(len - i < W ? len - i : W), zero);
        mask = first + count >= 32 ? 0 : mask >> (first + count) << (first + count);
    }
}

constexpr int kInFlight = 16;  // rows that a wave has under way

template <bool DB, bool GB, bool ADD>
__global__ __launch_bounds__(256) void embed_sums_kernel(EmbedGrad e, const uint64_t *keys, int64_t sum_waves,
                                                         int sum_blocks, int zero_rows_each, int64_t beside) {
    const int lane = threadIdx.x & (kWave - 1);
    if ((int)blockIdx.x >= sum_blocks) {  // rows below `beside` that no token has
        const int b = xcd_run(blockIdx.x - sum_blocks, gridDim.x - sum_blocks);
        const int groups = (int)((beside + zero_rows_each - 1) / zero_rows_each);
        const int64_t worker = b / groups;
        zero_rows<GB>(e, keys + worker * e.tokens, worker, (int64_t)(b % groups) * zero_rows_each, zero_rows_each, beside);
        return;
    }
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (w >= sum_waves) return;
    const int blocks = (int)((e.cols + kEmbedCols - 1) / kEmbedCols);
    const int64_t first_col = (w % blocks) * kEmbedCols;
    const Columns own = columns<4>(first_col + lane * 4, e.cols, first_col);
    const int seg = (int)(w / blocks % e.segments);
    const int64_t worker = w / blocks / e.segments;
    keys += worker * e.tokens;
    const int64_t begin = (int64_t)seg * e.seg;
    const int64_t end = begin + e.seg < e.tokens ? begin + e.seg : e.tokens;
    const uint32_t none = (uint32_t)e.vocab;  // padding: sorted behind every row
    const uint32_t before = begin > 0 ? (uint32_t)(keys[begin - 1] >> 32) : none;
    const int64_t base = worker * e.tokens;
    uint32_t cur = none;  // a row that goes on
    bool first = true;    // none has ended in this segment
    float sum[4] = {};
    for (int64_t g = begin; g < end; g += kWave) {
        const int have = (int)(end - g < kWave ? end - g : kWave);
        const uint64_t key = lane < have ? keys[g + lane] : (uint64_t)none << 32;
        const uint32_t key_id = (uint32_t)(key >> 32), key_at = (uint32_t)key;
        // the next token's id: a row ends where it differs
        const uint32_t key_next = lane < have && g + lane + 1 < e.tokens ? (uint32_t)(keys[g + lane + 1] >> 32) : none;
        for (int i0 = 0; i0 < have; i0 += kInFlight) {
            Raw<DB, 4> v[kInFlight];
            Raw<GB, 4> old[ADD ? kInFlight : 1];
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const uint32_t id = __builtin_amdgcn_readlane(key_id, i0 + i);
                const uint32_t t = id == none ? 0 : __builtin_amdgcn_readlane(key_at, i0 + i);
                v[i] = load_raw<DB, 4>(e.dy, (base + t) * e.cols, own.c, (int)e.cols);
                if constexpr (ADD)
                    old[i] = load_raw<GB, 4>(e.grad, (worker * e.vocab + (id == none ? 0 : id)) * e.cols, own.c, (int)e.cols);
            }
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const uint32_t id = __builtin_amdgcn_readlane(key_id, i0 + i);
                if (id == none) continue;
                float x[4];
                unpack(v[i], own.c, (int)e.cols, x, true);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] += x[j];
                cur = id;
                if (id != __builtin_amdgcn_readlane(key_next, i0 + i)) {
                    if (first && id == before)
                        write_partial(e, worker, seg, 0, own, sum);
                    else
                        write_row<GB, ADD>(e, worker, id, own, sum, old[ADD ? i : 0]);
                    first = false;
                    cur = none;
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = 0.0f;
                }
            }
        }
    }
    if (cur != none) write_partial(e, worker, seg, first && cur == before ? 0 : 1, own, sum);
}

constexpr int kJoined = 8;  // partial sums that a wave has under way

// A row that begins in segment `seg` and goes on in the next ones: its last
// partial there, then the first partials of the segments that it reaches.
template <bool GB, bool ADD>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedGrad e, const uint64_t *keys, int64_t waves) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (w >= waves) return;
    const int blocks = (int)((e.cols + kEmbedCols - 1) / kEmbedCols);
    const int64_t first_col = (w % blocks) * kEmbedCols;
    const Columns own = columns<4>(first_col + lane * 4, e.cols, first_col);
    const int seg = (int)(w / blocks % (e.segments - 1));
    const int64_t worker = w / blocks / (e.segments - 1);
    keys += worker * e.tokens;
    const int64_t begin = (int64_t)seg * e.seg, end = begin + e.seg;  // end < tokens: not the last segment
    // the row of the last token here, and of the first token of the segment i + lane
    const uint32_t none = (uint32_t)e.vocab, id = (uint32_t)(keys[end - 1] >> 32);
    auto first_of = [&](int i) {
        const int64_t at = (int64_t)(i + lane) * e.seg;
        return at < e.tokens ? (uint32_t)(keys[at] >> 32) : none;
    };
    const uint32_t before = begin > 0 ? (uint32_t)(keys[begin - 1] >> 32) : none;
    uint64_t reached = __ballot(first_of(seg + 1) == id);
    // one that began in an earlier segment is joined there
    if (id == none || !(reached & 1) || before == id) return;
    int last = seg;  // the last segment that it reaches
    while (reached == ~0ull) {
        last += kWave;
        reached = __ballot(first_of(last + 1) == id);
    }
    last += __builtin_ctzll(~reached);
    Raw<GB, 4> old;
    if constexpr (ADD) old = load_raw<GB, 4>(e.grad, (worker * e.vocab + id) * e.cols, own.c, (int)e.cols);
    const int64_t at = (worker * e.segments + seg) * 2 * e.cols;
    float sum[4];
    unpack(load_raw<false, 4>(e.partial, at + e.cols, own.c, (int)e.cols), own.c, (int)e.cols, sum, true);
    for (int i = 1; i <= last - seg; i += kJoined) {
        Raw<false, 4> v[kJoined];
#pragma unroll
        for (int k = 0; k < kJoined; ++k)
            v[k] = load_raw<false, 4>(e.partial, at + (int64_t)(i + k <= last - seg ? i + k : i) * 2 * e.cols, own.c, (int)e.cols);
#pragma unroll
        for (int k = 0; k < kJoined; ++k) {
            float x[4];
            unpack(v[k], own.c, (int)e.cols, x, true);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += i + k <= last - seg ? x[j] : 0.0f;
        }
    }
    write_row<GB, ADD>(e, worker, id, own, sum, old);
}

// The first of the rows that get their zeros beside the sort.
int64_t first_beside(const EmbedGrad &e) {
    const int64_t rows = kZeroBeside / (e.workers * e.cols * (e.grad_bf16 ? 2 : 4));
    return e.accumulate || rows <= 0 ? e.vocab : rows < e.vocab ? e.vocab - rows : 0;
}

template <bool DB, bool GB>
void launch_sums(const EmbedGrad &e, const uint64_t *keys, int64_t waves, hipStream_t s) {
    const int blocks = (int)((waves + 31) / 32 * 8);  // a multiple of the XCDs
    const int64_t bytes = e.cols * (GB ? 2 : 4);
    // (and few enough workgroups that a launch's threads stay below 2^32)
    int64_t rows = kZeroBytes / bytes, least = (e.workers * e.vocab + (1 << 23) - 1) >> 23;
    rows = rows < least ? least : rows;
    rows = rows < 1 ? 1 : rows > kMaxZeroRows ? kMaxZeroRows : rows;
    const int64_t beside = first_beside(e), zeros = e.accumulate ? 0 : e.workers * ((beside + rows - 1) / rows);
    const dim3 grid((unsigned)(blocks + zeros));
    if (e.accumulate)
        embed_sums_kernel<DB, GB, true><<<grid, 256, 0, s>>>(e, keys, waves, blocks, (int)rows, beside);
    else
        embed_sums_kernel<DB, GB, false><<<grid, 256, 0, s>>>(e, keys, waves, blocks, (int)rows, beside);
}

template <bool GB>
void launch_join(const EmbedGrad &e, const uint64_t *keys, int64_t waves, hipStream_t s) {
    const dim3 grid((unsigned)((waves + 3) / 4));
    if (e.accumulate)
        embed_join_kernel<GB, true><<<grid, 256, 0, s>>>(e, keys, waves);
    else
        embed_join_kernel<GB, false><<<grid, 256, 0, s>>>(e, keys, waves);
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

// At least 16 tokens a segment (all under way at once), and more where that gives over 16384 waves.
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
    const int passes = (bits + 7) / 8, width = (bits + passes - 1) / passes;
    const int64_t beside = first_beside(e), bytes = (e.vocab - beside) * e.cols * (e.grad_bf16 ? 2 : 4);
    const int pieces = (int)((bytes + kZeroPiece - 1) / kZeroPiece);
    const dim3 grid((unsigned)(e.workers * (chunks + pieces)));
    if (e.tokens <= kSortThreads)
        embed_sort_kernel<1><<<grid, kSortThreads, 0, s>>>(e, chunks, passes, width, beside, pieces);
    else if (e.tokens <= 2 * kSortThreads)
        embed_sort_kernel<2><<<grid, kSortThreads, 0, s>>>(e, chunks, passes, width, beside, pieces);
    else
        embed_sort_kernel<4><<<grid, kSortThreads, 0, s>>>(e, chunks, passes, width, beside, pieces);
}

void launch_embedding_merge(const EmbedGrad &e, int pass, hipStream_t s) {
    const int blocks = (int)((e.tokens + 255) / 256);
    embed_merge_kernel<<<dim3((unsigned)(e.workers * blocks)), 256, 0, s>>>(
        e.keys[pass & 1], e.keys[(pass + 1) & 1], e.tokens, (int64_t)kSortChunk << pass, blocks);
}

void launch_embedding_sums(const EmbedGrad &e, hipStream_t s) {
    const uint64_t *keys = e.keys[embed_merge_passes(e.tokens) & 1];
    const int64_t waves = sum_waves(e);
    if (e.dy_bf16)
        e.grad_bf16 ? launch_sums<true, true>(e, keys, waves, s) : launch_sums<true, false>(e, keys, waves, s);
    else
        e.grad_bf16 ? launch_sums<false, true>(e, keys, waves, s) : launch_sums<false, false>(e, keys, waves, s);
}

void launch_embedding_join(const EmbedGrad &e, hipStream_t s) {
    const uint64_t *keys = e.keys[embed_merge_passes(e.tokens) & 1];
    const int64_t waves = sum_waves(e) / e.segments * (e.segments - 1);
    if (e.grad_bf16)
        launch_join<true>(e, keys, waves, s);
    else
        launch_join<false>(e, keys, waves, s);
}

}  // namespace sm
