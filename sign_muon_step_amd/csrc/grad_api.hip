// grad_api.hip -- host side of the gradient operators declared in
// include/signmuon.h: argument checks, workspace layout and launches.
#include <cmath>

#include "signmuon.h"
#include "grad_internal.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 20;      // vocab and cols, as a matrix's rows and cols
constexpr int64_t kMaxN = ((int64_t)1 << 31) - 1;  // entries of one weight, as in the step
constexpr int32_t kMaxWorkers = 255;
constexpr int64_t kMaxTokens = (int64_t)1 << 25;   // over all workers: a launch's threads stay below 2^32
constexpr size_t kSectionAlign = 256;

inline size_t align_up(size_t x) { return (x + kSectionAlign - 1) / kSectionAlign * kSectionAlign; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool dtype_ok(int d) { return d == SIGNMUON_F32 || d == SIGNMUON_BF16; }

template <typename... P>
bool all_aligned(const P *...p) { return (aligned16(p) && ...); }

int check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SIGNMUON_OK;
    if (!ws || have < need) return SIGNMUON_EWORKSPACE;
    return aligned16(ws) ? SIGNMUON_OK : SIGNMUON_EALIGN;
}

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------
int check_embedding(int64_t workers, int64_t tokens, int64_t vocab, int64_t cols) {
    if (workers < 1 || tokens < 1 || vocab < 1 || cols < 1) return SIGNMUON_EINVAL;
    if (workers > kMaxWorkers || tokens > kMaxTokens / workers) return SIGNMUON_ERANGE;
    if (vocab > kMaxDim || cols > kMaxDim || vocab * cols > kMaxN) return SIGNMUON_ERANGE;
    return SIGNMUON_OK;
}

struct EmbedPlan {
    int32_t seg, segments;
    size_t keys[2], partial, total;
};

EmbedPlan embedding_plan(int64_t workers, int64_t tokens, int64_t cols) {
    EmbedPlan p;
    p.seg = sm::embed_segment((int32_t)workers, tokens, cols);
    p.segments = (int32_t)((tokens + p.seg - 1) / p.seg);
    const size_t keys = align_up((size_t)(workers * tokens) * sizeof(uint64_t));
    p.keys[0] = 0;
    p.keys[1] = keys;
    p.partial = sm::embed_merge_passes(tokens) > 0 ? 2 * keys : keys;
    // one segment shares no row with another
    p.total = p.partial + (p.segments > 1 ? (size_t)(workers * p.segments * 2 * cols) * sizeof(float) : 0);
    return p;
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
int check_norm(int64_t workers, int64_t rows, int64_t cols) {
    if (workers < 1 || rows < 1 || cols < 1) return SIGNMUON_EINVAL;
    if (workers > kMaxWorkers || rows > kMaxTokens / workers || cols > kMaxDim) return SIGNMUON_ERANGE;
    return SIGNMUON_OK;
}

size_t norm_workspace(int32_t workers, int64_t rows, int64_t cols) {
    const int32_t parts = sm::norm_parts(workers, rows, cols);
    return parts > 1 ? (size_t)((int64_t)workers * parts * 2 * cols) * sizeof(float) : 0;
}

// ---------------------------------------------------------------------------
// Root-mean-square norm: check_norm, and
// ---------------------------------------------------------------------------
size_t rms_workspace(int32_t workers, int64_t rows, int64_t cols) {
    const int32_t parts = sm::rms_parts(workers, rows, cols);
    return parts > 1 ? (size_t)((int64_t)workers * parts * cols) * sizeof(float) : 0;
}

// ---------------------------------------------------------------------------
// Gradient norms and clipping
// ---------------------------------------------------------------------------
struct ClipPlan {
    int32_t unit;   // entries
    int64_t units;  // of a worker
    size_t factors, total;
};

inline int64_t clip_units(int64_t n, int32_t unit) { return (n + unit - 1) / unit; }

// The sizes alone, then what a call reads and writes.
int check_gradients(const signmuon_gradient *grads, int32_t n_grads, int32_t workers, ClipPlan &p) {
    if (!grads || n_grads < 1 || workers < 1) return SIGNMUON_EINVAL;
    if (n_grads > SIGNMUON_MAX_MATRICES || workers > kMaxWorkers) return SIGNMUON_ERANGE;
    p.units = 0;
    for (int32_t i = 0; i < n_grads; ++i) {
        if (grads[i].n < 1) return SIGNMUON_EINVAL;
        if (grads[i].n > kMaxN) return SIGNMUON_ERANGE;
        p.units += clip_units(grads[i].n, sm::kClipUnit);
    }
    p.unit = sm::kClipUnit;
    if (p.units * workers < 512) {  // two workgroups a compute unit
        p.unit = sm::kClipSmallUnit;
        p.units = 0;
        for (int32_t i = 0; i < n_grads; ++i) p.units += clip_units(grads[i].n, p.unit);
    }
    p.factors = align_up((size_t)(p.units * workers) * sizeof(double));
    p.total = p.factors + (size_t)workers * sizeof(float);
    return SIGNMUON_OK;
}

// The norms of every worker, and, where `most` is given, what is clipped by them.
int run_gradients(const signmuon_gradient *grads, int32_t n_grads, int32_t workers, bool clip, float most,
                  float *norms, void *workspace, size_t workspace_bytes, hipStream_t st) {
    ClipPlan p{};
    if (int rc = check_gradients(grads, n_grads, workers, p)) return rc;
    if (!norms || (clip && (!std::isfinite(most) || most <= 0.0f))) return SIGNMUON_EINVAL;
    for (int32_t i = 0; i < n_grads; ++i) {
        if (!grads[i].grad || (clip && !grads[i].out)) return SIGNMUON_EINVAL;
        if (!dtype_ok(grads[i].dtype)) return SIGNMUON_EDTYPE;
        if (!aligned16(grads[i].grad) || (clip && !aligned16(grads[i].out))) return SIGNMUON_EALIGN;
    }
    if (!aligned16(norms)) return SIGNMUON_EALIGN;
    if (int rc = check_workspace(workspace, workspace_bytes, p.total)) return rc;
    char *ws = static_cast<char *>(workspace);
    // the batches of tensors, from the first to the last or back
    auto batches = [&](auto launch, bool back) -> int {
        int64_t unit = back ? p.units : 0;
        const int32_t last = (n_grads - 1) / sm::kClipTensors;
        for (int32_t k = 0; k <= last; ++k) {
            const int32_t i0 = (back ? last - k : k) * sm::kClipTensors;
            sm::ClipBatch b{};
            int64_t here = 0;
            for (int32_t i = i0; i < n_grads && i < i0 + sm::kClipTensors; ++i) {
                const int t = b.tensors++;
                b.grad[t] = grads[i].grad;
                b.out[t] = grads[i].out;
                b.n[t] = grads[i].n;
                b.first[t] = (int32_t)here;
                b.bf16[t] = grads[i].dtype == SIGNMUON_BF16;
                here += clip_units(grads[i].n, p.unit);
            }
            if (back) unit -= here;
            b.partial = reinterpret_cast<double *>(ws);
            b.factors = reinterpret_cast<const float *>(ws + p.factors);
            b.norms = norms;
            b.most = most;
            b.unit = p.unit;
            b.units = p.units;
            b.unit0 = unit;
            b.batch_units = (int32_t)here;
            b.workers = workers;
            if (!back) unit += here;
            launch(b, st);
            if (int rc = sm::launch_status()) return rc;
        }
        return SIGNMUON_OK;
    };
    if (int rc = batches(sm::launch_clip_norm, false)) return rc;
    if (!clip || p.units > sm::kClipFew) {
        sm::ClipFinish f{};
        f.partial = reinterpret_cast<const double *>(ws);
        f.norms = norms;
        f.factors = reinterpret_cast<float *>(ws + p.factors);
        f.units = p.units;
        f.most = clip ? most : 1.0f;
        f.workers = workers;
        sm::launch_clip_finish(f, st);
        if (int rc = sm::launch_status()) return rc;
    }
    return clip ? batches(sm::launch_clip_scale, true) : SIGNMUON_OK;
}

// ---------------------------------------------------------------------------
// Softmax cross entropy of an output layer: check_embedding, and
// ---------------------------------------------------------------------------
constexpr float kLog2E = 1.44269504088896340736f;
// What a piece of the vocabulary may take of the workspace where more than one
// tile's columns do: its maxima and sums, or its g, and the planes of its weights.
constexpr int64_t kLossForward = (int64_t)128 << 20, kLossBackward = (int64_t)1 << 30;
// What parts of k may take, forward; backward (of logits and of each gradient) kLossBackward.
// 14467 x 2202 x 8104 in fp32, 513 tiles for 256 places, takes 3.80 ms in five parts of 127 MB,
// 3.69 in the four that this holds and 5.85 in one; 15892 x 5428 x 3544 3.80 in two of 345 and 3.93 in one.
constexpr int64_t kLossForwardParts = (int64_t)512 << 20;

inline int loss_planes(int dtype) { return dtype == SIGNMUON_F32 ? 3 : 1; }
// Pairs of planes of a product of two operands (loss_pairs).
inline int loss_products(int a, int b) {
    return a == SIGNMUON_F32 && b == SIGNMUON_F32 ? 6 : a == SIGNMUON_F32 || b == SIGNMUON_F32 ? 3 : 1;
}

// Operands that the tiles read where they lie: BF16 rows of whole vectors.
inline bool loss_direct(int dtype, int64_t cols) { return dtype == SIGNMUON_BF16 && cols % 8 == 0; }

// Entries of the vocabulary in a piece: tiles, at most `most` entries, all pieces
// about as large.
int64_t loss_piece(int64_t vocab, int64_t most) {
    const int64_t tiles = (vocab + sm::kLossTile - 1) / sm::kLossTile;
    const int64_t each = most / sm::kLossTile > 1 ? most / sm::kLossTile : 1;
    const int64_t pieces = (tiles + each - 1) / each;
    return (tiles + pieces - 1) / pieces * sm::kLossTile;
}

// The tile and the parts of k of a product with `slices` slices, by a model of its time in
// slices of a tile of 256 x 256 (about 1.4 us): a round of tiles (one a compute unit, or two of
// 128 x 128) takes its slices and 4.5 more for the results, times a shape's two factors; a slice
// of an fp32 g's product 1.65, or 0.75 where one plane of it is taken; adding parts 3, or 4.5
// of logits, and 10 MB of them a slice. The large tile has the least traffic into LDS, two small ones a compute unit
// hide each other's results, and the middle one fills compute units that the large one leaves
// empty (us, large / middle / small):
//   logits 8192 x 50257 x 768                               571 / 666 / 660
//   logits 2048 x 10000 x 1024                               64 /  60 /  52
//   logits and dw, fp32, 1503 x 5003 x 512, three workers   159 / 118 / 127
//   logits and dw, fp32 W and dw, 2048 x 4000 x 2048        276 / 211 / 229
//   logits and dx 512 x 32000 x 4096                        256 / 310 / 322
// The compute units are those of a whole MI355X, not asked for, since the workspace's size is
// told without a device.
using sm::LossPlan;
using sm::LossTiles;
enum LossKind { kLogits, kNarrow, kWide };

LossTiles loss_tiles(LossKind kind, int64_t m, int64_t n, int64_t batch, int64_t slices, double slice, bool even,
                     int most_splits, bool summed = false) {
    struct Shape {
        int32_t tm, tn, slots;
        double slice, results;
    };
    const Shape shapes[3] = {{256, 256, 256, 1.0, 1.0},
                             {kind == kWide ? 128 : 256, kind == kWide ? 256 : 128, 256, kind == kNarrow ? 0.6 : 0.55, 0.7},
                             {128, 128, 512, kind == kNarrow ? 0.66 : 0.58, 0.5}};
    LossTiles best{};
    double best_time = 0.0;
    for (const Shape &t : shapes) {
        if (!even && t.tm * t.tn > 128 * 128) continue;
        const int64_t tiles = batch * ((m + t.tm - 1) / t.tm) * ((n + t.tn - 1) / t.tn);
        for (int64_t splits = 1; splits <= most_splits; ++splits) {
            const int64_t chunk = (slices + splits - 1) / splits, parts = (slices + chunk - 1) / chunk;
            if (parts < splits) continue;
            const double rounds = (double)((tiles * parts + t.slots - 1) / t.slots);
            double time = rounds * (t.slice * slice * (double)chunk + t.results * 4.5);
            if (parts > 1 || summed) time += (kind == kLogits ? 4.5 : 3.0) + (double)(parts * batch) * (double)m * (double)n * 8.0 / 1e7;
            if (best.tm == 0 || time < best_time) {
                best_time = time;
                best.tm = t.tm;
                best.tn = t.tn;
                best.splits = (int32_t)parts;
            }
        }
    }
    return best;
}

// Planes of an operand with `planes` that meet g: all for an fp32 result. A BF16 result, whose
// own rounding and g's are as large as one plane's, takes two (2.4e-3 of the result's norm off
// in all, where one plane would leave 2.9e-3 and the result's rounding alone is 1.7e-3).
inline int loss_meet(int planes, bool result32) { return result32 || planes == 1 ? planes : 2; }

// Up to so many tokens of all workers, g is held in fp32 and met in three planes for a BF16
// result too. A result of many tokens is off by g's rounding and its own, 2^(1/2) of the latter
// alone on average; where an entry or two of g decide, it may be off by 2.4 times: of few tokens that
// is every row, of many a rare target's row of dw, within half a step for g and half a step for
// itself; three planes would take three products for one there (dw of 8192 x 32000 x 4096: 1.65 ms).
// The count is of all workers, since one g serves dx and every worker's dw.
constexpr int64_t kLossFew = 128;

inline int64_t loss_slices(int64_t k, bool g32) {
    const int64_t slice = g32 ? sm::kLossWideSlice : sm::kLossSlice;
    return (k + slice - 1) / slice;
}

constexpr int kLossParts = 32;  // of k, at most
// Parts of k of rows x cols fp32 values that `budget` bytes hold.
inline int loss_most_parts(int64_t budget, int64_t rows, int64_t cols) {
    const int64_t most = budget / (rows * cols * (int64_t)sizeof(float));
    return most < 1 ? 1 : most < kLossParts ? (int)most : kLossParts;
}
inline int64_t loss_part_pitch(int64_t n) { return (n + 3) / 4 * 4; }
// Bytes of the logits' parts of k.
int64_t loss_logit_parts(const LossPlan &p, int64_t rows, int64_t vocab) {
    const int64_t here = vocab < p.piece ? vocab : p.piece;
    return p.logits.splits > 1 ? p.logits.splits * rows * loss_part_pitch(here) * (int64_t)sizeof(float) : 0;
}
// The logits' product of a piece, and what is made of parts of k.
int loss_logits(sm::LossTile &f, void *parts, bool grad, hipStream_t st) {
    f.out = parts;
    f.out_batch = f.m;
    f.out_pitch = loss_part_pitch(f.n);
    sm::launch_loss_logits(f, grad, st);
    if (int rc = sm::launch_status()) return rc;
    if (f.splits == 1) return SIGNMUON_OK;
    sm::launch_loss_parts(f, grad, st);
    return sm::launch_status();
}

}  // namespace

namespace sm {

LossPlan loss_plan(int64_t tokens, int64_t vocab, int64_t cols, int x_dtype, int w_dtype) {
    LossPlan p{};
    p.pitch = sm::loss_pitch(cols);
    int64_t most = kLossForward * 128 / (8 * tokens);
    const int64_t w_row = loss_direct(w_dtype, cols) ? 0 : loss_planes(w_dtype) * p.pitch * 2;
    if (w_row && kLossForward / w_row < most) most = kLossForward / w_row;
    p.piece = loss_piece(vocab, most);
    const int64_t here = vocab < p.piece ? vocab : p.piece;
    p.logits = loss_tiles(kLogits, tokens, here, 1, loss_products(x_dtype, w_dtype) * loss_slices(cols, false), 1.0, true,
                          loss_most_parts(kLossForwardParts, tokens, loss_part_pitch(here)));
    size_t at = 0;
    auto section = [&](int64_t bytes) {
        const size_t here = at;
        at += align_up((size_t)bytes);
        return here;
    };
    p.x = section(loss_direct(x_dtype, cols) ? 0 : loss_planes(x_dtype) * tokens * p.pitch * 2);
    p.w = section(w_row * p.piece);
    p.partial = section(tokens * (p.piece / (p.logits.tn / 2)) * (int64_t)sizeof(float2));
    p.part = section(loss_logit_parts(p, tokens, vocab));
    p.state = section(p.piece < vocab ? tokens * (int64_t)sizeof(float2) : 0);
    p.target = section(tokens * (int64_t)sizeof(float));
    p.total = at;
    return p;
}

LossPlan loss_grad_plan(int64_t workers, int64_t tokens, int64_t vocab, int64_t cols, int x_dtype, int w_dtype,
                        int grad_dtype, bool want_dw) {
    LossPlan p{};
    const int64_t rows = workers * tokens;
    p.pitch = sm::loss_pitch(cols);
    const bool x32 = x_dtype == SIGNMUON_F32, grad32 = grad_dtype == SIGNMUON_F32, few = rows <= kLossFew;
    const bool g32 = x32 || grad32 || few;
    p.few = few;
    p.g32 = g32;
    const int64_t entry = g32 ? 4 : 2;  // bytes of g's
    int64_t most = kLossBackward / (entry * rows);
    const int64_t w_row = loss_direct(w_dtype, cols) ? 0 : loss_planes(w_dtype) * p.pitch * 2;
    if (w_row && kLossBackward / w_row < most) most = kLossBackward / w_row;
    p.piece = loss_piece(vocab, most);
    const int64_t here = vocab < p.piece ? vocab : p.piece;
    const bool summed = p.piece < vocab || (few && !x32);  // that product has fp32 results
    p.logits = loss_tiles(kLogits, rows, here, 1, loss_products(x_dtype, w_dtype) * loss_slices(cols, false), 1.0, true,
                          loss_most_parts(kLossBackward, rows, loss_part_pitch(here)));
    p.dx = loss_tiles(g32 ? kWide : kNarrow, rows, cols, 1, loss_meet(loss_planes(w_dtype), x32) * loss_slices(here, g32),
                      !g32 ? 1.0 : x32 || few ? 1.65 : 0.75, cols % (x32 ? 4 : 8) == 0,
                      loss_most_parts(kLossBackward, rows, cols), summed);
    p.parts = summed || p.dx.splits > 1;
    // Parts of the tokens only where half of the compute units' places would be empty: 225 x 44 of
    // eight workers takes 24 us in parts and 196 without, 5003 x 515 of three 110 and 89.
    const bool whole = grad32 || few;
    const int64_t dw_tiles = workers * ((here + 127) / 128) * ((cols + 127) / 128);
    p.dw = loss_tiles(g32 ? kWide : kNarrow, here, cols, workers,
                      loss_meet(loss_planes(x_dtype), grad32) * loss_slices(tokens, g32), !g32 ? 1.0 : whole ? 1.65 : 0.75,
                      cols % (grad32 ? 4 : 8) == 0 && (grad32 || !few), dw_tiles <= 256 ? loss_most_parts(kLossBackward, workers * here, cols) : 1);
    size_t at = 0;
    auto section = [&](int64_t bytes) {
        const size_t here = at;
        at += align_up((size_t)bytes);
        return here;
    };
    p.x = section(loss_planes(x_dtype) * rows * p.pitch * 2);
    p.w = section(w_row * p.piece);
    for (size_t &r : p.row) r = section(rows * 4);
    p.g = section(entry * rows * p.piece);
    p.sum = section(p.piece < vocab && !x32 ? rows * cols * (int64_t)sizeof(float) : 0);
    // the parts of each product are read before the next one's are written
    const int64_t dx_part = p.parts ? p.dx.splits * rows * cols * (int64_t)sizeof(float) : 0;
    const int64_t dw_part = want_dw && p.dw.splits > 1 ? p.dw.splits * workers * here * cols * (int64_t)sizeof(float) : 0;
    const int64_t logit_part = loss_logit_parts(p, rows, vocab), part = dx_part > dw_part ? dx_part : dw_part;
    p.part = section(part > logit_part ? part : logit_part);
    p.total = at;
    return p;
}

}  // namespace sm

namespace {

// The pairs of planes i of a and j of b with i + j below the longer one's count. An
// fp32 a (in one piece) meets each plane of b with as many of its own.
void loss_pairs(sm::LossTile &f, int na, int nb, bool whole_a = false) {
    const int most = na > nb ? na : nb;
    f.pairs = 0;
    f.order_a = f.order_b = 0;
    auto pair = [&](int a, int b) {
        f.order_a |= (uint32_t)a << (2 * f.pairs);
        f.order_b |= (uint32_t)b << (2 * f.pairs);
        ++f.pairs;
    };
    for (int j = 0; j < nb; ++j) {
        const int here = na < most - j ? na : most - j;
        for (int i = 0; i < (whole_a ? 1 : here); ++i) pair(i, j);
    }
}

// The tile, and the slices of each part of k.
void loss_set_tiles(sm::LossTile &f, const LossTiles &t) {
    f.tm = t.tm;
    f.tn = t.tn;
    const int64_t slices = f.pairs * loss_slices(f.k, f.g32 && f.planes > 0);
    f.chunk = (int32_t)((slices + t.splits - 1) / t.splits);
    f.splits = (int32_t)((slices + f.chunk - 1) / f.chunk);
}

// One operand's planes, in the workspace or where it lies.
void loss_operand(const void *(&planes)[sm::kLossPlanes], int n, const void *at, int64_t plane_entries) {
    for (int i = 0; i < n; ++i) planes[i] = static_cast<const uint16_t *>(at) + i * plane_entries;
}

sm::LossPlanes loss_to_planes(const void *in, int dtype, int64_t rows, int64_t cols, int64_t pitch, void *to) {
    sm::LossPlanes f{};
    f.in = in;
    f.planes = loss_planes(dtype);
    for (int i = 0; i < f.planes; ++i) f.out[i] = static_cast<uint16_t *>(to) + i * rows * pitch;
    f.rows = rows;
    f.cols = cols;
    f.pitch = pitch;
    f.bf16 = dtype == SIGNMUON_BF16;
    return f;
}

inline int64_t entry_bytes(int dtype) { return dtype == SIGNMUON_BF16 ? 2 : 4; }
inline const void *at_entry(const void *p, int64_t i, int dtype) {
    return static_cast<const char *>(p) + i * entry_bytes(dtype);
}

// ---------------------------------------------------------------------------
// 8-bit floating point
// ---------------------------------------------------------------------------
constexpr int64_t kMaxK = (int64_t)1 << 22;     // a tile's rows of an operand lie within 2^31 bytes
constexpr int64_t kMaxF8Cols = (int64_t)1 << 21;  // and so do a wave's rows of out
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;  // of a launch

inline bool f8_ok(int f) { return f == SIGNMUON_E4M3 || f == SIGNMUON_E5M2; }

int check_f8_matmul(int64_t batch, int64_t m, int64_t n, int64_t k) {
    if (batch < 1 || m < 1 || n < 1 || k < 1) return SIGNMUON_EINVAL;
    if (batch > kMaxWorkers || m > kMaxTokens || n > kMaxF8Cols || k > kMaxK) return SIGNMUON_ERANGE;
    const sm::F8Plan p = sm::f8_plan(batch, m, n, k);
    if (p.tile == 16) return batch * ((n + 15) / 16) * p.waves * 64 > kMaxThreads ? SIGNMUON_ERANGE : SIGNMUON_OK;
    const int64_t tiles = ((m + p.tile - 1) / p.tile) * ((n + p.tile - 1) / p.tile);
    return tiles * batch * p.splits > INT32_MAX / 2 ? SIGNMUON_ERANGE : SIGNMUON_OK;
}

size_t f8_workspace(int64_t batch, int64_t m, int64_t n, int64_t k) {
    const sm::F8Plan p = sm::f8_plan(batch, m, n, k);
    return p.splits > 1 ? (size_t)(p.splits * batch * m * n) * sizeof(float) : 0;
}

}  // namespace

extern "C" {

int signmuon_embedding(const void *ids, signmuon_itype id_type, const void *table,
                       signmuon_dtype table_dtype, int64_t tokens, int64_t vocab, int64_t cols,
                       float scale, void *y, signmuon_dtype y_dtype, signmuon_stream stream) {
    if (!ids || !table || !y) return SIGNMUON_EINVAL;
    if (int rc = check_embedding(1, tokens, vocab, cols)) return rc;
    if (!std::isfinite(scale)) return SIGNMUON_EINVAL;
    if ((id_type != SIGNMUON_I32 && id_type != SIGNMUON_I64) || !dtype_ok(table_dtype) || !dtype_ok(y_dtype))
        return SIGNMUON_EDTYPE;
    if (!all_aligned(ids, table, y)) return SIGNMUON_EALIGN;
    sm::Embed e{};
    e.ids = ids;
    e.table = table;
    e.y = y;
    e.tokens = tokens;
    e.vocab = vocab;
    e.cols = cols;
    e.scale = scale;
    e.id64 = id_type == SIGNMUON_I64;
    e.table_bf16 = table_dtype == SIGNMUON_BF16;
    e.y_bf16 = y_dtype == SIGNMUON_BF16;
    sm::launch_embedding(e, static_cast<hipStream_t>(stream));
    return sm::launch_status();
}

size_t signmuon_embedding_workspace_bytes(int32_t workers, int64_t tokens, int64_t vocab, int64_t cols) {
    if (check_embedding(workers, tokens, vocab, cols) != SIGNMUON_OK) return 0;
    return embedding_plan(workers, tokens, cols).total;
}

int signmuon_embedding_backward(const void *ids, signmuon_itype id_type, const void *dy,
                                signmuon_dtype dy_dtype, int32_t workers, int64_t tokens,
                                int64_t vocab, int64_t cols, float scale, void *grad,
                                signmuon_dtype grad_dtype, int32_t accumulate, void *workspace,
                                size_t workspace_bytes, signmuon_stream stream) {
    if (!ids || !dy || !grad) return SIGNMUON_EINVAL;
    if (int rc = check_embedding(workers, tokens, vocab, cols)) return rc;
    if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return SIGNMUON_EINVAL;
    if ((id_type != SIGNMUON_I32 && id_type != SIGNMUON_I64) || !dtype_ok(dy_dtype) || !dtype_ok(grad_dtype))
        return SIGNMUON_EDTYPE;
    if (!all_aligned(ids, dy, grad)) return SIGNMUON_EALIGN;
    const EmbedPlan p = embedding_plan(workers, tokens, cols);
    if (int rc = check_workspace(workspace, workspace_bytes, p.total)) return rc;
    char *ws = static_cast<char *>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sm::EmbedGrad e{};
    e.ids = ids;
    e.dy = dy;
    e.grad = grad;
    e.keys[0] = reinterpret_cast<uint64_t *>(ws + p.keys[0]);
    e.keys[1] = reinterpret_cast<uint64_t *>(ws + p.keys[1]);
    e.partial = reinterpret_cast<float *>(ws + p.partial);
    e.tokens = tokens;
    e.vocab = vocab;
    e.cols = cols;
    e.workers = workers;
    e.seg = p.seg;
    e.segments = p.segments;
    e.scale = scale;
    e.id64 = id_type == SIGNMUON_I64;
    e.dy_bf16 = dy_dtype == SIGNMUON_BF16;
    e.grad_bf16 = grad_dtype == SIGNMUON_BF16;
    e.accumulate = accumulate != 0;
    sm::launch_embedding_sort(e, st);
    if (int rc = sm::launch_status()) return rc;
    for (int pass = 0; pass < sm::embed_merge_passes(tokens); ++pass) {
        sm::launch_embedding_merge(e, pass, st);
        if (int rc = sm::launch_status()) return rc;
    }
    sm::launch_embedding_sums(e, st);
    if (int rc = sm::launch_status()) return rc;
    if (e.segments == 1) return SIGNMUON_OK;
    sm::launch_embedding_join(e, st);
    return sm::launch_status();
}

int signmuon_layer_norm(const void *x, signmuon_dtype x_dtype, int64_t rows, int64_t cols,
                        const float *gamma, const float *beta, float eps, void *y, float *mean,
                        float *rstd, signmuon_stream stream) {
    if (!x || !gamma || !y) return SIGNMUON_EINVAL;
    if (int rc = check_norm(1, rows, cols)) return rc;
    if (!std::isfinite(eps) || eps <= 0.0f) return SIGNMUON_EINVAL;
    if (!dtype_ok(x_dtype)) return SIGNMUON_EDTYPE;
    if (!all_aligned(x, gamma, beta, y, mean, rstd)) return SIGNMUON_EALIGN;
    sm::Norm n{};
    n.x = x;
    n.gamma = gamma;
    n.beta = beta;
    n.y = y;
    n.mean = mean;
    n.rstd = rstd;
    n.rows = rows;
    n.cols = cols;
    n.eps = eps;
    n.bf16 = x_dtype == SIGNMUON_BF16;
    sm::launch_layer_norm(n, static_cast<hipStream_t>(stream));
    return sm::launch_status();
}

size_t signmuon_layer_norm_workspace_bytes(int32_t workers, int64_t rows, int64_t cols) {
    if (check_norm(workers, rows, cols) != SIGNMUON_OK) return 0;
    return norm_workspace(workers, rows, cols);
}

int signmuon_layer_norm_backward(const void *dy, const void *x, signmuon_dtype x_dtype,
                                 int32_t workers, int64_t rows, int64_t cols, const float *gamma,
                                 const float *mean, const float *rstd, void *dx, void *dgamma,
                                 void *dbeta, signmuon_dtype grad_dtype, void *workspace,
                                 size_t workspace_bytes, signmuon_stream stream) {
    if (!dy || !x || !gamma || !mean || !rstd || (!dx && !dgamma && !dbeta)) return SIGNMUON_EINVAL;
    if (int rc = check_norm(workers, rows, cols)) return rc;
    if (!dtype_ok(x_dtype) || !dtype_ok(grad_dtype)) return SIGNMUON_EDTYPE;
    if (!all_aligned(dy, x, gamma, mean, rstd, dx, dgamma, dbeta)) return SIGNMUON_EALIGN;
    if (int rc = check_workspace(workspace, workspace_bytes, norm_workspace(workers, rows, cols))) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sm::NormGrad n{};
    n.dy = dy;
    n.x = x;
    n.gamma = gamma;
    n.mean = mean;
    n.rstd = rstd;
    n.dx = dx;
    n.dgamma = dgamma;
    n.dbeta = dbeta;
    n.partial = static_cast<float *>(workspace);
    n.rows = rows;
    n.cols = cols;
    n.workers = workers;
    n.parts = sm::norm_parts(workers, rows, cols);
    n.bf16 = x_dtype == SIGNMUON_BF16;
    n.grad_bf16 = grad_dtype == SIGNMUON_BF16;
    sm::launch_layer_norm_backward(n, st);
    if (int rc = sm::launch_status()) return rc;
    if (n.parts == 1 || (!dgamma && !dbeta)) return SIGNMUON_OK;
    sm::launch_layer_norm_sums(n, st);
    return sm::launch_status();
}

size_t signmuon_f8_pitch(int64_t k) { return k < 1 || k > kMaxTokens ? 0 : (size_t)sm::f8_pitch(k); }

size_t signmuon_f8_scale_pitch(int64_t k) {
    return k < 1 || k > kMaxTokens ? 0 : (size_t)sm::f8_scale_pitch(k);
}

int signmuon_f8_quant(const void *x, signmuon_dtype x_dtype, int32_t batch, int64_t rows,
                      int64_t cols, signmuon_f8 format, void *q, uint8_t *q_scale, void *qt,
                      uint8_t *qt_scale, signmuon_stream stream) {
    if (!x || (!q && !qt) || !q != !q_scale || !qt != !qt_scale) return SIGNMUON_EINVAL;
    if (batch < 1 || rows < 1 || cols < 1) return SIGNMUON_EINVAL;
    if (batch > kMaxWorkers || rows > kMaxTokens || cols > kMaxTokens) return SIGNMUON_ERANGE;
    const int64_t row_tiles = (rows + 127) / 128, col_tiles = (cols + 127) / 128;
    if (batch * row_tiles * col_tiles * 256 > kMaxThreads) return SIGNMUON_ERANGE;
    if (!dtype_ok(x_dtype) || !f8_ok(format)) return SIGNMUON_EDTYPE;
    if (!all_aligned(x, q, q_scale, qt, qt_scale)) return SIGNMUON_EALIGN;
    sm::F8Quant f{};
    f.x = x;
    f.q = static_cast<uint8_t *>(q);
    f.q_scale = q_scale;
    f.qt = static_cast<uint8_t *>(qt);
    f.qt_scale = qt_scale;
    f.rows = rows;
    f.cols = cols;
    f.pitch = sm::f8_pitch(cols);
    f.scale_pitch = sm::f8_scale_pitch(cols);
    f.tpitch = sm::f8_pitch(rows);
    f.tscale_pitch = sm::f8_scale_pitch(rows);
    f.batch = batch;
    f.row_tiles = (int32_t)row_tiles;
    f.col_tiles = (int32_t)col_tiles;
    f.bf16 = x_dtype == SIGNMUON_BF16;
    f.e5m2 = format == SIGNMUON_E5M2;
    sm::launch_f8_quant(f, static_cast<hipStream_t>(stream));
    return sm::launch_status();
}

size_t signmuon_f8_matmul_workspace_bytes(int32_t batch, int64_t m, int64_t n, int64_t k) {
    if (check_f8_matmul(batch, m, n, k) != SIGNMUON_OK) return 0;
    return f8_workspace(batch, m, n, k);
}

int signmuon_f8_matmul(const void *a, const uint8_t *a_scale, signmuon_f8 a_format, const void *b,
                       const uint8_t *b_scale, signmuon_f8 b_format, int32_t batch, int64_t m,
                       int64_t n, int64_t k, int32_t b_shared, void *out, signmuon_dtype out_dtype,
                       void *workspace, size_t workspace_bytes, signmuon_stream stream) {
    if (!a || !a_scale || !b || !b_scale || !out || (b_shared != 0 && b_shared != 1)) return SIGNMUON_EINVAL;
    if (int rc = check_f8_matmul(batch, m, n, k)) return rc;
    if (!f8_ok(a_format) || !f8_ok(b_format) || !dtype_ok(out_dtype)) return SIGNMUON_EDTYPE;
    if (!all_aligned(a, a_scale, b, b_scale, out)) return SIGNMUON_EALIGN;
    // rows of a shared b are one product: fuller tiles. Not where that product would
    // want more workspace than the batch (whose size is asked for without b_shared),
    // such as parts of k where up to 32 rows an entry need none: 8 x 16 rows of 11008 x
    // 4096 take 90 us, and 21 as one product.
    if (b_shared && batch > 1 && batch * m <= kMaxTokens && check_f8_matmul(1, batch * m, n, k) == SIGNMUON_OK &&
        f8_workspace(1, batch * m, n, k) <= f8_workspace(batch, m, n, k)) {
        m *= batch;
        batch = 1;
    }
    if (int rc = check_workspace(workspace, workspace_bytes, f8_workspace(batch, m, n, k))) return rc;
    const sm::F8Plan p = sm::f8_plan(batch, m, n, k);
    sm::F8Matmul f{};
    f.a = static_cast<const uint8_t *>(a);
    f.a_scale = a_scale;
    f.b = static_cast<const uint8_t *>(b);
    f.b_scale = b_scale;
    f.out = out;
    f.partial = static_cast<float *>(workspace);
    f.m = m;
    f.n = n;
    f.pitch = sm::f8_pitch(k);
    f.scale_pitch = sm::f8_scale_pitch(k);
    f.a_stride = m * f.pitch;
    f.as_stride = m * f.scale_pitch;
    f.b_stride = b_shared ? 0 : n * f.pitch;
    f.bs_stride = b_shared ? 0 : n * f.scale_pitch;
    f.batch = batch;
    f.blocks = (int32_t)(f.pitch / sm::kF8Block);
    f.splits = p.splits;
    f.chunk = p.chunk;
    f.tile = p.tile;
    f.waves = p.waves;
    f.a_e5m2 = a_format == SIGNMUON_E5M2;
    f.b_e5m2 = b_format == SIGNMUON_E5M2;
    f.out_bf16 = out_dtype == SIGNMUON_BF16;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sm::launch_f8_matmul(f, st);
    if (int rc = sm::launch_status()) return rc;
    if (f.splits == 1) return SIGNMUON_OK;
    sm::launch_f8_sums(f, st);
    return sm::launch_status();
}

int signmuon_rms_norm(const void *x, const void *residual, signmuon_dtype x_dtype, int64_t rows,
                      int64_t cols, const float *gamma, float eps, void *h, void *y,
                      signmuon_f8 format, void *q, uint8_t *q_scale, float *rstd,
                      signmuon_stream stream) {
    if (!x || !gamma || (!y && !q) || !q != !q_scale || (h && !residual)) return SIGNMUON_EINVAL;
    if (int rc = check_norm(1, rows, cols)) return rc;
    if (!std::isfinite(eps) || eps <= 0.0f) return SIGNMUON_EINVAL;
    if (!dtype_ok(x_dtype) || (q && !f8_ok(format))) return SIGNMUON_EDTYPE;
    if (!all_aligned(x, residual, gamma, h, y, q, q_scale, rstd)) return SIGNMUON_EALIGN;
    sm::RmsNorm n{};
    n.x = x;
    n.residual = residual;
    n.gamma = gamma;
    n.h = h;
    n.y = y;
    n.q = static_cast<uint8_t *>(q);
    n.q_scale = q_scale;
    n.rstd = rstd;
    n.rows = rows;
    n.cols = cols;
    n.pitch = sm::f8_pitch(cols);
    n.scale_pitch = sm::f8_scale_pitch(cols);
    n.eps = eps;
    n.bf16 = x_dtype == SIGNMUON_BF16;
    n.e5m2 = format == SIGNMUON_E5M2;
    sm::launch_rms_norm(n, static_cast<hipStream_t>(stream));
    return sm::launch_status();
}

size_t signmuon_rms_norm_workspace_bytes(int32_t workers, int64_t rows, int64_t cols) {
    if (check_norm(workers, rows, cols) != SIGNMUON_OK) return 0;
    return rms_workspace(workers, rows, cols);
}

int signmuon_rms_norm_backward(const void *dy, const void *dh, const void *h, signmuon_dtype x_dtype,
                               int32_t workers, int64_t rows, int64_t cols, const float *gamma,
                               const float *rstd, void *dx, void *dgamma, signmuon_dtype grad_dtype,
                               void *workspace, size_t workspace_bytes, signmuon_stream stream) {
    if (!dy || !h || !gamma || !rstd || (!dx && !dgamma)) return SIGNMUON_EINVAL;
    if (int rc = check_norm(workers, rows, cols)) return rc;
    if (!dtype_ok(x_dtype) || !dtype_ok(grad_dtype)) return SIGNMUON_EDTYPE;
    if (!all_aligned(dy, dh, h, gamma, rstd, dx, dgamma)) return SIGNMUON_EALIGN;
    if (int rc = check_workspace(workspace, workspace_bytes, rms_workspace(workers, rows, cols))) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sm::RmsGrad n{};
    n.dy = dy;
    n.dh = dh;
    n.h = h;
    n.gamma = gamma;
    n.rstd = rstd;
    n.dx = dx;
    n.dgamma = dgamma;
    n.partial = static_cast<float *>(workspace);
    n.rows = rows;
    n.cols = cols;
    n.workers = workers;
    n.parts = sm::rms_parts(workers, rows, cols);
    n.bf16 = x_dtype == SIGNMUON_BF16;
    n.grad_bf16 = grad_dtype == SIGNMUON_BF16;
    sm::launch_rms_norm_backward(n, st);
    if (int rc = sm::launch_status()) return rc;
    if (n.parts == 1 || !dgamma) return SIGNMUON_OK;
    sm::launch_rms_norm_sums(n, st);
    return sm::launch_status();
}

size_t signmuon_grad_norm_workspace_bytes(const signmuon_gradient *grads, int32_t n_grads, int32_t workers) {
    ClipPlan p{};
    return check_gradients(grads, n_grads, workers, p) == SIGNMUON_OK ? p.total : 0;
}

int signmuon_grad_norm(const signmuon_gradient *grads, int32_t n_grads, int32_t workers, float *norms,
                       void *workspace, size_t workspace_bytes, signmuon_stream stream) {
    return run_gradients(grads, n_grads, workers, false, 0.0f, norms, workspace, workspace_bytes,
                         static_cast<hipStream_t>(stream));
}

int signmuon_clip_grads(const signmuon_gradient *grads, int32_t n_grads, int32_t workers, float max_norm,
                        float *norms, void *workspace, size_t workspace_bytes, signmuon_stream stream) {
    return run_gradients(grads, n_grads, workers, true, max_norm, norms, workspace, workspace_bytes,
                         static_cast<hipStream_t>(stream));
}

size_t signmuon_linear_cross_entropy_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols,
                                                     signmuon_dtype x_dtype, signmuon_dtype w_dtype) {
    if (check_embedding(1, tokens, vocab, cols) != SIGNMUON_OK || !dtype_ok(x_dtype) || !dtype_ok(w_dtype)) return 0;
    return sm::loss_plan(tokens, vocab, cols, x_dtype, w_dtype).total;
}

int signmuon_linear_cross_entropy(const void *x, signmuon_dtype x_dtype, const void *w, signmuon_dtype w_dtype,
                                  const void *targets, signmuon_itype target_type, int64_t tokens,
                                  int64_t vocab, int64_t cols, float scale, float *loss, float *lse,
                                  void *workspace, size_t workspace_bytes, signmuon_stream stream) {
    if (!x || !w || !targets || (!loss && !lse)) return SIGNMUON_EINVAL;
    if (int rc = check_embedding(1, tokens, vocab, cols)) return rc;
    if (!std::isfinite(scale)) return SIGNMUON_EINVAL;
    if ((target_type != SIGNMUON_I32 && target_type != SIGNMUON_I64) || !dtype_ok(x_dtype) || !dtype_ok(w_dtype))
        return SIGNMUON_EDTYPE;
    if (!all_aligned(x, w, targets, loss, lse)) return SIGNMUON_EALIGN;
    const LossPlan p = sm::loss_plan(tokens, vocab, cols, x_dtype, w_dtype);
    if (int rc = check_workspace(workspace, workspace_bytes, p.total)) return rc;
    char *ws = static_cast<char *>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool direct_x = loss_direct(x_dtype, cols), direct_w = loss_direct(w_dtype, cols);
    const int nx = loss_planes(x_dtype), nw = loss_planes(w_dtype);
    if (!direct_x) {
        sm::launch_loss_planes(loss_to_planes(x, x_dtype, tokens, cols, p.pitch, ws + p.x), st);
        if (int rc = sm::launch_status()) return rc;
    }
    for (int64_t v0 = 0; v0 < vocab; v0 += p.piece) {
        const int64_t here = vocab - v0 < p.piece ? vocab - v0 : p.piece;
        const void *rows = at_entry(w, v0 * cols, w_dtype);
        if (!direct_w) {
            sm::launch_loss_planes(loss_to_planes(rows, w_dtype, here, cols, p.pitch, ws + p.w), st);
            if (int rc = sm::launch_status()) return rc;
        }
        sm::LossTile f{};
        loss_operand(f.a, nx, direct_x ? x : ws + p.x, tokens * p.pitch);
        loss_operand(f.b, nw, direct_w ? rows : ws + p.w, here * p.pitch);
        f.a_pitch = f.b_pitch = p.pitch * 2;
        f.m = tokens;
        f.n = here;
        f.k = cols;
        f.batch = 1;
        loss_pairs(f, nx, nw);
        loss_set_tiles(f, p.logits);
        f.plain_a = f.pairs > 1 ? x : nullptr;
        f.plain_a16 = x_dtype == SIGNMUON_BF16;
        f.plain_b = rows;
        f.plain_b16 = w_dtype == SIGNMUON_BF16;
        f.rows[0] = targets;
        f.row_step = target_type == SIGNMUON_I64 ? 8 : 4;
        f.partial = reinterpret_cast<float2 *>(ws + p.partial);
        f.target = reinterpret_cast<float *>(ws + p.target);
        f.vocab0 = v0;
        f.factor = scale * kLog2E;
        if (int rc = loss_logits(f, ws + p.part, false, st)) return rc;
        sm::LossJoin j{};
        j.partial = f.partial;
        j.state = reinterpret_cast<float2 *>(ws + p.state);
        j.target = f.target;
        j.targets = targets;
        j.targets64 = target_type == SIGNMUON_I64;
        j.loss = loss;
        j.lse = lse;
        j.rows = tokens;
        const int64_t block = f.splits > 1 ? sm::kLossBlock : f.tn / 2;
        j.blocks = (here + block - 1) / block;
        j.vocab = vocab;
        j.first = v0 == 0;
        j.last = v0 + here == vocab;
        sm::launch_loss_join(j, st);
        if (int rc = sm::launch_status()) return rc;
    }
    return SIGNMUON_OK;
}

size_t signmuon_linear_cross_entropy_backward_workspace_bytes(int32_t workers, int64_t tokens, int64_t vocab,
                                                              int64_t cols, signmuon_dtype x_dtype,
                                                              signmuon_dtype w_dtype, signmuon_dtype grad_dtype) {
    if (check_embedding(workers, tokens, vocab, cols) != SIGNMUON_OK || !dtype_ok(x_dtype) || !dtype_ok(w_dtype) ||
        !dtype_ok(grad_dtype))
        return 0;
    return sm::loss_grad_plan(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype, true).total;
}

int signmuon_linear_cross_entropy_backward(const void *x, signmuon_dtype x_dtype, const void *w,
                                           signmuon_dtype w_dtype, const void *targets,
                                           signmuon_itype target_type, int32_t workers, int64_t tokens,
                                           int64_t vocab, int64_t cols, float scale, const float *lse,
                                           const float *dloss, void *dx, void *dw, signmuon_dtype grad_dtype,
                                           int32_t accumulate, void *workspace, size_t workspace_bytes,
                                           signmuon_stream stream) {
    if (!x || !w || !targets || !lse || !dloss || (!dx && !dw)) return SIGNMUON_EINVAL;
    if (int rc = check_embedding(workers, tokens, vocab, cols)) return rc;
    if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return SIGNMUON_EINVAL;
    if ((target_type != SIGNMUON_I32 && target_type != SIGNMUON_I64) || !dtype_ok(x_dtype) || !dtype_ok(w_dtype) ||
        !dtype_ok(grad_dtype))
        return SIGNMUON_EDTYPE;
    if (!all_aligned(x, w, targets, lse, dloss, dx, dw)) return SIGNMUON_EALIGN;
    const LossPlan p = sm::loss_grad_plan(workers, tokens, vocab, cols, x_dtype, w_dtype, grad_dtype, dw != nullptr);
    if (int rc = check_workspace(workspace, workspace_bytes, p.total)) return rc;
    char *ws = static_cast<char *>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t rows = workers * tokens;
    const bool direct_w = loss_direct(w_dtype, cols);
    const bool x32 = x_dtype == SIGNMUON_F32, grad32 = grad_dtype == SIGNMUON_F32;
    const int nx = loss_planes(x_dtype), nw = loss_planes(w_dtype);
    void *const g = ws + p.g;
    const bool few = p.few, g32 = p.g32;
    const int64_t g_entry = g32 ? 4 : 2;
    sm::LossPlanes xs = loss_to_planes(x, x_dtype, rows, cols, p.pitch, ws + p.x);
    xs.targets = targets;
    xs.targets64 = target_type == SIGNMUON_I64;
    xs.lse = lse;
    xs.dloss = dloss;
    xs.row_target = reinterpret_cast<int32_t *>(ws + p.row[0]);
    xs.row_base = reinterpret_cast<float *>(ws + p.row[1]);
    xs.row_d = reinterpret_cast<float *>(ws + p.row[2]);
    xs.vocab = vocab;
    xs.scale = scale;
    sm::launch_loss_planes(xs, st);
    if (int rc = sm::launch_status()) return rc;
    for (int64_t v0 = 0; v0 < vocab; v0 += p.piece) {
        const int64_t here = vocab - v0 < p.piece ? vocab - v0 : p.piece;
        const int64_t g_pitch = (here + sm::kLossTile - 1) / sm::kLossTile * sm::kLossTile;
        const bool first = v0 == 0, last = v0 + here == vocab;
        const void *w_rows = at_entry(w, v0 * cols, w_dtype);
        if (!direct_w) {
            sm::launch_loss_planes(loss_to_planes(w_rows, w_dtype, here, cols, p.pitch, ws + p.w), st);
            if (int rc = sm::launch_status()) return rc;
        }
        sm::LossTile f{};
        loss_operand(f.a, nx, ws + p.x, rows * p.pitch);
        loss_operand(f.b, nw, direct_w ? w_rows : ws + p.w, here * p.pitch);
        f.a_pitch = f.b_pitch = p.pitch * 2;
        f.m = rows;
        f.n = here;
        f.k = cols;
        f.batch = 1;
        loss_pairs(f, nx, nw);
        loss_set_tiles(f, p.logits);
        for (int i = 0; i < 3; ++i) f.rows[i] = ws + p.row[i];
        f.row_step = 4;
        f.plain_a = f.pairs > 1 ? x : nullptr;
        f.plain_a16 = x_dtype == SIGNMUON_BF16;
        f.plain_b = w_rows;
        f.plain_b16 = w_dtype == SIGNMUON_BF16;
        f.g = g;
        f.g32 = g32;
        f.g_pitch = g_pitch;
        f.vocab0 = v0;
        f.factor = scale * kLog2E;
        if (int rc = loss_logits(f, ws + p.part, true, st)) return rc;
        if (dx) {
            sm::LossTile d{};
            d.a[0] = g;
            loss_operand(d.b, nw, f.b[0], here * p.pitch);
            d.a_pitch = g_pitch * g_entry;
            d.b_pitch = p.pitch * 2;
            d.m = rows;
            d.n = cols;
            d.k = here;
            d.batch = 1;
            d.g32 = g32;
            d.planes = x32 || few ? 3 : 1;
            loss_pairs(d, d.planes, loss_meet(nw, x32), g32);
            loss_set_tiles(d, p.dx);
            d.out_batch = rows;
            d.out_pitch = cols;
            // in parts, or over several pieces, the sums so far lie in dx itself or in fp32 beside it
            float *const sums = x32 ? static_cast<float *>(dx) : reinterpret_cast<float *>(ws + p.sum);
            d.out = p.parts ? ws + p.part : dx;
            d.out_bf16 = !p.parts && !x32;
            sm::launch_loss_dx(d, st);
            if (int rc = sm::launch_status()) return rc;
            if (p.parts) {
                sm::LossSums u{};
                u.partial = reinterpret_cast<const float *>(ws + p.part);
                u.prev = first ? nullptr : sums;
                u.out = last ? dx : sums;
                u.total = u.pitch = rows * cols;
                u.splits = d.splits;
                u.out_bf16 = last && !x32;
                sm::launch_loss_sums(u, st);
                if (int rc = sm::launch_status()) return rc;
            }
        }
        if (dw) {
            sm::LossTile d{};
            d.a[0] = g;
            loss_operand(d.b, nx, ws + p.x, rows * p.pitch);
            d.a_pitch = g_pitch * g_entry;
            d.b_pitch = p.pitch * 2;
            d.a_batch = tokens * d.a_pitch;
            d.b_batch = tokens * d.b_pitch;
            d.m = here;
            d.n = cols;
            d.k = tokens;
            d.batch = workers;
            d.g32 = g32;
            d.planes = grad32 || few ? 3 : 1;
            loss_pairs(d, d.planes, loss_meet(nx, grad32), g32);
            const bool parts = p.dw.splits > 1;
            d.out = parts ? ws + p.part : const_cast<void *>(at_entry(dw, v0 * cols, grad_dtype));
            d.out_batch = parts ? here : vocab;
            d.out_pitch = cols;
            d.out_bf16 = !parts && !grad32;
            d.add = !parts && accumulate;
            loss_set_tiles(d, p.dw);
            sm::launch_loss_dw(d, st);
            if (int rc = sm::launch_status()) return rc;
            if (parts) {
                // a piece of several workers' dw is in as many places
                const int32_t places = here < vocab ? workers : 1;
                sm::LossSums u{};
                u.total = workers / places * here * cols;
                u.splits = d.splits;
                u.prev_bf16 = u.out_bf16 = !grad32;
                for (int32_t i = 0; i < places; ++i) {
                    u.out = const_cast<void *>(at_entry(dw, (i * vocab + v0) * cols, grad_dtype));
                    u.partial = reinterpret_cast<const float *>(ws + p.part) + i * here * cols;
                    u.prev = accumulate ? u.out : nullptr;
                    u.pitch = workers * here * cols;
                    sm::launch_loss_sums(u, st);
                    if (int rc = sm::launch_status()) return rc;
                }
            }
        }
    }
    return SIGNMUON_OK;
}

}  // extern "C"
