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

}  // extern "C"
