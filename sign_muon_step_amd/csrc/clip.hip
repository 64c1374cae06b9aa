// clip.hip -- the 2-norm of each worker's gradients over all weights, and
// clipping by it.
//
//   norm_m = sqrt(sum over all entries g of worker m of g^2)
//   out = g * min(1, most / norm_m)
//
// Bound by memory: the norm reads every gradient once; clipping, which can
// only begin when all of them are known, reads them again and writes them.
//
// Squares are added in fp64: no size of a gradient passes its range, and a sum
// of 10^10 terms keeps fp32's accuracy. A workgroup adds a unit (a run of
// kClipUnit entries of one tensor and worker) and writes one partial sum; the
// partial sums of a worker are added in order by clip_finish_kernel, so a norm
// is the same on every run.
#include "grad_internal.h"

namespace sm {
namespace {

constexpr int kThreads = 256;
constexpr int kVectors = kClipUnit / (kThreads * 8);  // of 8 entries a thread

// A unit's tensor, and what of it the unit covers. The batch lies in scalar
// registers' reach: the index is the workgroup's.
struct Unit {
    int tensor;
    int64_t at, end;  // entries of the worker's part of the tensor
};

__device__ __forceinline__ Unit unit_of(const ClipBatch &b, int unit) {
    int low = 0, high = b.tensors;
    while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (b.first[mid] <= unit)
            low = mid;
        else
            high = mid;
    }
    Unit o;
    o.tensor = low;
    o.at = (int64_t)(unit - b.first[low]) * kClipUnit;
    o.end = o.at + kClipUnit < b.n[low] ? o.at + kClipUnit : b.n[low];
    return o;
}

// Sum over the workgroup, in one order.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double lds[THREADS / kWave];
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) v += lds[w];
    return v;
}

template <bool BF16>
__device__ __forceinline__ double unit_squares(const void *grad, int64_t base, const Unit &u) {
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int64_t at = u.at + (int64_t)(i * kThreads + threadIdx.x) * 8;
        float v[8];
        load_n<BF16>(grad, base + at, left(u.end, at), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) total = fma((double)v[j], (double)v[j], total);
    }
    return total;
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(ClipBatch b) {
    const Unit u = unit_of(b, blockIdx.x);
    const int64_t worker = blockIdx.y, base = worker * b.n[u.tensor];
    const double total = block_sum<kThreads>(b.bf16[u.tensor] ? unit_squares<true>(b.grad[u.tensor], base, u)
                                                              : unit_squares<false>(b.grad[u.tensor], base, u));
    if (threadIdx.x == 0) b.partial[worker * b.units + b.unit0 + blockIdx.x] = total;
}

// A worker's norm and factor.
__global__ __launch_bounds__(1024) void clip_finish_kernel(ClipFinish f) {
    const double *p = f.partial + (int64_t)blockIdx.x * f.units;
    double total = 0.0;
    for (int64_t i = threadIdx.x; i < f.units; i += 1024) total += p[i];
    const double norm = sqrt(block_sum<1024>(total));
    if (threadIdx.x) return;
    f.norms[blockIdx.x] = (float)norm;
    // a norm that is not a number makes every entry of the worker one
    const double factor = (double)f.most / norm;
    f.factors[blockIdx.x] = factor > 1.0 ? 1.0f : (float)factor;
}

template <bool BF16>
__device__ __forceinline__ void scale_unit(const void *grad, void *out, int64_t base, const Unit &u, float factor) {
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int64_t at = u.at + (int64_t)(i * kThreads + threadIdx.x) * 8;
        const int have = left(u.end, at);
        float v[8];
        load_n<BF16>(grad, base + at, have, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= factor;
        store_n<BF16>(out, base + at, have, v);
    }
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipBatch b) {
    const Unit u = unit_of(b, blockIdx.x);
    const int64_t worker = blockIdx.y, base = worker * b.n[u.tensor];
    const float factor = b.factors[worker];
    const void *grad = b.grad[u.tensor];
    void *out = b.out[u.tensor];
    if (factor == 1.0f && out == grad) return;  // in place, and nothing to clip
    if (b.bf16[u.tensor])
        scale_unit<true>(grad, out, base, u, factor);
    else
        scale_unit<false>(grad, out, base, u, factor);
}

}  // namespace

void launch_clip_norm(const ClipBatch &b, hipStream_t s) {
    clip_norm_kernel<<<dim3((unsigned)b.batch_units, (unsigned)b.workers), kThreads, 0, s>>>(b);
}

void launch_clip_finish(const ClipFinish &f, hipStream_t s) {
    clip_finish_kernel<<<dim3((unsigned)f.workers), 1024, 0, s>>>(f);
}

void launch_clip_scale(const ClipBatch &b, hipStream_t s) {
    clip_scale_kernel<<<dim3((unsigned)b.batch_units, (unsigned)b.workers), kThreads, 0, s>>>(b);
}

}  // namespace sm
