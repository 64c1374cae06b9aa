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
// entries of one tensor and worker) and writes one partial sum; the partial
// sums of a worker are added in order, so a norm is the same on every run. Units
// are of 16384 entries, or of 2048 where that leaves compute units without one.
// Few partial sums are added by every workgroup that needs the factor, many by
// clip_finish_kernel. Measured: 629 M entries of FP32 read twice and written once 1.38 ms
// (5.5 TB/s: the norm reads at 5.7, the scaling goes through the tensors backwards and finds the
// last ones in the caches); 51 tensors of eight workers 69 to 86 us; one of 256 x 256 and four workers 9 us, most
// of it issuing two launches.
#include "grad_internal.h"

namespace sm {
namespace {

constexpr int kThreads = 256;

// A unit's tensor, and what of it the unit covers. The batch lies in scalar
// registers' reach: the index is the workgroup's.
struct Unit {
    int tensor;
    int64_t at, end;  // entries of the worker's part of the tensor
};

template <int UNIT>
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
    o.at = (int64_t)(unit - b.first[low]) * UNIT;
    o.end = o.at + UNIT < b.n[low] ? o.at + UNIT : b.n[low];
    return o;
}

// Eight entries as they lie in memory.
template <bool BF16>
__device__ __forceinline__ Raw<BF16, 8> fetch(const void *p, int64_t at) {
    Raw<BF16, 8> o;
    const char *q = static_cast<const char *>(p) + at * (BF16 ? 2 : 4);
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
        const u32x4 t = *reinterpret_cast<const u32x4_any *>(q + 16 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[4 * h + j] = t[j];
    }
    return o;
}
template <bool BF16>
__device__ __forceinline__ void open(const Raw<BF16, 8> &o, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __uint_as_float(BF16 ? (j % 2 ? o.w[j / 2] & 0xffff0000u : o.w[j / 2] << 16) : o.w[BF16 ? 0 : j]);
}

// use(entry, v) for each eight of a thread's entries of a unit, all loads of a whole
// unit before the first is used; have: how many of the eight exist.
template <bool BF16, int UNIT, class F>
__device__ __forceinline__ void each(const void *grad, int64_t base, const Unit &u, F &&use) {
    constexpr int kVectors = UNIT / (kThreads * 8);
    if (u.end - u.at == UNIT) {
        Raw<BF16, 8> raw[kVectors];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) raw[i] = fetch<BF16>(grad, base + u.at + (i * kThreads + threadIdx.x) * 8);
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            float v[8];
            open<BF16>(raw[i], v);
            use(u.at + (i * kThreads + threadIdx.x) * 8, 8, v);
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < kVectors; ++i) {
        const int64_t at = u.at + (i * kThreads + threadIdx.x) * 8;
        const int have = left(u.end, at);
        float v[8];
        load_n<BF16>(grad, base + at, have, v);
        use(at, have, v);
    }
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

template <bool BF16, int UNIT>
__device__ __forceinline__ double unit_squares(const void *grad, int64_t base, const Unit &u) {
    double total = 0.0;
    each<BF16, UNIT>(grad, base, u, [&](int64_t, int, const float(&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) total = fma((double)v[j], (double)v[j], total);
    });
    return total;
}

template <int UNIT>
__global__ __launch_bounds__(kThreads) void clip_norm_kernel(ClipBatch b) {
    const Unit u = unit_of<UNIT>(b, blockIdx.x);
    const int64_t worker = blockIdx.y, base = worker * b.n[u.tensor];
    const double total = block_sum<kThreads>(b.bf16[u.tensor] ? unit_squares<true, UNIT>(b.grad[u.tensor], base, u)
                                                              : unit_squares<false, UNIT>(b.grad[u.tensor], base, u));
    if (threadIdx.x == 0) b.partial[worker * b.units + b.unit0 + blockIdx.x] = total;
}

// A worker's norm, in all threads.
template <int THREADS>
__device__ __forceinline__ double worker_norm(const double *partial, int64_t units) {
    double total = 0.0;
    for (int64_t i = threadIdx.x; i < units; i += THREADS) total += partial[i];
    return sqrt(block_sum<THREADS>(total));
}

// A norm that is not a number leaves the worker no entry that is one.
__device__ __forceinline__ float factor_of(float most, double norm) {
    const double factor = (double)most / norm;
    return factor > 1.0 ? 1.0f : (float)factor;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void clip_finish_kernel(ClipFinish f) {
    const double norm = worker_norm<THREADS>(f.partial + (int64_t)blockIdx.x * f.units, f.units);
    if (threadIdx.x) return;
    f.norms[blockIdx.x] = (float)norm;
    f.factors[blockIdx.x] = factor_of(f.most, norm);
}

// v times the factor, for a store in the type that is to be the product's one rounding.
// A BF16 value's product has up to 32 bits. Rounded to fp32 and then to 8 bits it comes out as
// if rounded once, unless fp32's value is the middle of two BF16 ones and the product is not
// (one in 2^17): such a value takes one step of fp32 towards the product, which fp64 holds.
// (51 tensors of BF16: 67.5 us so, 68.7 with every product made in fp64 and cut.)
template <bool BF16>
__device__ __forceinline__ void scale8(float (&v)[8], float factor) {
    float out[8];
    bool middle = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        out[j] = v[j] * factor;
        middle |= BF16 && (__float_as_uint(out[j]) & 0xffffu) == 0x8000u;
    }
    if (middle)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t bits = __float_as_uint(out[j]);
            const double left = (double)v[j] * (double)factor - (double)out[j];
            if ((bits & 0xffffu) == 0x8000u && left != 0.0)
                out[j] = __uint_as_float((left < 0.0) == (out[j] < 0.0) ? bits + 1 : bits - 1);
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = out[j];
}

template <bool BF16, int UNIT>
__device__ __forceinline__ void scale_unit(const void *grad, void *out, int64_t base, const Unit &u, float factor) {
    each<BF16, UNIT>(grad, base, u, [&](int64_t at, int have, float(&v)[8]) {
        scale8<BF16>(v, factor);
        store_n<BF16>(out, base + at, have, v);
    });
}

// The units from the last one back: what the norm read last may still be in the caches.
// FEW: the factor is made here.
template <int UNIT, bool FEW>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipBatch b) {
    const Unit u = unit_of<UNIT>(b, b.batch_units - 1 - blockIdx.x);
    const int64_t worker = b.workers - 1 - blockIdx.y, base = worker * b.n[u.tensor];
    float factor;
    if constexpr (FEW) {
        const double norm = worker_norm<kThreads>(b.partial + worker * b.units, b.units);
        factor = factor_of(b.most, norm);
        if (blockIdx.x == 0 && b.unit0 == 0 && threadIdx.x == 0) b.norms[worker] = (float)norm;
    } else {
        factor = b.factors[worker];
    }
    const void *grad = b.grad[u.tensor];
    void *out = b.out[u.tensor];
    if (factor == 1.0f && out == grad) return;  // in place, and nothing to clip
    if (b.bf16[u.tensor])
        scale_unit<true, UNIT>(grad, out, base, u, factor);
    else
        scale_unit<false, UNIT>(grad, out, base, u, factor);
}

template <int UNIT>
void launch_scale(const ClipBatch &b, hipStream_t s) {
    const dim3 grid((unsigned)b.batch_units, (unsigned)b.workers);
    if (b.units <= kClipFew)
        clip_scale_kernel<UNIT, true><<<grid, kThreads, 0, s>>>(b);
    else
        clip_scale_kernel<UNIT, false><<<grid, kThreads, 0, s>>>(b);
}

}  // namespace

void launch_clip_norm(const ClipBatch &b, hipStream_t s) {
    const dim3 grid((unsigned)b.batch_units, (unsigned)b.workers);
    if (b.unit == kClipUnit)
        clip_norm_kernel<kClipUnit><<<grid, kThreads, 0, s>>>(b);
    else
        clip_norm_kernel<kClipSmallUnit><<<grid, kThreads, 0, s>>>(b);
}

void launch_clip_finish(const ClipFinish &f, hipStream_t s) {
    if (f.units <= kClipFew)
        clip_finish_kernel<kThreads><<<dim3((unsigned)f.workers), kThreads, 0, s>>>(f);
    else
        clip_finish_kernel<1024><<<dim3((unsigned)f.workers), 1024, 0, s>>>(f);
}

void launch_clip_scale(const ClipBatch &b, hipStream_t s) {
    b.unit == kClipUnit ? launch_scale<kClipUnit>(b, s) : launch_scale<kClipSmallUnit>(b, s);
}

}  // namespace sm
