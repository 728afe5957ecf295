// k_norm.cu -- the RMS norm between two products, with the residual's
// addition and a BF16 or 8-bit result, and the row quantiser (sm_100a).
//
// For a row of `cols` values, in FP32 throughout:
//   s = x + residual             (residual_out receives s, rounded once)
//   v = s * w / sqrt(mean(s^2) + eps)
//   y = bf16(v)                  and / or
//   scale = max|v| / 127, q = rint(v / scale)
// The norm is taken of the unrounded sum, so y does not depend on the type
// the residual is kept in.  With p = s * w the factor 1/sqrt(..) is common to
// the row: it cancels in q = rint(p * 127 / max|p|), and the sum of squares
// and max|p| are reduced in the same pass.  The quantiser is the same kernel
// without the norm (p = x, factor 1).
//
// A row is read once, held in registers (at most 32 values a thread) and
// written once, so the kernel is bound by memory for many rows and by the
// latency of load, reduction and store for few.  Rows of at most 1024 values
// go one to a warp (shuffles alone), longer ones one to a block.
//
// max|p| is taken over the bit patterns of |p|, in which NaN is above Inf and
// Inf above every finite value: a row that is not finite cannot hide it.  Its
// q are 0 and its scale is NaN, so a product with it is NaN.
#include <algorithm>

#include <cuda_bf16.h>

#include "s12_device.cuh"
#include "s12_launch.h"

namespace s12 {
namespace norm {

constexpr int kVec = 8;         // values a thread loads and stores at a time
constexpr int kMaxVecs = 4;     // vectors a thread holds
constexpr int kMaxThreads = 1024;
constexpr int kWarpRows = 4;    // rows of a block when each has a warp
static_assert(S12_NORM_MAX_COLS == kVec * kMaxVecs * kMaxThreads, "the longest row fills one block");

struct Args {
    const void *x;
    const void *res;
    void *res_out;
    const uint16_t *w;
    uint16_t *y;
    int8_t *q;
    float *scale;
    long long rows;
    int cols;
    float eps;
    int x_f32, res_f32;
};

__device__ __forceinline__ void unpack(const uint4 &a, float (&v)[kVec]) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&v)[kVec]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The vectors at columns 8 * (t + i * n) of a row, zeros past its end.
template <int NV>
__device__ __forceinline__ void load_row(const void *base, size_t row0, int cols, bool f32, int t, int n,
                                         float (&v)[NV][kVec]) {
    if (f32) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + row0);
        float4 a[NV][2];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * n;
            a[i][0] = a[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c * kVec < cols) {
                a[i][0] = src[2 * c];
                a[i][1] = src[2 * c + 1];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[i][4 * h] = a[i][h].x;
                v[i][4 * h + 1] = a[i][h].y;
                v[i][4 * h + 2] = a[i][h].z;
                v[i][4 * h + 3] = a[i][h].w;
            }
    } else {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + row0);
        uint4 a[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * n;
            a[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c * kVec < cols) a[i] = src[c];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) unpack(a[i], v[i]);
    }
}

// Four values to 8 bits, the nearest integers.
__device__ __forceinline__ uint32_t to_eight(float a, float b, float c, float d) {
    uint32_t lo, v;
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(lo) : "r"(__float2int_rn(d)), "r"(__float2int_rn(c)), "r"(0));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(__float2int_rn(b)), "r"(__float2int_rn(a)), "r"(lo));
    return v;
}

// s * weight.
template <int NV>
__device__ __forceinline__ void weigh(const Args &a, int t, int n, float (&s)[NV][kVec]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * n;
        if (a.w && c * kVec < a.cols) {
            float w[kVec];
            unpack(reinterpret_cast<const uint4 *>(a.w)[c], w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) s[i][k] *= w[k];
        }
    }
}

template <int NV>
__device__ __forceinline__ uint32_t largest(const float (&s)[NV][kVec]) {
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < kVec; ++k) top = max(top, __float_as_uint(s[i][k]) & 0x7FFFFFFFu);
    return top;
}

template <int NV>
__device__ __forceinline__ float squares(const float (&s)[NV][kVec]) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < kVec; ++k) ss = fmaf(s[i][k], s[i][k], ss);
    return ss;
}

// The sum of a row whose squares leave FP32's range, and its products with the
// weights: the row times 2^-by, which is exact, has its largest value or the root
// of eps near 1.  `part`: the thread's values s where it `keeps` them, else its p;
// it becomes p * 2^-by, f the factor and top the largest that go with it.  A row
// of zeros or one that is not finite is left as it is (false).  A function of its
// own, on local memory: in the row's registers it took 5 % of all rows' time, so
// it takes 3 (4096 rows of 8192: 40.2 us without it, 41.4 with it, 42.3 inline;
// one row of 4096 2.16, 2.20 and 2.16).
template <class Reduce>
__device__ __noinline__ bool rescale(float *part, int vecs, bool keeps, float mine, const uint16_t *w, int cols,
                                     float eps, int t, int n, float &f, uint32_t &top, Reduce reduce) {
    uint32_t big = __float_as_uint(__fsqrt_rn(mine));
    if (keeps) {
        big = 0u;
        for (int i = 0; i < vecs * kVec; ++i) big = max(big, __float_as_uint(part[i]) & 0x7FFFFFFFu);
    }
    float ss = 0.f;
    reduce(ss, big, 1);
    if (big == 0u || big >= 0x7F800000u) return false;
    const int by = max(ilogbf(__uint_as_float(big)), eps > 0.f ? ilogbf(eps) / 2 : -149);
    ss = keeps ? 0.f : scalbnf(mine, -2 * by);
    top = 0u;
    for (int i = 0; i < vecs * kVec; ++i) {
        float v = scalbnf(part[i], -by);
        if (keeps) {
            const int c = (t + i / kVec * n) * kVec + i % kVec;
            ss = fmaf(v, v, ss);
            if (w && c < cols) v *= __uint_as_float(static_cast<uint32_t>(w[c]) << 16);
        }
        part[i] = v;
        top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
    }
    reduce(ss, top, 2);
    f = __frsqrt_rn(ss / static_cast<float>(cols) + scalbnf(eps, -2 * by));
    return true;
}

// A mean square (with eps) below this is not taken from FP32's squares: above it
// what they lose (2^-150 each) is far below the sum's rounding, and p * f is
// within 2^-130 of v where p is subnormal.
constexpr float kLeast = 0x1p-40f, kMost = 3.4028234e38f;

// One row by n threads (t = 0 .. n-1), `reduce` summing ss and taking the
// largest top over them (its last argument: how often it was called before).
// PLAIN: the quantiser (x to q and scale, nothing else), which needs fewer
// registers.
template <int NV, bool PLAIN, class Reduce>
__device__ __forceinline__ void do_row(const Args &a, long long row, int t, int n, Reduce reduce) {
    const size_t row0 = static_cast<size_t>(row) * static_cast<size_t>(a.cols);
    float s[NV][kVec];
    load_row<NV>(a.x, row0, a.cols, a.x_f32 != 0, t, n, s);
    if (!PLAIN && a.res) {
        float r[NV][kVec];
        load_row<NV>(a.res, row0, a.cols, a.res_f32 != 0, t, n, r);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < kVec; ++k) s[i][k] += r[i][k];
    }
    if (!PLAIN && a.res_out) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * n;
            if (c * kVec < a.cols) {
                if (a.res_f32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.res_out) + row0) + 2 * c;
                    dst[0] = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
                    dst[1] = make_float4(s[i][4], s[i][5], s[i][6], s[i][7]);
                } else {
                    reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.res_out) + row0)[c] = pack(s[i]);
                }
            }
        }
    }
    const float mine = PLAIN ? 0.f : squares(s);
    // A thread keeps its part of a row whose squares may leave FP32's range, before
    // it is multiplied.  No thread's sum is more than the row's, so where the row's
    // mean is below kLeast all of them have kept theirs.
    float part[NV * kVec];
    const bool keeps = !PLAIN && !(mine >= (a.eps < kLeast ? kLeast * S12_NORM_MAX_COLS : 0.f) && mine <= kMost);
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < NV * kVec; ++i) part[i] = s[i / kVec][i % kVec];
    };
    if (keeps) put();
    if (!PLAIN) weigh(a, t, n, s);
    float ss = mine;
    uint32_t top = largest(s);
    reduce(ss, top, 0);
    // (a row of zeros with eps = 0 stays a row of zeros)
    const float ms = ss / static_cast<float>(a.cols) + a.eps;
    float f = PLAIN ? 1.f : ms == 0.f ? 0.f : __frsqrt_rn(ms);
    if (!PLAIN && !(ms >= kLeast && ms <= kMost)) {
        if (!keeps) put();
        if (rescale(part, NV, keeps, mine, a.w, a.cols, a.eps, t, n, f, top, reduce)) {
#pragma unroll
            for (int i = 0; i < NV * kVec; ++i) s[i / kVec][i % kVec] = part[i];
        }
    }
    if (!PLAIN && a.y) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * n;
            if (c * kVec < a.cols) {
                float v[kVec];
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[k] = s[i][k] * f;
                reinterpret_cast<uint4 *>(a.y + row0)[c] = pack(v);
            }
        }
    }
    if (PLAIN || a.q) {
        const bool finite = top < 0x7F800000u;
        // 127 / max|p| overflows for the smallest maxima: those rows are
        // scaled up by 2^64 first (exact: their values are that small)
        const float m = __uint_as_float(top);
        float g = finite && top ? 127.f / m : 0.f;
        if (top < 0x0D000000u) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < kVec; ++k) s[i][k] *= 18446744073709551616.f;
            g = top ? 127.f / (m * 18446744073709551616.f) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * n;
            if (c * kVec < a.cols) {
                float v[kVec];
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[k] = finite ? s[i][k] * g : 0.f;
                reinterpret_cast<uint2 *>(a.q + row0)[c] =
                    make_uint2(to_eight(v[0], v[1], v[2], v[3]), to_eight(v[4], v[5], v[6], v[7]));
            }
        }
        if (t == 0) a.scale[row] = finite ? m * f / 127.f : __uint_as_float(0x7FC00000u);
    }
}

__device__ __forceinline__ void warp_reduce(float &ss, uint32_t &top) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
}

// One row to a warp.
template <int NV, bool PLAIN>
__global__ void __launch_bounds__(32 * kWarpRows) warp_kernel(const Args a) {
    grid_launch_dependents();
    const long long row = static_cast<long long>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5);
    if (row >= a.rows) return;
    grid_dependency_wait();
    do_row<NV, PLAIN>(a, row, threadIdx.x & 31, 32, [](float &ss, uint32_t &top, int) { warp_reduce(ss, top); });
}

// One row to a block of at most THREADS threads, BLOCKS of them on an SM.
template <int NV, bool PLAIN, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) block_kernel(const Args a) {
    __shared__ float part[3][32];
    __shared__ uint32_t tops[3][32];
    grid_launch_dependents();
    grid_dependency_wait();
    do_row<NV, PLAIN>(a, blockIdx.x, threadIdx.x, blockDim.x, [&](float &ss, uint32_t &top, int at) {
        warp_reduce(ss, top);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
            part[at][warp] = ss;
            tops[at][warp] = top;
        }
        __syncthreads();
        ss = lane < warps ? part[at][lane] : 0.f;
        top = lane < warps ? tops[at][lane] : 0u;
        warp_reduce(ss, top);
    });
}

}  // namespace norm

namespace {

template <class Kernel>
int launch_rows(Kernel kern, unsigned grid, unsigned threads, const norm::Args &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? S12_OK : S12_ERR_CUDA;
}

template <bool PLAIN>
int launch_kind(const norm::Args &a, int sms, cudaStream_t stream) {
    using namespace norm;
    const int vecs = a.cols / kVec;
    if (a.cols <= 32 * kVec * kMaxVecs) {
        const int nv = (vecs + 31) / 32;
        const unsigned grid = static_cast<unsigned>((a.rows + kWarpRows - 1) / kWarpRows);
        if (nv == 1) return launch_rows(warp_kernel<1, PLAIN>, grid, 32 * kWarpRows, a, stream);
        if (nv == 2) return launch_rows(warp_kernel<2, PLAIN>, grid, 32 * kWarpRows, a, stream);
        return launch_rows(warp_kernel<4, PLAIN>, grid, 32 * kWarpRows, a, stream);
    }
    // Few rows: as many threads as vectors, so that each loads once (one row of
    // 4096: 2.2 us).  Many rows: four vectors a thread, so that more rows share
    // an SM (4096 rows of 8192, norm and quantiser: 45 and 24 us, against 49
    // and 28 with two and 62 and 41 with one).
    const unsigned grid = static_cast<unsigned>(a.rows);
    const bool few = a.rows <= 2 * sms;
    const int nv = few && vecs <= kMaxThreads ? 1 : few && vecs <= 2 * kMaxThreads ? 2 : 4;
    const unsigned threads = static_cast<unsigned>(((vecs + nv - 1) / nv + 31) / 32 * 32);
    if (nv == 1) return launch_rows(block_kernel<1, PLAIN, kMaxThreads, 1>, grid, threads, a, stream);
    if (nv == 2) return launch_rows(block_kernel<2, PLAIN, kMaxThreads, 1>, grid, threads, a, stream);
    if (threads <= 256) return launch_rows(block_kernel<4, PLAIN, 256, PLAIN ? 6 : 4>, grid, threads, a, stream);
    return launch_rows(block_kernel<4, PLAIN, kMaxThreads, 1>, grid, threads, a, stream);
}

}  // namespace

int launch_norm(const NormCall &c, cudaStream_t stream) {
    norm::Args a = {};
    a.x = c.x;
    a.res = c.residual;
    a.res_out = c.residual_out;
    a.w = c.weight;
    a.y = c.y;
    a.q = c.q;
    a.scale = c.scale;
    a.rows = c.rows;
    a.cols = static_cast<int>(c.cols);
    a.eps = c.eps;
    a.x_f32 = c.x_type == S12_TYPE_F32;
    a.res_f32 = c.residual_type == S12_TYPE_F32;
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return S12_ERR_CUDA;
    return c.normed ? launch_kind<false>(a, sms, stream) : launch_kind<true>(a, sms, stream);
}

}  // namespace s12
