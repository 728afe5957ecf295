// k_gemm_i8.cu -- 8-bit integer product with a scale for each token and each
// output channel, on the tcgen05 tensor cores (sm_100a):
//
//   y[m][n] = x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k]
//
// x: M x K int8, w: N x K int8, sums in int32 (exact for K < 2^17), y BF16 or
// FP32, rounded once.  Computed as Y^T = W * X^T, as the fused GEMM: 128 rows
// of W are the tensor core's M and up to 256 tokens its N, so one kernel
// serves a single token (N = 16: bound by reading W) and prompts (bound by
// the tensor cores).
//
// One CTA per SM, six warps with fixed roles: a TMA producer (128 columns of W
// and X a stage, 128-byte swizzle), the MMA issuer (four tcgen05.mma.kind::i8
// of K = 32 a stage), and four epilogue warps that read the accumulators from
// TMEM, scale and store them.  There are two accumulators, so that the next
// tile is multiplied while one is stored.
//
// Work split.  As many whole waves of tiles as there are go one tile to a CTA,
// neighbours at the same time (they share rows of W or X in L2); the columns
// of the tiles that are left are dealt to all CTAs in equal ranges.  A tile
// that several CTAs share is finished by the last of them to arrive, which
// adds the parts.  Integer sums do not depend on their order.
#include <algorithm>

#include <cuda_bf16.h>

#include "s12_device.cuh"
#include "s12_launch.h"
#include "s12_tc.cuh"

namespace s12 {
namespace gemm8 {

using namespace tc;

constexpr int kRows = 128;    // rows of W per tile (UMMA M)
constexpr int kChunk = 128;   // columns per stage: one swizzle atom
constexpr int kMaxTokens = 256;
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kWBytes = kRows * kChunk;

struct __align__(64) Params {
    CUtensorMap tm_w;  // u8 [N][K], box 128 x 128, 128-byte swizzle, zeros past the ends
    CUtensorMap tm_x;  // u8 [M][K], box 128 x tokens
    const float *x_scale, *w_scale;
    void *y;
    int y_f32;
    long long M, N;
    int tokens;              // per tile, a multiple of 16
    int chunks;              // stages per tile
    int tiles_m, waves;      // token tiles; whole waves of tiles
    long long tile0, units;  // first tile after the whole waves, and the stages from there on
    uint32_t *cnt;           // workspace: one arrival counter per CTA (zero between calls)
    uint32_t *err;
    int32_t *part;           // workspace: [CTAs][2][tokens][kRows] parts
    int stages;
    uint32_t stage_bytes, acc_cols, tmem_cols;
};

// D[tmem] (+)= A[smem] * B[smem] for one 128 x N x 32 step, int8 -> int32.
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: int8 x int8 -> int32, both operands K-major, M =
// 128, N = n.
__device__ __forceinline__ uint32_t instr_desc(int n) {
    return (2u << 4)                                  // D format int32
           | (1u << 7)                                // A format signed
           | (1u << 10)                               // B format signed
           | (static_cast<uint32_t>(n >> 3) << 17)    // N / 8
           | (static_cast<uint32_t>(kRows >> 4) << 24);  // M / 16
}

// The stretches of work of one CTA, in order: whole tiles, then its range of
// the rest.  [k0, k1): the stages of the tile.
struct Work {
    long long tile;
    int k0, k1;
};

__device__ __forceinline__ long long range_start(const Params &p, long long c) { return c * p.units / gridDim.x; }

struct Walk {
    int wave;
    long long u, u1;  // position in the rest

    __device__ __forceinline__ explicit Walk(const Params &p)
        : wave(0), u(range_start(p, blockIdx.x)), u1(range_start(p, blockIdx.x + 1)) {}

    __device__ __forceinline__ bool next(const Params &p, Work &w) {
        if (wave < p.waves) {
            w.tile = static_cast<long long>(wave) * gridDim.x + blockIdx.x;
            w.k0 = 0;
            w.k1 = p.chunks;
            ++wave;
            return true;
        }
        if (u >= u1) return false;
        const long long t = u / p.chunks, t0 = t * p.chunks;
        w.tile = p.tile0 + t;
        w.k0 = static_cast<int>(u - t0);
        w.k1 = static_cast<int>(min(static_cast<long long>(p.chunks), u1 - t0));
        u = t0 + w.k1;
        return true;
    }
};

// CTAs [first, last] that share tile t of the rest.
__device__ __forceinline__ void sharers(const Params &p, long long t, int &first, int &last) {
    const long long t0 = t * p.chunks, t1 = t0 + p.chunks;
    int c = blockIdx.x;
    while (c > 0 && range_start(p, c) > t0) --c;
    first = c;
    c = blockIdx.x;
    while (c + 1 < static_cast<int>(gridDim.x) && range_start(p, c + 1) < t1) ++c;
    last = c;
}

// Arrive on a shared tile's counter, the one of its first CTA (a CTA is the
// first of one shared tile at most); true for the last arrival, which also
// sets it back to zero.
__device__ __forceinline__ bool arrive(const Params &p, int first, int last) {
    uint32_t want = 0;
    for (int c = first; c <= last; ++c) want += range_start(p, c) < range_start(p, c + 1) ? 1u : 0u;
    if (atomicAdd(p.cnt + first, 1u) + 1 != want) return false;
    atomicExch(p.cnt + first, 0u);
    return true;
}

// A wait gave up: the caller's word says so, and the CTA unwinds.
__device__ __forceinline__ void give_up(const Params &p, uint32_t abort_word) {
    raise_flag(p.err, S12_FLAG_TIMEOUT);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(abort_word), "r"(1u) : "memory");
}

struct Layout {
    uint32_t full, empty, acc_full, acc_empty, done;  // mbarriers
    uint32_t tmem_slot, last, abort, shared_done;     // 4-byte words
    uint32_t stages;
};

__device__ __forceinline__ Layout layout(uint32_t sb) {
    Layout L;
    L.full = sb;
    L.empty = sb + 8 * kMaxStages;
    L.acc_full = sb + 16 * kMaxStages;
    L.acc_empty = L.acc_full + 16;
    L.done = L.acc_empty + 16;
    L.tmem_slot = L.done + 8;
    L.last = L.tmem_slot + 4;
    L.abort = L.last + 4;        // a wait of this CTA gave up
    L.shared_done = L.abort + 4; // shared tiles whose counter this CTA has arrived on
    L.stages = sb + 1024;
    return L;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void put_y(const Params &p, long long m, long long n, float v) {
    const size_t o = static_cast<size_t>(m) * static_cast<size_t>(p.N) + static_cast<size_t>(n);
    if (p.y_f32)
        static_cast<float *>(p.y)[o] = v;
    else
        static_cast<uint16_t *>(p.y)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// 32 TMEM lanes x 16 consecutive columns into 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// The accumulators at `tmem` (this CTA's part [k0, k1) of tile w.tile): y, or
// a part and, for the tile's last arrival, y from all parts.  Lane i of TMEM
// is row i of the tile, a warp reads the 32 lanes of its quadrant.
__device__ __forceinline__ void epilogue(const Params &p, const Layout &L, const Work &w, uint32_t tmem, int quad,
                                         int lane, uint32_t bar_empty) {
    const int row = quad * 32 + lane;
    const long long n = w.tile / p.tiles_m * kRows + row, m0 = w.tile % p.tiles_m * p.tokens;
    const bool whole = w.k0 == 0 && w.k1 == p.chunks;
    const bool first_thread = quad == 0 && lane == 0;
    const float sw = n < p.N ? __ldg(p.w_scale + n) : 0.f;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // the CTA's range starts in this tile (slot 0) or reaches into it (1)
    int32_t *mine = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (w.k0 > 0 ? 0 : 1)) * p.tokens * kRows;
    for (int c = 0; c < p.tokens; c += 16) {
        uint32_t v[16];
        tmem_ld16(taddr + static_cast<uint32_t>(c), v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const long long m = m0 + c + i;
            if (!whole)
                __stcg(mine + static_cast<size_t>(c + i) * kRows + row, static_cast<int32_t>(v[i]));
            else if (m < p.M && n < p.N)
                put_y(p, m, n, static_cast<float>(static_cast<int32_t>(v[i])) * __ldg(p.x_scale + m) * sw);
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(bar_empty);
    if (whole) return;
    __threadfence();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
    int first, last;
    sharers(p, w.tile - p.tile0, first, last);
    if (first_thread) {
        sts32(L.last, arrive(p, first, last) ? 1u : 0u);
        sts32(L.shared_done, lds32(L.shared_done) + 1);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
    if (!lds32(L.last)) return;
    __threadfence();
    const long long t0 = (w.tile - p.tile0) * p.chunks;
    for (int c = 0; c < p.tokens; ++c) {
        const long long m = m0 + c;
        if (m >= p.M) break;
        int32_t s = 0;
        for (int v = first; v <= last; ++v) {
            const long long vs = range_start(p, v);
            if (vs < range_start(p, v + 1))
                s += __ldcg(p.part + (static_cast<size_t>(v) * 2 + (vs > t0 ? 0 : 1)) * p.tokens * kRows +
                            static_cast<size_t>(c) * kRows + row);
        }
        if (n < p.N) put_y(p, m, n, static_cast<float>(s) * __ldg(p.x_scale + m) * sw);
    }
}

__global__ void __launch_bounds__(kThreads, 1) gemm_i8_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sb = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const Layout L = layout(sb);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.stages;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            bar_init(L.full + 8 * s, 1);
            bar_init(L.empty + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            bar_init(L.acc_full + 8 * a, 1);
            bar_init(L.acc_empty + 8 * a, kEpiWarps);
        }
        bar_init(L.done, 1);
        sts32(L.abort, 0u);
        sts32(L.shared_done, 0u);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(L.tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds32(L.tmem_slot);
    grid_launch_dependents();
    grid_dependency_wait();  // x, w, y and the workspace may belong to earlier kernels
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            int s = 0;
            uint32_t round = 0;
            long long issued = 0;
            bool ok = true;
            Walk walk(p);
            for (Work w; ok && walk.next(p, w);) {
                const int n0 = static_cast<int>(w.tile / p.tiles_m) * kRows;
                const int m0 = static_cast<int>(w.tile % p.tiles_m) * p.tokens;
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!bar_wait(L.empty + 8 * s, (round & 1u) ^ 1u)) {
                        give_up(p, L.abort);
                        ok = false;
                        break;
                    }
                    const uint32_t st = L.stages + static_cast<uint32_t>(s) * p.stage_bytes;
                    bar_expect_tx(L.full + 8 * s, p.stage_bytes);
                    tma2d(st, &p.tm_w, k * kChunk, n0, L.full + 8 * s, pol);
                    tma2d(st + kWBytes, &p.tm_x, k * kChunk, m0, L.full + 8 * s, pol);
                    ++issued;
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // every copy lands before the CTA leaves
            for (long long i = issued > S ? issued - S : 0; i < issued; ++i)
                bar_wait(L.full + 8 * static_cast<uint32_t>(i % S), static_cast<uint32_t>((i / S) & 1));
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = instr_desc(p.tokens);
            int s = 0;
            uint32_t round = 0, tile = 0;
            bool ok = true;
            Walk walk(p);
            for (Work w; ok && walk.next(p, w); ++tile) {
                const uint32_t a = tile & 1u;
                ok = bar_wait(L.acc_empty + 8 * a, ((tile >> 1) & 1u) ^ 1u);
                for (int k = w.k0; ok && k < w.k1; ++k) {
                    if (!(ok = bar_wait(L.full + 8 * s, round & 1u))) break;
                    tc_fence_after();
                    const uint32_t st = L.stages + static_cast<uint32_t>(s) * p.stage_bytes;
#pragma unroll
                    for (int kk = 0; kk < kChunk / 32; ++kk)
                        umma_i8(tmem + a * p.acc_cols, smem_desc_sw128(st + 32u * kk),
                                smem_desc_sw128(st + kWBytes + 32u * kk), idesc, k > w.k0 || kk > 0);
                    umma_commit(L.empty + 8 * s);
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                }
                if (ok) umma_commit(L.acc_full + 8 * a);
            }
            if (!ok) give_up(p, L.abort);
            // every product issued has completed before TMEM is freed
            umma_commit(L.done);
            bar_wait(L.done, 0);
        }
    } else {
        const int quad = warp & 3;  // the TMEM lanes that this warp may read
        uint32_t tile = 0;
        Walk walk(p);
        for (Work w; walk.next(p, w); ++tile) {
            const uint32_t a = tile & 1u;
            const bool ok = bar_wait(L.acc_full + 8 * a, (tile >> 1) & 1u);
            // (all epilogue warps go on, or none)
            uint32_t all;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 p, %1, 0;\n\t"
                "barrier.red.and.pred q, 1, %2, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(all)
                : "r"(ok ? 1u : 0u), "n"(32 * kEpiWarps)
                : "memory");
            if (!all) {
                if (lane == 0) give_up(p, L.abort);
                break;
            }
            tc_fence_after();
            epilogue(p, L, w, tmem + a * p.acc_cols, quad, lane, L.acc_empty + 8 * a);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
    if (threadIdx.x == 0 && lds32(L.abort)) {
        // the shared tiles that this CTA did not get to still see its
        // arrival, so that their counters return to zero
        const uint32_t done = lds32(L.shared_done);
        uint32_t k = 0;
        Walk walk(p);
        walk.wave = p.waves;
        for (Work w; walk.next(p, w);) {
            if (w.k0 == 0 && w.k1 == p.chunks) continue;
            if (k++ < done) continue;
            int first, last;
            sharers(p, w.tile - p.tile0, first, last);
            arrive(p, first, last);
        }
    }
}

}  // namespace gemm8

// ---------------------------------------------------------------------------
// Host side.

namespace {

constexpr uint32_t kSmemLimit = 227 * 1024;

struct Plan8 {
    int tokens, tiles_m;
    size_t cnt_bytes, part_bytes;
};

Plan8 plan8(int64_t M, int sms) {
    Plan8 pl;
    // token tiles of equal size, as few as 256 rows allow
    const int64_t tiles = (M + gemm8::kMaxTokens - 1) / gemm8::kMaxTokens;
    pl.tiles_m = static_cast<int>(tiles);
    pl.tokens = static_cast<int>(((M + tiles - 1) / tiles + 15) / 16 * 16);
    // the counters first and their size by the device alone: calls of other
    // shapes may use the workspace in turn
    pl.cnt_bytes = align_up(static_cast<uint64_t>(sms) * 4, kAlign);
    pl.part_bytes = static_cast<size_t>(sms) * 2 * pl.tokens * gemm8::kRows * 4;
    return pl;
}

}  // namespace

size_t gemm_i8_ws_bytes(int64_t M) {
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return 0;
    const Plan8 pl = plan8(M, sms);
    return pl.cnt_bytes + pl.part_bytes;
}

int launch_gemm_i8(const Gemm8Call &c, void *ws, size_t ws_bytes, cudaStream_t stream) {
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return S12_ERR_CUDA;
    const Plan8 pl = plan8(c.M, sms);
    if (ws_bytes < pl.cnt_bytes + pl.part_bytes) return S12_ERR_CAPACITY;
    gemm8::Params p = {};
    if (make_tmap_u8_2d(&p.tm_w, c.w, c.K, c.N, c.K, gemm8::kChunk, gemm8::kRows, 128) != S12_OK ||
        make_tmap_u8_2d(&p.tm_x, c.x, c.K, c.M, c.K, gemm8::kChunk, pl.tokens, 128) != S12_OK)
        return S12_ERR_CUDA;
    p.x_scale = c.x_scale;
    p.w_scale = c.w_scale;
    p.y = c.y;
    p.err = c.err;
    p.y_f32 = c.y_type == S12_TYPE_F32;
    p.M = c.M;
    p.N = c.N;
    p.tokens = pl.tokens;
    p.chunks = static_cast<int>((c.K + gemm8::kChunk - 1) / gemm8::kChunk);
    p.tiles_m = pl.tiles_m;
    const long long tiles = (c.N + gemm8::kRows - 1) / gemm8::kRows * pl.tiles_m;
    const int grid = static_cast<int>(std::min<long long>(sms, tiles * p.chunks));
    p.waves = static_cast<int>(tiles / grid);
    p.tile0 = static_cast<long long>(p.waves) * grid;
    p.units = (tiles - p.tile0) * p.chunks;
    p.cnt = static_cast<uint32_t *>(ws);
    p.part = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + pl.cnt_bytes);
    p.stage_bytes = gemm8::kWBytes + static_cast<uint32_t>(pl.tokens) * gemm8::kChunk;
    p.stages = static_cast<int>(std::min<uint32_t>(gemm8::kMaxStages, (kSmemLimit - 2048) / p.stage_bytes));
    p.acc_cols = 32;
    while (p.acc_cols < static_cast<uint32_t>(pl.tokens)) p.acc_cols <<= 1;
    p.tmem_cols = 2 * p.acc_cols;
    const uint32_t smem = 2048 + static_cast<uint32_t>(p.stages) * p.stage_bytes;
    if (cudaFuncSetAttribute(gemm8::gemm_i8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return S12_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(gemm8::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemm8::gemm_i8_kernel, p) == cudaSuccess ? S12_OK : S12_ERR_CUDA;
}

}  // namespace s12
