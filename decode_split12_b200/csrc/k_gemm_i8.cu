// k_gemm_i8.cu -- 8-bit integer product with a scale for each token and each
// output channel, on the tcgen05 tensor cores (sm_100a):
//
//   y[m][n] = x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k]
//
// x: M x K int8, w: N x K int8, sums in int32 (exact for K < 2^17), y BF16 or
// FP32, rounded once.  Computed as Y^T = W * X^T, as the fused GEMM: rows of W
// are the tensor core's M and up to 256 tokens its N.  A few tokens (eight, and
// little work) take a kernel of dot products, further down.
//
// One CTA per SM, ten warps with fixed roles: a TMA producer (128 columns of W
// and X a stage, 128-byte swizzle), the MMA issuer (four tcgen05.mma.kind::i8
// of K = 32 a stage), and eight epilogue warps that read the accumulators from
// TMEM, scale and store them (two to a scheduler: one alone waits for its own
// results most of the time).  There are two accumulators, so that the next
// tile is multiplied while one is stored.
//
// CG = 1: a CTA multiplies 128 rows of W.  CG = 2 (more than 128 tokens): two
// CTAs share one product of 256 rows and up to 256 tokens (cta_group::2).  Each
// loads its own rows of W and half of the tokens, 32 KB a stage instead of 48:
// at 128 x 256 x 128 the tensor cores take a stage faster than L2 delivers 48.
//
// Work split.  The tiles that fill no whole wave of the grid come first: their
// stages are dealt to the CTAs in equal ranges, a few of them a tile.
// The whole waves follow, one tile to a CTA, neighbours at the same time (they
// share rows of W or X in L2), and hide the joining of the shared tiles.  A
// CTA that holds a part of a tile writes its sums to the workspace; the last
// to arrive adds the others' to its own, scales and stores.  Integer sums do
// not depend on their order.
//
// Measured (us in a graph, weights not in L2; bytes against a measured copy's 6.53
// TB/s, operations against 4.5 POP/s nominal): 1 token of 4096 x 14336 12.0 (0.75 of
// the bytes), of 28672 x 8192 39.7 (0.91); 19 tokens of 5000 x 2064 8.8; 64 of 28672 x
// 8192 48.8 (0.75; cuBLAS's integer product 53.5); 256 tokens 61.0 (0.63; 58.0: the
// tensor cores' 27 us and the bytes' 39 do not quite overlap); 4096 tokens of 14336 x
// 4096 167 (2.9 POP/s, 0.64 of the operations; 155).
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
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kWBytes = kRows * kChunk;

struct __align__(64) Params {
    CUtensorMap tm_w;  // u8 [N][K], box 128 x 128, 128-byte swizzle, zeros past the ends
    CUtensorMap tm_x;  // u8 [M][K], box 128 x tokens / CG
    const float *x_scale, *w_scale;
    void *y;
    int y_f32;
    long long M, N;
    int tokens;              // per tile, a multiple of 16
    int chunks;              // stages per tile
    int tiles_m, waves;      // token tiles; whole waves of tiles
    int rest, ranges;        // tiles before them, and the workers (from 0) that their stages are dealt to
    long long units;         // those tiles' stages
    uint32_t *err;
    uint32_t *cnt;           // workspace's head: one arrival counter per CTA (zero between calls)
    int32_t *part;           // workspace: [CTAs][2][tokens][kRows] parts of shared tiles
    int stages;
    uint32_t stage_bytes, acc_cols, tmem_cols;  // of one CTA
};

// D[tmem] (+)= A[smem] * B[smem] for one (128 CG) x N x 32 step, int8 -> int32.
template <int CG>
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Instruction descriptor: int8 x int8 -> int32, both operands K-major, M =
// 128 CG, N = n.
template <int CG>
__device__ __forceinline__ uint32_t instr_desc(int n) {
    return (2u << 4)                                  // D format int32
           | (1u << 7)                                // A format signed
           | (1u << 10)                               // B format signed
           | (static_cast<uint32_t>(n >> 3) << 17)    // N / 8
           | (static_cast<uint32_t>(CG * kRows >> 4) << 24);  // M / 16
}

// The pair's other half.  An address of this CTA's shared memory as the
// leader's (rank 0) address of the same place.
__device__ __forceinline__ uint32_t leader_addr(uint32_t a) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Arrive on a barrier of the leader.
__device__ __forceinline__ void arrive_at_leader(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}

// Bounded wait for a phase that the other CTA takes part in.
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (clock64() - t0 > kWaitCycles) return false;
    }
}

// TMA copy into this CTA that completes on the leader's barrier.
__device__ __forceinline__ void tma2d_pair(uint32_t dst, const CUtensorMap *tm, int c0, int c1, uint32_t leader_bar,
                                           uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(tm), "r"(c0), "r"(c1), "r"(leader_bar), "l"(policy)
        : "memory");
}

// Arrive on `bar` of both CTAs once every product that this thread issued so
// far has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (CG == 1)
        umma_commit(bar);
    else
        commit_pair(bar);
}

// The stretches of work of one worker (a CTA or a pair), in order: its range of
// the first tiles, then whole ones.  [k0, k1): the stages of the tile.
struct Work {
    long long tile;
    int k0, k1;

    __device__ __forceinline__ bool whole(const Params &p) const { return k0 == 0 && k1 == p.chunks; }
};

// First stage of worker c's range.
__device__ __forceinline__ long long range_start(const Params &p, int c) {
    return c < p.ranges ? c * p.units / p.ranges : p.units;
}

template <int CG>
struct Walk {
    int wave;
    long long u, u1;  // position in the first tiles

    __device__ __forceinline__ explicit Walk(const Params &p)
        : wave(0), u(range_start(p, blockIdx.x / CG)), u1(range_start(p, blockIdx.x / CG + 1)) {}

    __device__ __forceinline__ bool next(const Params &p, Work &w) {
        if (u < u1) {
            w.tile = u / p.chunks;
            const long long t0 = w.tile * p.chunks;
            w.k0 = static_cast<int>(u - t0);
            w.k1 = static_cast<int>(min(static_cast<long long>(p.chunks), u1 - t0));
            u = t0 + w.k1;
            return true;
        }
        if (wave == p.waves) return false;
        w.tile = p.rest + static_cast<long long>(wave) * (gridDim.x / CG) + blockIdx.x / CG;
        w.k0 = 0;
        w.k1 = p.chunks;
        ++wave;
        return true;
    }
};

// The workers [first, last] that share tile t (there are no more ranges than
// stages, so every one of them holds some).  The first one's counter is the
// tile's: a worker is the first of one shared tile at most.
__device__ __forceinline__ void sharers(const Params &p, long long t, int &first, int &last) {
    auto owner = [&](long long u) { return static_cast<int>(((u + 1) * p.ranges + p.units - 1) / p.units - 1); };
    first = owner(t * p.chunks);
    last = owner((t + 1) * p.chunks - 1);
}

// Arrive on a shared tile's counter (each CTA of a pair has its own); true for
// the last arrival, which also sets it back to zero.
template <int CG>
__device__ __forceinline__ bool arrive(const Params &p, int first, int last) {
    uint32_t *cnt = p.cnt + first * CG + blockIdx.x % CG;
    if (atomicAdd(cnt, 1u) != static_cast<uint32_t>(last - first)) return false;
    atomicExch(cnt, 0u);
    return true;
}

// Worker c's part of a shared tile (this CTA's rows): slot 1 for the tile that
// it is the first of, slot 0 for the one that its range starts inside.
template <int CG>
__device__ __forceinline__ int32_t *part_of(const Params &p, int c, bool is_first) {
    return p.part + ((static_cast<size_t>(c) * CG + blockIdx.x % CG) * 2 + (is_first ? 1 : 0)) * p.tokens * kRows;
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

// 32 TMEM lanes x 16 consecutive columns into 16 registers per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, int32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// Sixteen sums of one output channel, tokens m .. m + 15 of which the first
// `here` exist: scaled and stored.  sx: the lane's token scale (lane i holds
// that of token m + i).  `live`: the channel exists.
__device__ __forceinline__ void put16(const Params &p, const int32_t (&v)[16], long long m, int here, long long n,
                                      bool live, float sx, float sw) {
    const size_t o = static_cast<size_t>(m) * static_cast<size_t>(p.N) + static_cast<size_t>(n);
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        f[i] = static_cast<float>(v[i]) * __shfl_sync(0xFFFFFFFFu, sx, i) * sw;
    if (!live) return;
    if (p.y_f32) {
        float *y = static_cast<float *>(p.y) + o;
#pragma unroll
        for (int i = 0; i < 16; ++i, y += p.N)
            if (i < here) *y = f[i];
    } else {
        uint16_t *y = static_cast<uint16_t *>(p.y) + o;
#pragma unroll
        for (int i = 0; i < 16; ++i, y += p.N)
            if (i < here) *y = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
    }
}

// Add the other workers' parts of a tile, from place `at` on, to sums v of 16
// tokens of which the first `here` exist; PB parts of NV tokens in flight.
template <int CG, int PB, int NV>
__device__ __forceinline__ void add_parts(const Params &p, int32_t (&v)[16], int first, int last, int at, int here) {
    for (int o = first; o <= last; o += PB) {
        int32_t t[PB][NV];
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const bool other = o + b <= last && o + b != static_cast<int>(blockIdx.x / CG);
            const int32_t *src = part_of<CG>(p, other ? o + b : first, o + b == first) + at;
#pragma unroll
            for (int i = 0; i < NV; ++i) t[b][i] = other && i < here ? __ldcg(src + i * kRows) : 0;
        }
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += t[b][i];
    }
}

// The accumulators at `tmem`, of this worker's stages of tile w.tile: y, or a
// part and, for the tile's last arrival, y from all parts.  Lane i of TMEM is
// this CTA's row i of the tile; a warp reads the 32 lanes of its quadrant, and
// every second sixteen tokens (`odd`: the second ones).
template <int CG>
__device__ __forceinline__ void epilogue(const Params &p, const Layout &L, const Work &w, uint32_t tmem, int quad,
                                         int odd, int lane, uint32_t bar_empty) {
    const int row = quad * 32 + lane;
    const long long n = (w.tile / p.tiles_m * CG + blockIdx.x % CG) * kRows + row, m0 = w.tile % p.tiles_m * p.tokens;
    const int m_here = static_cast<int>(min(static_cast<long long>(p.tokens), p.M - m0));
    const bool live = n < p.N;
    const float sw = live ? p.w_scale[n] : 0.f;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    int first = 0, last = 0;
    bool store = true;
    if (!w.whole(p)) {
        sharers(p, w.tile, first, last);
        int32_t *mine = part_of<CG>(p, blockIdx.x / CG, w.k0 == 0) + row;
        for (int c = 16 * odd; c < m_here; c += 32) {
            int32_t v[16];
            tmem_ld16(taddr + static_cast<uint32_t>(c), v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < m_here) __stcg(mine + (c + i) * kRows, v[i]);
        }
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
        if (quad == 0 && odd == 0 && lane == 0) {
            sts32(L.last, arrive<CG>(p, first, last) ? 1u : 0u);
            sts32(L.shared_done, lds32(L.shared_done) + 1);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
        store = lds32(L.last) != 0;
        if (store) __threadfence();
    }
    if (store) {
        auto token_scale = [&](int c) {
            return c + (lane & 15) < m_here ? p.x_scale[m0 + c + (lane & 15)] : 0.f;
        };
        float sx = token_scale(16 * odd);
        for (int c = 16 * odd; c < m_here; c += 32) {
            int32_t v[16];
            tmem_ld16(taddr + static_cast<uint32_t>(c), v);
            const float sx1 = token_scale(c + 32);
            tmem_wait_ld();
            if (first != last) {
                if (m_here <= 4)
                    add_parts<CG, 8, 4>(p, v, first, last, c * kRows + row, m_here);
                else
                    add_parts<CG, 4, 16>(p, v, first, last, c * kRows + row, m_here - c);
            }
            put16(p, v, m0 + c, m_here - c, n, live, sx, sw);
            sx = sx1;
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
        if (CG == 1)
            bar_arrive(bar_empty);
        else
            arrive_at_leader(bar_empty);
    }
}

template <int CG>
__global__ void __launch_bounds__(kThreads, 1) gemm_i8_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sb = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const Layout L = layout(sb);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.stages;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            bar_init(L.full + 8 * s, 1);
            bar_init(L.empty + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            bar_init(L.acc_full + 8 * a, 1);
            bar_init(L.acc_empty + 8 * a, kEpiWarps * CG);
        }
        bar_init(L.done, 1);
        sts32(L.abort, 0u);
        sts32(L.shared_done, 0u);
        fence_barrier_init();
    }
    if (warp == 1) {
        if (CG == 1) {
            tmem_alloc(L.tmem_slot, p.tmem_cols);
            tmem_relinquish();
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(L.tmem_slot),
                         "r"(p.tmem_cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // the other CTA's barriers are there
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
            Walk<CG> walk(p);
            const int x_rows = p.tokens / CG;
            for (Work w; ok && walk.next(p, w);) {
                const int n0 = (static_cast<int>(w.tile / p.tiles_m) * CG + static_cast<int>(rank)) * kRows;
                const int m0 = static_cast<int>(w.tile % p.tiles_m) * p.tokens + static_cast<int>(rank) * x_rows;
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!bar_wait(L.empty + 8 * s, (round & 1u) ^ 1u)) {
                        give_up(p, L.abort);
                        ok = false;
                        break;
                    }
                    const uint32_t st = L.stages + static_cast<uint32_t>(s) * p.stage_bytes, bar = L.full + 8 * s;
                    if (rank == 0) bar_expect_tx(bar, CG * p.stage_bytes);
                    if (CG == 1) {
                        tma2d(st, &p.tm_w, k * kChunk, n0, bar, pol);
                        tma2d(st + kWBytes, &p.tm_x, k * kChunk, m0, bar, pol);
                    } else {
                        tma2d_pair(st, &p.tm_w, k * kChunk, n0, leader_addr(bar), pol);
                        tma2d_pair(st + kWBytes, &p.tm_x, k * kChunk, m0, leader_addr(bar), pol);
                    }
                    ++issued;
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                }
            }
            // every copy lands before the CTA leaves (the leader's barriers
            // stand for both CTAs' copies)
            if (rank == 0)
                for (long long i = issued > S ? issued - S : 0; i < issued; ++i)
                    bar_wait(L.full + 8 * static_cast<uint32_t>(i % S), static_cast<uint32_t>((i / S) & 1));
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = instr_desc<CG>(p.tokens);
            int s = 0;
            uint32_t round = 0, tile = 0;
            bool ok = true;
            Walk<CG> walk(p);
            for (Work w; ok && walk.next(p, w); ++tile) {
                const uint32_t a = tile & 1u;
                const uint32_t free_bar = L.acc_empty + 8 * a, free_par = ((tile >> 1) & 1u) ^ 1u;
                ok = CG == 1 ? bar_wait(free_bar, free_par) : pair_wait(free_bar, free_par);
                for (int k = w.k0; ok && k < w.k1; ++k) {
                    ok = CG == 1 ? bar_wait(L.full + 8 * s, round & 1u) : pair_wait(L.full + 8 * s, round & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = L.stages + static_cast<uint32_t>(s) * p.stage_bytes;
#pragma unroll
                    for (int kk = 0; kk < kChunk / 32; ++kk)
                        umma_i8<CG>(tmem + a * p.acc_cols, smem_desc_sw128(st + 32u * kk),
                                    smem_desc_sw128(st + kWBytes + 32u * kk), idesc, k > w.k0 || kk > 0);
                    commit<CG>(L.empty + 8 * s);
                    if (++s == S) {
                        s = 0;
                        ++round;
                    }
                }
                if (ok) commit<CG>(L.acc_full + 8 * a);
            }
            if (!ok) give_up(p, L.abort);
            // every product issued has completed before TMEM is freed
            commit<CG>(L.done);
        }
        if (lane == 0) bar_wait(L.done, 0);
    } else {
        const int quad = warp & 3, odd = (warp - 2) >> 2;  // the TMEM lanes that this warp may read, its tokens
        uint32_t tile = 0;
        Walk<CG> walk(p);
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
            epilogue<CG>(p, L, w, tmem + a * p.acc_cols, quad, odd, lane, L.acc_empty + 8 * a);
        }
    }
    __syncthreads();
    // (the other CTA's products read this one's shared memory, its arrivals
    // go to this one's barriers)
    if (CG == 2) cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (CG == 1)
            tmem_dealloc(tmem, p.tmem_cols);
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols)
                         : "memory");
    }
    if (threadIdx.x == 0 && lds32(L.abort)) {
        // the shared tiles that this CTA did not get to still see its
        // arrival, so that their counters return to zero
        const uint32_t done = lds32(L.shared_done);
        uint32_t k = 0;
        Walk<CG> walk(p);
        walk.wave = p.waves;
        for (Work w; walk.next(p, w);) {
            if (w.whole(p) || k++ < done) continue;
            int first, last;
            sharers(p, w.tile, first, last);
            arrive<CG>(p, first, last);
        }
    }
}

// ---------------------------------------------------------------------------
// A few tokens: no tensor cores, whose product starts late and is joined from
// parts.  A group of `split` warps takes four rows of W, each thread 16 bytes of
// them at a time, so that much of W is on its way at once; four products a dp4a,
// sums across the group at the end.

constexpr int kDotThreads = 256, kDotRows = 4;

struct DotParams {
    const int8_t *x, *w;
    const float *x_scale, *w_scale;
    void *y;
    long long N;
    int y_f32, M, K;
    int split;  // warps to a group of rows: 1, 2, 4 or 8
};

__device__ __forceinline__ int dot16(const int4 &a, const int4 &b, int sum) {
    return __dp4a(a.w, b.w, __dp4a(a.z, b.z, __dp4a(a.y, b.y, __dp4a(a.x, b.x, sum))));
}

// MT tokens (the last ones may not be there).
template <int MT>
__global__ void __launch_bounds__(kDotThreads, 2) dot_i8_kernel(const __grid_constant__ DotParams p) {
    constexpr int kDotWarps = kDotThreads / 32, kBatch = MT <= 2 ? 4 : 2;
    __shared__ int part[kDotWarps][kDotRows * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = 32 * p.split, t = threadIdx.x % threads;
    const long long n0 = (static_cast<long long>(blockIdx.x) * (kDotWarps / p.split) + warp / p.split) * kDotRows;
    const int8_t *row[kDotRows];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)  // (rows past the last are the last, and not stored)
        row[r] = p.w + min(n0 + r, p.N - 1) * p.K;
    int sum[kDotRows][MT];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[r][m] = 0;
    grid_launch_dependents();
    // x, w and y may belong to earlier kernels (hence no loads as constants here)
    grid_dependency_wait();
    for (int k0 = t * 16; k0 < p.K; k0 += kBatch * threads * 16) {
        int4 wv[kBatch][kDotRows];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int r = 0; r < kDotRows; ++r) {
                const int k = k0 + b * threads * 16;
                wv[b][r] = make_int4(0, 0, 0, 0);
                if (k < p.K) wv[b][r] = __ldcs(reinterpret_cast<const int4 *>(row[r] + k));
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int k = k0 + b * threads * 16;
            if (k < p.K) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const int4 xv =
                        *reinterpret_cast<const int4 *>(p.x + static_cast<size_t>(min(m, p.M - 1)) * p.K + k);
#pragma unroll
                    for (int r = 0; r < kDotRows; ++r) sum[r][m] = dot16(wv[b][r], xv, sum[r][m]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int s = __reduce_add_sync(0xFFFFFFFFu, sum[r][m]);
            if (lane == 0) part[warp][r * MT + m] = s;
        }
    __syncthreads();
    if (t < kDotRows * MT) {
        const int r = t / MT, m = t - r * MT;
        const long long n = n0 + r;
        if (n < p.N && m < p.M) {
            int s = 0;
            for (int i = 0; i < p.split; ++i) s += part[warp + i][t];
            const float v = static_cast<float>(s) * p.x_scale[m] * p.w_scale[n];
            const size_t at = static_cast<size_t>(m) * p.N + n;
            if (p.y_f32)
                static_cast<float *>(p.y)[at] = v;
            else
                static_cast<uint16_t *>(p.y)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
    }
}

}  // namespace gemm8

// ---------------------------------------------------------------------------
// Host side.

namespace {

constexpr uint32_t kSmemLimit = 227 * 1024;
constexpr int kDotTokens = 8;
// More tokens than this: two CTAs a product (14336 x 4096, one and two, us: 96
// tokens 15.6 and 16.5, 128 16.0 and 17.1, 256 20.2 and 18.9, 512 36 and 29, 4096
// 186 and 175).
constexpr int kPairTokens = 128;

struct Plan8 {
    int cg, tokens, tiles_m;
    size_t cnt_bytes, part_bytes;
};

Plan8 plan8(int64_t M, int sms) {
    Plan8 pl;
    pl.cg = M > kPairTokens ? 2 : 1;
    // token tiles of equal size, as few as 256 tokens each allow
    const int64_t tiles = (M + gemm8::kMaxTokens - 1) / gemm8::kMaxTokens, step = 16 * pl.cg;
    pl.tiles_m = static_cast<int>(tiles);
    pl.tokens = static_cast<int>(((M + tiles - 1) / tiles + step - 1) / step * step);
    pl.cnt_bytes = S12_WS_HEAD;  // (a counter for each CTA)
    pl.part_bytes = static_cast<size_t>(sms) * 2 * pl.tokens * gemm8::kRows * 4;
    return pl;
}

// How many workers the `rest` tiles before the whole waves are dealt to, of
// `workers` in all.  Dealing evens the load out: it saves about chunks * (1 -
// rest / workers) stages, each of which takes its bytes at some 53 a cycle.
// Joining costs some 3000 cycles, and 20 a token for each part; where that is
// more, a tile stays whole, and the parts of large tiles are few.
int ranges_of(int rest, int workers, int chunks, uint32_t stage_bytes, int tokens) {
    if (rest == 0) return 0;
    const int share = tokens <= 64 ? 8 : 4;
    const int ranges = static_cast<int>(
        std::min<long long>({workers, static_cast<long long>(rest) * share, static_cast<long long>(rest) * chunks}));
    const double saved = chunks * (1.0 - static_cast<double>(rest) / ranges) * stage_bytes / 53.0;
    const double parts = static_cast<double>(ranges) / rest;
    return saved > 3000.0 + 20.0 * tokens * parts ? ranges : rest;
}

// Warps to a group of rows: the fewest columns' time.  The blocks go in waves of
// two an SM, and a wave takes its warps' columns of a row and some 1300 more (it
// starts, and its sums are reduced), whether it is full or not.  One token, us, by
// 1, 2, 4 and 8 warps:
//   900 x 4112    5.03  3.69  2.94  2.64 *     7000 x 12304  18.3 * 18.8   18.5   18.7
//   1800 x 4112   5.44  4.12  3.37 * 4.67      7000 x 28016  36.7   37.6   35.6 * 34.8
//   3500 x 4112   6.21  4.99 * 5.74  7.00      14000 x 1040   5.7 *  7.1   11.6   20.3
//   3500 x 20000  20.3  15.0 * 17.1  16.3      14000 x 4112  14.2   14.0 * 15.6   23.8
//   7000 x 4112   7.84 * 9.08  9.00  12.8      30000 x 4112  25.8 * 25.8   29.8   49.3
//   7000 x 10000  14.8 * 16.3  16.5  17.0      30000 x 12304 66.5   62.7 * 63.1   66.8
// (* is what is taken; over 138 sizes of 1 to 8 tokens it is within 4.5 % of the
// best of the four, and 0.1 % on average).
int dot_split(int64_t N, int64_t K, int sms) {
    const int64_t groups = (N + gemm8::kDotRows - 1) / gemm8::kDotRows, warps = gemm8::kDotThreads / 32;
    int best = 1;
    int64_t least = 0;
    for (int split = 1; split <= warps; split *= 2) {
        const int64_t blocks = (groups * split + warps - 1) / warps, waves = (blocks + 2 * sms - 1) / (2 * sms);
        const int64_t cost = waves * (K / split + 1300);
        if (split > 1 && cost >= least) continue;
        least = cost;
        best = split;
    }
    return best;
}

template <int CG>
int run8(const gemm8::Params &p, int workers, uint32_t smem, cudaStream_t stream) {
    auto kern = gemm8::gemm_i8_kernel<CG>;
    // (always the same limit: another thread's call may be between this line and its launch)
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
        return S12_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(workers * CG);
    cfg.blockDim = dim3(gemm8::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {CG, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = CG;  // (a cluster only for pairs)
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? S12_OK : S12_ERR_CUDA;
}

template <int MT>
int run_dot(const gemm8::DotParams &p, cudaStream_t stream) {
    const long long rows = gemm8::kDotThreads / 32 / p.split * gemm8::kDotRows;  // of a block
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.N + rows - 1) / rows));
    cfg.blockDim = dim3(gemm8::kDotThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemm8::dot_i8_kernel<MT>, p) == cudaSuccess ? S12_OK : S12_ERR_CUDA;
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
    if (sms > S12_WS_HEAD / 4) return S12_ERR_DEVICE;
    const Plan8 pl = plan8(c.M, sms);
    if (ws_bytes < pl.cnt_bytes + pl.part_bytes) return S12_ERR_CAPACITY;
    // The dot products against the tensor cores, us: 1 token 14336 x 4096 12.1 and
    // 14.7, 2 tokens 28672 x 8192 39.7 and 43.7, 3 tokens 14336 x 4096 14.7 both, 8
    // tokens 4096 x 4096 6.6 and 11.0, 14336 x 4096 18.9 and 14.6.
    if (c.M <= 2 || (c.M <= kDotTokens && static_cast<unsigned long long>(c.M) * c.N * c.K <= 3ull << 26)) {
        gemm8::DotParams d = {c.x, c.w, c.x_scale, c.w_scale, c.y, c.N, c.y_type == S12_TYPE_F32,
                              static_cast<int>(c.M), static_cast<int>(c.K), 1};
        d.split = dot_split(c.N, c.K, sms);
        if (c.M == 1) return run_dot<1>(d, stream);
        if (c.M == 2) return run_dot<2>(d, stream);
        if (c.M <= 4) return run_dot<4>(d, stream);
        return run_dot<8>(d, stream);
    }
    gemm8::Params p = {};
    if (make_tmap_u8_2d(&p.tm_w, c.w, c.K, c.N, c.K, gemm8::kChunk, gemm8::kRows, 128) != S12_OK ||
        make_tmap_u8_2d(&p.tm_x, c.x, c.K, c.M, c.K, gemm8::kChunk, pl.tokens / pl.cg, 128) != S12_OK)
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
    const int rows = gemm8::kRows * pl.cg, all = sms / pl.cg;
    const long long tiles = (c.N + rows - 1) / rows * pl.tiles_m;
    p.stage_bytes = gemm8::kWBytes + static_cast<uint32_t>(pl.tokens / pl.cg) * gemm8::kChunk;
    p.waves = static_cast<int>(tiles / all);
    p.rest = static_cast<int>(tiles % all);
    p.units = static_cast<long long>(p.rest) * p.chunks;
    p.ranges = ranges_of(p.rest, all, p.chunks, p.stage_bytes, pl.tokens);
    const int workers = p.waves ? all : p.ranges;
    p.cnt = static_cast<uint32_t *>(ws);
    p.part = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + pl.cnt_bytes);
    p.stages = static_cast<int>(std::min<uint32_t>(gemm8::kMaxStages, (kSmemLimit - 2048) / p.stage_bytes));
    p.acc_cols = 32;
    while (p.acc_cols < static_cast<uint32_t>(pl.tokens)) p.acc_cols <<= 1;
    p.tmem_cols = 2 * p.acc_cols;
    const uint32_t smem = 2048 + static_cast<uint32_t>(p.stages) * p.stage_bytes;
    return pl.cg == 1 ? run8<1>(p, workers, smem, stream) : run8<2>(p, workers, smem, stream);
}

}  // namespace s12
