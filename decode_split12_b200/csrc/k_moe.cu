// k_moe.cu -- a whole mixture-of-experts layer for a few tokens, over Split12
// expert weights, in one kernel (sm_100a):
//
//   scores[t][e] = sum_k router[e][k] * x[t][k]
//   the top_k experts of each token and their softmax weights w[t][s]
//   h[t][s]      = silu(Wgate_e x_t) * (Wup_e x_t)        e = ids[t][s]
//   y[t]         = sum_s w[t][s] * (Wdown_e h[t][s])
//
// Bound.  Every expert that some token is sent to is read once, compressed:
// 12.3 bits a weight, 3 * F * H weights an expert.  All else is small, so the
// kernel is bound by HBM, and what matters is that the copies never pause and
// that a weight costs few instructions.
//
// Steps, by one cooperative grid of one CTA per SM:
//   0. x is rewritten in the order the products read it; scores; every CTA
//      selects the experts and sorts the (token, slot) pairs by expert itself.
//   1. gate/up products; their sums go to the workspace by ranges of columns.
//      The grid meets, adds the ranges, applies the SwiGLU, and meets again.
//   2. down products, sums by ranges; the grid meets and adds ranges and slots.
// The first copies of step 2 are issued before the grid meets: weights do not
// depend on it.
//
// Two kernels share these steps, and a rule on the products' size chooses.
// Small: as in the GEMV, a warp takes 16 rows x 2 tiles of weights a stage from
// its own ring of two, decodes them in registers into the A operand of
// mma.m16n8k16, and multiplies 8 tokens at a time; a warp waits for no other, and
// a call starts fast.  Large: weights are decoded into TMEM and multiplied there
// by up to 64 pairs (tcgen05), below.
//
// Decode.  Weights i and i + 4 of eight share a register, because their code nibbles
// are 16 bits apart: a pair's exponents are one mask and one multiply-add of
// the code word, its signs and mantissas one byte permute, and one bit select
// joins them: 17 instructions for 8 weights.  x and h are kept with the same
// pairs in a register.  h is kept as the sum of two BF16 values, so that it
// carries 16 bits of mantissa and y is rounded once, where it is stored.
//
// All sums have a fixed order, so y is the same on every call.  Every wait is
// bounded.  One that gives up raises S12_FLAG_TIMEOUT and a word that the other
// waits watch; the CTAs then leave, and the last one clears the words.
//
// Measured (5e-4 of the weights 10 to 100 times as large as the rest; us in a
// graph, and the experts' compressed bytes against a measured copy's 6.53 TB/s):
//   8 experts of 14336 x 4096, top 2:  1 token 149 (0.56), 2 tokens that meet 3
//     experts 212 (0.59), 8 that meet 7 421 (0.69), 16 tokens 482 (0.69), 64 tokens
//     507 (0.65; 489 with the pairs spread evenly, up to 554 where one expert has
//     more than 40 of them)
//   32 experts of 1408 x 2176, top 4:  1 token 53, 9 tokens that meet 21 to 24
//     experts 113 to 128 (0.40), 64 193 (0.36)
//   64 experts of 1024 x 2048, top 8:  1 token 57, 16 tokens 160 (0.49), 64 200 (0.47)
// Copies of the kernels without a part (us; results wrong, timed only), for 64 tokens
// and one token of the 8 experts:
//   as they are 507, 150; escapes not put right 465, 128; no metadata read (and so
//   no escapes) 470, 133; nothing decoded, nor put right 455, 120; neither 388, 116
// So no part alone binds either kernel, and their schedulers issue in less than half
// of the cycles: they wait.  A call of one token begins and ends in about 25 us (the
// choice of experts, three meetings of the grid at 1.3 us, the sums).
// Version 2 containers: 1 token 174, 64 tokens 758, 64 tokens of the 64 experts 218.
// The counts of a row's earlier tiles are added up anew for every unit (a stage with
// escapes, in the small kernel), which grows with the square of a row.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "s12_device.cuh"
#include "s12_launch.h"
#include "s12_stage.cuh"
#include "s12_tc.cuh"

namespace s12 {
namespace moe {

using namespace stage;

constexpr int kWarps = 16;   // warps per CTA of the kernel for few pairs, one CTA per SM
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;   // stages per warp ring
constexpr int kSegSmall = 8, kSegLarge = 64;  // (token, slot) pairs that share one read of an expert's weights
constexpr int kMaxSlots = S12_MOE_MAX_TOKENS * S12_MOE_MAX_TOP_K;
constexpr int kMaxSegs = S12_MOE_MAX_EXPERTS + kMaxSlots / kSegSmall;
constexpr uint32_t kRingBytes = kWarps * kStages * kStageBytes;

// A matrix of all experts: expert after expert, rows_e rows each.
struct __align__(64) Mat {
    CUtensorMap tm_raw;   // u8 {128, T, R} (strides 128, K), box {128, 2, 16} or {128, 1, 128}, 128-byte swizzle
    CUtensorMap tm_code;  // u8 {64, T, R} (strides 64, K/2), box {64, 2, 16} or {64, 1, 128}, 64-byte swizzle
    const void *meta;     // version 1: base u8[n_tiles]; version 2: (base | count << 8) u16[n_tiles]
    const uint32_t *off;  // version 1: esc_off u32[n_tiles + 1]; version 2: row_esc u32[R + 1]
    const uint16_t *esc;
    uint32_t n_esc;
    int R, T;    // rows of all experts, tiles per row
    int G;       // 16-row groups per expert
    uint32_t S;  // stages per row group
};

// Words that the grid meets at.
enum { kBarRoute, kBarPack, kBarSums, kBarHidden, kBarDown, kNext1, kNext2, kExits, kAbort, kSyncWords };
static_assert(kSyncWords * 4 <= S12_WS_HEAD, "they lie in the workspace's head");

struct __align__(64) Params {
    Mat up, down;
    const uint16_t *x, *router;
    const int32_t *ids_in;
    const float *weights_in;
    int32_t *ids;
    float *weights;
    void *y;
    uint32_t *err;
    int tokens, experts, top_k, H, F;
    int renorm, y_f32;
    int seg;         // pairs of a segment at most
    int local;       // few pairs: every CTA routes for itself, with x in shared memory
    uint32_t range;  // stages of an item
    uint32_t pool;   // many pairs: bytes of shared memory for stages
    // workspace
    uint32_t *sync;         // kSyncWords, zero between calls
    double *scores;         // [tokens][experts]
    uint8_t *xp, *hi, *lo;  // x, and h as two BF16 values, in the products' order
    float *gu, *d;          // sums of the two steps: [ranges][slots][2F], [ranges][slots][H]
};

struct Shared {
    float weight[kMaxSlots];
    int16_t expert[kMaxSlots];  // of each (token, slot), -1 for none
    uint16_t token[kMaxSlots];  // of each pair of the list: the (token, slot) pairs by expert
    uint16_t place[kMaxSlots];  // of each (token, slot) in the list
    uint16_t segment[kMaxSlots];  // of each of the list
    int count[S12_MOE_MAX_EXPERTS], first[S12_MOE_MAX_EXPERTS], next[S12_MOE_MAX_EXPERTS];
    uint16_t seg_expert[kMaxSegs], seg_first[kMaxSegs];
    uint8_t seg_n[kMaxSegs];
    int n_segs, most;  // segments; pairs of the largest
    int ok, last;
};

// Order of x and h, in 16-byte pieces of 8 values, which come as 0 4 1 5 2 6 3 7.
// Few pairs: tile, then 16-column chunk of a lane's 64, then half chunk, then
// which of n tokens or pairs, then which 64 columns of the tile.  A warp's load
// of one half chunk is then contiguous over them.  Many: tile, then which 64
// columns, then which of n pairs, then the piece of the 64 columns, with the 128-byte
// swizzle.  h (and x, where many pairs share an expert) comes segment by segment.
__device__ __forceinline__ size_t piece_at(int tile, int chunk, int half, int n, int i, int qh) {
    return ((((static_cast<size_t>(tile) * 4 + chunk) * 2 + half) * n + i) * 2 + qh) * 16;
}

// Piece c8 of a row.
template <bool LARGE>
__device__ __forceinline__ size_t piece_of(int c8, int n, int i) {
    const int in = c8 & 15;  // of the tile: 64 columns, chunk, half
    if (LARGE) return (static_cast<size_t>(c8 >> 3) * n + i) * 128 + (((c8 & 7) ^ (i & 7)) << 4);
    return piece_at(c8 >> 4, (in >> 1) & 3, in & 1, n, i, in >> 3);
}

// ---------------------------------------------------------------------------
// Meeting of the grid.

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void give_up(const Params &p) {
    raise_flag(p.err, S12_FLAG_TIMEOUT);
    atomicExch(p.sync + kAbort, 1u);
}

// Every thread of the grid has come here, and what it wrote is visible;
// false (for the whole CTA) when a wait of the grid gave up.
__device__ __forceinline__ bool grid_meet(const Params &p, Shared *sm, int word) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(p.sync + word, 1u);
        int ok = 1;
        const long long t0 = clock64();
        while (ld_acquire(p.sync + word) < gridDim.x) {
            if (ld_acquire(p.sync + kAbort)) {
                ok = 0;
                break;
            }
            if (clock64() - t0 > kWaitCycles) {
                give_up(p);
                ok = 0;
                break;
            }
        }
        sm->ok = ok;
    }
    __syncthreads();
    return sm->ok != 0;
}

// ---------------------------------------------------------------------------
// Step 0: x in the products' order, scores, experts.

// Piece c8 of token t, to place i of n.
template <bool LARGE>
__device__ __forceinline__ void pack_piece(const Params &p, uint8_t *to, int t, int c8, int n, int i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p.x + static_cast<size_t>(t) * p.H) + c8);
    *reinterpret_cast<uint4 *>(to + piece_of<LARGE>(c8, n, i)) = make_uint4(
        prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u), prmt(v.y, v.w, 0x7632u));
}

// x token by token.
__device__ __forceinline__ void pack_x(const Params &p, uint8_t *to, int i0, int step) {
    const int per_row = p.H / 8;
    const int n = p.tokens * per_row;
    for (int i = i0; i < n; i += step) {
        const int t = i / per_row, c8 = i - t * per_row;  // piece c8 of token t
        pack_piece<false>(p, to, t, c8, p.tokens, t);
    }
}

// x segment by segment, a copy for each pair.
__device__ __forceinline__ void pack_sorted(const Params &p, const Shared *sm, int pairs) {
    const int per_row = p.H / 8;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < pairs * per_row; i += gridDim.x * blockDim.x) {
        const int at = i / per_row, c8 = i - at * per_row, seg = sm->segment[at], first = sm->seg_first[seg];
        pack_piece<true>(p, p.xp + static_cast<size_t>(first) * p.H * 2, sm->token[at], c8, sm->seg_n[seg], at - first);
    }
}

// Value c of eight.
__device__ __forceinline__ double value_of(const uint4 &a, int c) {
    const uint32_t u = c < 4 ? (c < 2 ? a.x : a.y) : (c < 6 ? a.z : a.w);
    return static_cast<double>(__uint_as_float(c & 1 ? u & 0xFFFF0000u : u << 16));
}

// Scores of TT tokens and TE experts to a warp, in 64 bits throughout, because
// the choice of experts hangs on the order of the scores: a product of BF16
// values is exact there, and none is too large or too small.  What it costs are
// the conversions (12 a cycle and SM; products 60), and code: eight loads in
// flight instead of four, with their 64 conversions each, took 1 us longer.
template <int TT, int TE>
__device__ __forceinline__ void score(const Params &p, double *scores, int u0, int step) {
    const int lane = threadIdx.x & 31;
    const int nt = (p.tokens + TT - 1) / TT, ne = (p.experts + TE - 1) / TE;
    for (int u = u0; u < nt * ne; u += step) {
        const int t0 = u / ne * TT, e0 = u % ne * TE;
        double acc[TT][TE];
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int j = 0; j < TE; ++j) acc[i][j] = 0.0;
        constexpr int kBatch = TT == 1 ? 4 : 1;  // loads in flight
        for (int k0 = lane * 8; k0 < p.H; k0 += 256 * kBatch) {
            uint4 xr[kBatch][TT], rr[kBatch][TE];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int k = k0 + 256 * b;
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    const size_t t = min(t0 + i, p.tokens - 1);
                    xr[b][i] = make_uint4(0u, 0u, 0u, 0u);
                    if (k < p.H) xr[b][i] = __ldg(reinterpret_cast<const uint4 *>(p.x + t * p.H + k));
                }
#pragma unroll
                for (int j = 0; j < TE; ++j) {
                    const size_t e = min(e0 + j, p.experts - 1);
                    rr[b][j] = make_uint4(0u, 0u, 0u, 0u);
                    if (k < p.H) rr[b][j] = __ldg(reinterpret_cast<const uint4 *>(p.router + e * p.H + k));
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (k0 - lane * 8 + 256 * b >= p.H) break;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    double xv[TT];
#pragma unroll
                    for (int i = 0; i < TT; ++i) xv[i] = value_of(xr[b][i], c);
#pragma unroll
                    for (int j = 0; j < TE; ++j) {
                        const double rv = value_of(rr[b][j], c);
#pragma unroll
                        for (int i = 0; i < TT; ++i) acc[i][j] = fma(xv[i], rv, acc[i][j]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < TT; ++i)
#pragma unroll
            for (int j = 0; j < TE; ++j) {
                double s = acc[i][j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                if (lane == 0 && t0 + i < p.tokens && e0 + j < p.experts)
                    scores[static_cast<size_t>(t0 + i) * p.experts + e0 + j] = s;
            }
    }
}

// The experts and weights of token t, by one warp: the top_k largest scores,
// the lower index first where two are equal.  A NaN among the scores counts as
// -infinity in their order and makes all the token's weights NaN, also those of
// experts whose own scores are numbers.
__device__ __forceinline__ void select_experts(const Params &p, Shared *sm, const double *scores, int t) {
    constexpr int kPer = S12_MOE_MAX_EXPERTS / 32;
    const int lane = threadIdx.x & 31;
    const double *row = scores + static_cast<size_t>(t) * p.experts;
    const double low = -__longlong_as_double(0x7FF0000000000000ll);
    // scores as integers of the same order, 0 for an expert that is chosen or not there
    unsigned long long key[kPer];
    double v[kPer];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        key[i] = 0;
        v[i] = low;
        if (32 * i >= p.experts) continue;
        const int e = lane + 32 * i;
        if (e < p.experts) {
            v[i] = row[e];
            if (v[i] != v[i]) {
                v[i] = low;
                nan = true;
            }
            const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v[i] + 0.0));
            key[i] = b >> 63 ? ~b : b | 1ull << 63;  // (-infinity: 2^52 - 1)
        }
    }
    nan = __any_sync(0xFFFFFFFFu, nan);
    double top = 0.0;
    float mine = 0.f;  // lane s < top_k: the weight of slot s before its division
    int chosen = -1;
    for (int s = 0; s < p.top_k; ++s) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (32 * i < p.experts && key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t hi = static_cast<uint32_t>(best >> 32), most = __reduce_max_sync(0xFFFFFFFFu, hi);
        const uint32_t lo = hi == most ? static_cast<uint32_t>(best) : 0u, least = __reduce_max_sync(0xFFFFFFFFu, lo);
        at = __reduce_min_sync(0xFFFFFFFFu, hi == most && lo == least && best ? at : 0x7FFFFFFF);
        const unsigned long long k = (static_cast<unsigned long long>(most) << 32) | least;
        const double value = __longlong_as_double(static_cast<long long>(k >> 63 ? k & ~(1ull << 63) : ~k));
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (at == lane + 32 * i) key[i] = 0;
        if (s == 0) top = value;
        if (lane == s) {
            chosen = at;
            mine = expf(static_cast<float>(value - top));
        }
    }
    float sum = 0.f;
    if (p.renorm) {
        sum = mine;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (32 * i < p.experts && lane + 32 * i < p.experts) sum += expf(static_cast<float>(v[i] - top));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < p.top_k) {
        const int i = t * p.top_k + lane;
        const float weight = nan ? __uint_as_float(0x7FC00000u) : mine / sum;
        sm->expert[i] = static_cast<int16_t>(chosen);
        sm->weight[i] = weight;
        if (blockIdx.x == 0) {
            if (p.ids) p.ids[i] = chosen;
            if (p.weights) p.weights[i] = weight;
        }
    }
}

// Every CTA for itself: the (token, slot) pairs sorted by expert (by index
// inside one), cut into segments of at most p.seg.
__device__ __forceinline__ void route(const Params &p, Shared *sm, const double *scores) {
    const int slots = p.tokens * p.top_k, tid = threadIdx.x;
    if (p.ids_in) {
        for (int i = tid; i < slots; i += blockDim.x) {
            const int e = __ldg(p.ids_in + i);
            sm->expert[i] = static_cast<int16_t>(e >= 0 && e < p.experts ? e : -1);
            sm->weight[i] = __ldg(p.weights_in + i);
        }
    } else {
        for (int t = tid >> 5; t < p.tokens; t += blockDim.x >> 5) select_experts(p, sm, scores, t);
    }
    for (int e = tid; e < p.experts; e += blockDim.x) sm->count[e] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += blockDim.x)
        if (sm->expert[i] >= 0) atomicAdd(&sm->count[sm->expert[i]], 1);
    __syncthreads();
    if (tid < 32) {
        constexpr int kPer = S12_MOE_MAX_EXPERTS / 32;
        int pairs = 0, segs = 0, most = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = tid * kPer + i, n = e < p.experts ? sm->count[e] : 0;
            pairs += n;
            segs += (n + p.seg - 1) / p.seg;
            most = max(most, min(n, p.seg));
        }
        int pairs_to = pairs, segs_to = segs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xFFFFFFFFu, pairs_to, o), b = __shfl_up_sync(0xFFFFFFFFu, segs_to, o);
            if (tid >= o) {
                pairs_to += a;
                segs_to += b;
            }
        }
        int at = pairs_to - pairs, seg = segs_to - segs;
        for (int i = 0; i < kPer; ++i) {
            const int e = tid * kPer + i, n = e < p.experts ? sm->count[e] : 0;
            if (e < p.experts) {
                sm->first[e] = sm->next[e] = at;
                sm->count[e] = seg;  // (from here on the expert's first segment)
            }
            for (int k = 0; k < n; k += p.seg, ++seg) {
                sm->seg_expert[seg] = static_cast<uint16_t>(e);
                sm->seg_first[seg] = static_cast<uint16_t>(at + k);
                sm->seg_n[seg] = static_cast<uint8_t>(min(n - k, p.seg));
            }
            at += n;
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (tid == 31) {
            sm->n_segs = segs_to;
            sm->most = most;
        }
    }
    __syncthreads();
    if (tid < 32) {
        // 32 slots at a time, in order: those of one expert follow one another
        for (int i0 = 0; i0 < slots; i0 += 32) {
            const int i = i0 + tid, e = i < slots ? sm->expert[i] : -1;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
            const int rank = __popc(same & ((1u << tid) - 1u));
            int at = 0;
            if (e >= 0) at = sm->next[e] + rank;
            __syncwarp();
            if (e >= 0) {
                if (rank == 0) sm->next[e] = at + __popc(same);
                sm->place[i] = static_cast<uint16_t>(at);
                sm->token[at] = static_cast<uint16_t>(i / p.top_k);
                sm->segment[at] = static_cast<uint16_t>(sm->count[e] + (at - sm->first[e]) / p.seg);
            }
            __syncwarp();
        }
    }
    __syncthreads();
}

template <int PH>
__device__ __forceinline__ const Mat &mat(const Params &p) {
    return PH == 1 ? p.up : p.down;
}

// The warp's ring: stages issued and consumed so far, over both steps.
struct Ring {
    uint32_t bars, base;
    int issued, consumed;
};

// The end of a CTA: the last one sets the workspace's words back to zero.
__device__ __forceinline__ void leave(const Params &p, Shared *sm) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        sm->last = atomicAdd(p.sync + kExits, 1u) + 1 == gridDim.x;
    }
    __syncthreads();
    if (sm->last) {
        __threadfence();
        if (threadIdx.x < kSyncWords) p.sync[threadIdx.x] = 0u;
    }
}

// ---------------------------------------------------------------------------
// Decode.

// Eight weights as the pairs (0, 4), (1, 5), (2, 6), (3, 7): raw bytes R0 (0
// to 3) and R1 (4 to 7), code nibbles C, B2 = base << 7 in both halves.  base
// + 15 at most 256 << 7 stays inside its half, and the select takes bits 7 to
// 14 of the sum alone, so an escape's nibble disturbs no other weight.
__device__ __forceinline__ void decode_pairs(uint32_t R0, uint32_t R1, uint32_t C, uint32_t B2, uint32_t *out) {
    const uint32_t D = C >> 8;
    const uint32_t e[4] = {(C & 0x000F000Fu) * 128u + B2, (C & 0x00F000F0u) * 8u + B2, (D & 0x000F000Fu) * 128u + B2,
                           (D & 0x00F000F0u) * 8u + B2};
    const uint32_t b[4] = {prmt(R0, R1, 0x4400u), prmt(R0, R1, 0x5511u), prmt(R0, R1, 0x6622u), prmt(R0, R1, 0x7733u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = (b[i] & 0x807F807Fu) | (e[i] & 0x7F807F80u);
}

// The exact values of the escapes among 16 decoded weights (code words C),
// stream index idx on; reads at or past `limit` are skipped and flagged.  `ev`
// is the value at index `known`, which was read ahead: most tile rows with
// escapes have one, and it comes from far away.
__device__ __forceinline__ void patch(uint32_t (&w)[8], uint2 C, uint32_t idx, uint32_t limit, uint32_t known,
                                      uint32_t ev, const uint16_t *__restrict__ esc, uint32_t *err) {
    uint64_t mm = (static_cast<uint64_t>(escape_nibbles(C.y)) << 32) | escape_nibbles(C.x);
    while (mm) {
        const int j = (__ffsll(static_cast<long long>(mm)) - 1) >> 2;
        mm &= mm - 1;
        uint32_t v = 0;
        if (idx < limit)
            v = idx == known ? ev : __ldg(esc + idx);
        else
            raise_flag(err, S12_FLAG_ESC_RANGE);
        ++idx;
        const int at = (j >> 3) * 4 + (j & 3);              // the pair, and the half of it
        const uint32_t sel = j & 4 ? 0x5410u : 0x3254u;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r == at) w[r] = prmt(w[r], v, sel);
    }
}

// ---------------------------------------------------------------------------
// Results.

__device__ __forceinline__ void put_y(const Params &p, size_t o, float v) {
    if (p.y_f32)
        static_cast<float *>(p.y)[o] = v;
    else
        static_cast<uint16_t *>(p.y)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// The lane's 16 values of one half chunk pair (two pieces).
__device__ __forceinline__ void load_x(uint32_t (&xw)[8], const uint8_t *src, size_t half, bool live) {
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (live) {
        a = *reinterpret_cast<const uint4 *>(src);
        b = *reinterpret_cast<const uint4 *>(src + half);
    }
    xw[0] = a.x; xw[1] = a.y; xw[2] = a.z; xw[3] = a.w;
    xw[4] = b.x; xw[5] = b.y; xw[6] = b.z; xw[7] = b.w;
}

// The chunk's four products.  One would wait for the one before it on the same
// sums, so each has sums of its own.
__device__ __forceinline__ void chunk_mma(float (&acc)[4][4], const uint32_t (&wa)[8], const uint32_t (&wb)[8],
                                          const uint32_t (&xw)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        mma16816(acc[i], wa[2 * i], wb[2 * i], wa[2 * i + 1], wb[2 * i + 1], xw[2 * i], xw[2 * i + 1]);
}

// ---------------------------------------------------------------------------
// Few tokens an expert: at most eight pairs share a read of an expert's
// weights.
//
// An item is a row group by a few stages of its columns.  Warps take items as
// they come for them (two are known in advance, the rest come from a counter
// of the grid), and write an item's sums to its place in the workspace, where
// the next step adds up the ranges of a row group in their order.  So warps
// never wait for one another inside a step, every SM works until the items are
// gone (dealt in equal ranges, the slowest SM took a fifth longer than the
// average), and which warp has which item does not change any sum.  The price
// is 64 bytes written a pair for 6 KB of weights or more, and a meeting of the
// grid before and after the sums of step 1; the first weights of step 2 are
// copied meanwhile.

struct Step {
    uint32_t items;      // of the step: row groups by ranges
    uint32_t stages;     // of a range (the last range of a row group may have fewer)
    uint32_t ranges;     // of a row group
    uint32_t m1, m2, d2;  // reciprocals of `ranges` and of d2, the blocks of row groups (step 1) or segments (step 2)
};

struct SmallShared {
    unsigned long long bars[kWarps * kStages];
    Shared s;
    Step step[2];
};

// n / d with m = ceil(2^32 / d): the product is at most one too large.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t m, uint32_t d) {
    const uint32_t q = d == 1 ? n : __umulhi(n, m);
    return q * d > n ? q - 1 : q;
}

__device__ __forceinline__ uint32_t reciprocal(uint32_t d) {
    return static_cast<uint32_t>(((1ull << 32) + d - 1) / d);
}

struct Item {
    uint32_t seg, grp, range;
};

template <int PH>
__device__ __forceinline__ Item item_at(const Step &st, uint32_t it) {
    const uint32_t t = divide(it, st.m1, st.ranges), u = divide(t, st.m2, st.d2), v = t - u * st.d2;
    Item o;
    o.range = it - t * st.ranges;
    o.seg = PH == 1 ? u : v;  // step 1 by segments, step 2 by row groups
    o.grp = PH == 1 ? v : u;
    return o;
}

// `per`: row groups that go together (of one segment).
template <int PH>
__device__ __forceinline__ Step plan_step(const Params &p, const Shared *sm, int per) {
    const Mat &m = mat<PH>(p);
    const uint32_t blocks = static_cast<uint32_t>((m.G + per - 1) / per), segs = static_cast<uint32_t>(sm->n_segs);
    Step st;
    st.stages = min(p.range, m.S);
    st.ranges = (m.S + st.stages - 1) / st.stages;
    st.items = segs * blocks * st.ranges;
    st.d2 = PH == 1 ? blocks : segs;
    st.m1 = reciprocal(st.ranges);
    st.m2 = reciprocal(st.d2);
    return st;
}

// One stage of a warp.
struct Desc {
    uint32_t row16;  // 16-row group of the matrix
    int j;           // first tile
    uint32_t it;     // item of the step
    bool live, last;  // a stage at all; the item's last
};

// The warp's way through a step.
template <int PH>
struct Feed {
    uint32_t it, ahead;  // the item at hand, and the one after it (lane 0 knows)
    uint32_t s, n;       // its next stage, and its stages
    uint32_t row16;
    int j;               // first tile of the item

    __device__ __forceinline__ void take(const Params &p, const SmallShared *sm, uint32_t item) {
        const Step &st = sm->step[PH - 1];
        const Mat &m = mat<PH>(p);
        it = item;
        s = n = 0;
        if (it >= st.items) return;
        const Item at = item_at<PH>(st, it);
        n = min(st.stages, m.S - at.range * st.stages);
        row16 = sm->s.seg_expert[at.seg] * static_cast<uint32_t>(m.G) + at.grp;
        j = static_cast<int>(at.range * st.stages) * kNT;
    }

    __device__ __forceinline__ void start(const Params &p, const SmallShared *sm) {
        const uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);  // (neighbours share metadata)
        take(p, sm, u);
        ahead = u + gridDim.x * kWarps;
    }

    __device__ __forceinline__ Desc next(const Params &p, const SmallShared *sm) {
        if (s == n && n != 0) {
            take(p, sm, __shfl_sync(0xFFFFFFFFu, ahead, 0));
            // (the answer is not needed before the next item)
            if ((threadIdx.x & 31) == 0)
                ahead = 2 * gridDim.x * kWarps + atomicAdd(p.sync + (PH == 1 ? kNext1 : kNext2), 1u);
        }
        Desc d;
        d.live = s < n;
        d.row16 = row16;
        d.j = j + static_cast<int>(s) * kNT;
        d.it = it;
        d.last = s + 1 == n;
        if (d.live) ++s;
        return d;
    }
};

template <int PH>
__device__ __forceinline__ void issue_at(const Params &p, Ring &r, const Desc &d) {
    if ((threadIdx.x & 31) == 0) {
        const uint32_t s = static_cast<uint32_t>(r.issued & 1), st = r.base + s * kStageBytes, bar = r.bars + 8u * s;
        const uint64_t pol = policy_evict_first();
        const Mat &m = mat<PH>(p);
        mbar_expect_tx_s(bar, kStageBytes);
        tma3d(st, &m.tm_raw, 0, d.j, static_cast<int>(d.row16) * kRowsPerGroup, bar, pol);
        tma3d(st + kRawStage, &m.tm_code, 0, d.j, static_cast<int>(d.row16) * kRowsPerGroup, bar, pol);
    }
    ++r.issued;
}

// Metadata of a stage, a lane for each tile row (row = lane % 16, tile = lane /
// 16), as loaded words.
struct Words {
    uint32_t w0, w1, w2;  // version 1: base, esc_off[t], esc_off[t + 1]; version 2: tmeta[t]
    uint32_t ev;          // version 1: the tile row's first escape (read_ahead)
};

template <int V>
__device__ __forceinline__ Words load_words(const Mat &m, const Desc &d) {
    const int lane = threadIdx.x & 31, t = d.j + (lane >> 4);
    Words w = {0u, 0u, 0u, 0u};
    if (d.live && t < m.T) {
        const size_t at = (static_cast<size_t>(d.row16) * kRowsPerGroup + (lane & 15)) * m.T + t;
        if (V == 1) {
            w.w0 = __ldg(static_cast<const uint8_t *>(m.meta) + at);
            w.w1 = __ldg(m.off + at);
            w.w2 = __ldg(m.off + at + 1);
        } else {
            w.w0 = __ldg(static_cast<const uint16_t *>(m.meta) + at);
        }
    }
    return w;
}

// The first escape of each tile row, a stage ahead of its use and a stage after
// the words that say where it is.
template <int V>
__device__ __forceinline__ void read_ahead(const Mat &m, Words &w) {
    if (V == 1 && w.w1 != w.w2 && w.w1 < m.n_esc) w.ev = __ldg(m.esc + w.w1);
}

// The products of one stage: the decoded weights of each 16-column chunk and
// its index go to `multiply`; `refill` is called once the stage's bytes are in
// registers.
template <int V, class Multiply, class Refill>
__device__ __forceinline__ void stage_products(const Params &p, const Mat &m, const Desc &d, const Words &wd,
                                               uint32_t st, Multiply multiply, Refill refill) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, tq = q >> 1, qh = q & 1;
    const uint32_t line = static_cast<uint32_t>(2 * g + tq), rsw = line & 7u, csw = static_cast<uint32_t>(g) & 3u;
    const uint32_t oR = st + line * 128u, oC = st + kRawStage + line * 64u;
    const uint32_t own = V == 1 ? wd.w0 : wd.w0 & 0xFFu;
    if (p.err && own > static_cast<uint32_t>(kMaxBase)) raise_flag(p.err, S12_FLAG_BASE);
    const int src = tq * 16 + g;  // the lane with the words of row g's tile; row g + 8: 8 lanes on
    const uint32_t B2A = __shfl_sync(0xFFFFFFFFu, own, src) * 0x00800080u;
    const uint32_t B2B = __shfl_sync(0xFFFFFFFFu, own, src + 8) * 0x00800080u;
    const bool anyesc = __any_sync(0xFFFFFFFFu, V == 1 ? wd.w1 != wd.w2 : wd.w0 >> 8 != 0u);
    const uint4 cA0 = lds128(oC + (((2u * qh) ^ csw) << 4)), cA1 = lds128(oC + (((2u * qh + 1u) ^ csw) << 4));
    const uint4 cB0 = lds128(oC + (((2u * qh) ^ csw) << 4) + 1024);
    const uint4 cB1 = lds128(oC + (((2u * qh + 1u) ^ csw) << 4) + 1024);
    // escapes of the lane's two tile rows: counts by chunk, stream indexes
    uint32_t nA = 0, nB = 0, iA = 0, iB = 0, limA = 0, limB = 0, knownA = ~0u, knownB = ~0u, evA = 0, evB = 0;
    if (anyesc) {
        // (a lane's first half of a tile row counts from the span's start, the
        // second half back from its end)
        uint32_t sA, eA, sB, eB;
        if (V == 1) {
            sA = __shfl_sync(0xFFFFFFFFu, wd.w1, src);
            eA = __shfl_sync(0xFFFFFFFFu, wd.w2, src);
            sB = __shfl_sync(0xFFFFFFFFu, wd.w1, src + 8);
            eB = __shfl_sync(0xFFFFFFFFu, wd.w2, src + 8);
            evA = __shfl_sync(0xFFFFFFFFu, wd.ev, src);
            evB = __shfl_sync(0xFFFFFFFFu, wd.ev, src + 8);
            knownA = sA;
            knownB = sB;
        } else {
            // row_esc and the counts of the row's earlier tiles
            const int r = static_cast<int>(d.row16) * kRowsPerGroup + g;
            const uint32_t n = wd.w0 >> 8;
            sA = __ldg(m.off + r) + prefix_count_v2(m, r, d.j, q);
            sB = __ldg(m.off + r + 8) + prefix_count_v2(m, r + 8, d.j, q);
            const uint32_t mA = __shfl_sync(0xFFFFFFFFu, n, g), mB = __shfl_sync(0xFFFFFFFFu, n, g + 8);
            sA += tq ? mA : 0u;
            sB += tq ? mB : 0u;
            eA = sA + __shfl_sync(0xFFFFFFFFu, n, src);
            eB = sB + __shfl_sync(0xFFFFFFFFu, n, src + 8);
        }
        if (sA != eA) nA = chunk_counts(cA0, cA1);
        if (sB != eB) nB = chunk_counts(cB0, cB1);
        const uint32_t allA = (nA * 0x01010101u) >> 24, allB = (nB * 0x01010101u) >> 24;
        const uint32_t pairA = allA + __shfl_xor_sync(0xFFFFFFFFu, allA, 1);
        const uint32_t pairB = allB + __shfl_xor_sync(0xFFFFFFFFu, allB, 1);
        if (p.err && d.j + tq < m.T && qh == 0 && (pairA != eA - sA || pairB != eB - sB))
            raise_flag(p.err, S12_FLAG_ESC_COUNT);
        iA = qh ? eA - allA : sA;
        iB = qh ? eB - allB : sB;
        limA = sA <= eA ? min(eA, m.n_esc) : 0u;
        limB = sB <= eB ? min(eB, m.n_esc) : 0u;
    }
    const bool patches = __any_sync(0xFFFFFFFFu, (nA | nB) != 0u);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 rA = lds128(oR + (((4u * qh + c) ^ rsw) << 4));
        const uint4 rB = lds128(oR + (((4u * qh + c) ^ rsw) << 4) + 2048);
        if (c == 3) refill();
        const uint4 kA = c < 2 ? cA0 : cA1, kB = c < 2 ? cB0 : cB1;
        uint32_t wa[8], wb[8];
        decode_pairs(rA.x, rA.y, c & 1 ? kA.z : kA.x, B2A, wa);
        decode_pairs(rA.z, rA.w, c & 1 ? kA.w : kA.y, B2A, wa + 4);
        decode_pairs(rB.x, rB.y, c & 1 ? kB.z : kB.x, B2B, wb);
        decode_pairs(rB.z, rB.w, c & 1 ? kB.w : kB.y, B2B, wb + 4);
        if (patches) {
            const uint32_t hereA = (nA >> (8 * c)) & 0xFFu, hereB = (nB >> (8 * c)) & 0xFFu;
            const uint2 CA = c & 1 ? make_uint2(kA.z, kA.w) : make_uint2(kA.x, kA.y);
            const uint2 CB = c & 1 ? make_uint2(kB.z, kB.w) : make_uint2(kB.x, kB.y);
            if (hereA) patch(wa, CA, iA, limA, knownA, evA, m.esc, p.err);
            if (hereB) patch(wb, CB, iB, limB, knownB, evB, m.esc, p.err);
            iA += hereA;
            iB += hereB;
        }
        multiply(c, wa, wb);
    }
}

// One step by one warp.  d0 and d1 are its first stages (their copies are in
// flight).  False when a wait gave up.
template <int V, int PH>
__device__ __forceinline__ bool small_step(const Params &p, const SmallShared *sm, const uint8_t *x, Ring &rg,
                                           Feed<PH> &feed, Desc d0, Desc d1) {
    const Mat &m = mat<PH>(p);
    const Step &st = sm->step[PH - 1];
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, tq = q >> 1, qh = q & 1;
    const int slots = p.tokens * p.top_k;
    uint32_t half = static_cast<uint32_t>(p.tokens) * 32u;  // (of step 2: the segment's pairs)
    const size_t rows = static_cast<size_t>(m.G) * kRowsPerGroup;  // of an expert
    float acc[4][4] = {};  // four chains of products
    Words w0 = load_words<V>(m, d0);
    read_ahead<V>(m, w0);
    const uint8_t *xl = nullptr;  // the lane's column of x or h
    float *to = nullptr;          // its places of the item's sums, for pairs 2q and 2q + 1
    int pairs = 0;
    bool fresh = true;
    while (d0.live) {
        Words w1 = load_words<V>(m, d1);
        if (fresh) {
            const Item at = item_at<PH>(st, d0.it);
            const int first = sm->s.seg_first[at.seg];
            pairs = sm->s.seg_n[at.seg];
            // (columns past the last pair repeat it; their results are dropped)
            const int i = min(g, pairs - 1);
            if (PH == 1) {
                xl = x + static_cast<size_t>(sm->s.token[first + i]) * 32 + qh * 16;
            } else {
                half = static_cast<uint32_t>(pairs) * 32u;
                xl = x + static_cast<size_t>(first) * p.F * 2 + i * 32 + qh * 16;
            }
            to = (PH == 1 ? p.gu : p.d) + (static_cast<size_t>(at.range) * slots + first + 2 * q) * rows +
                 static_cast<size_t>(at.grp) * kRowsPerGroup + g;
        }
        const uint32_t slot = static_cast<uint32_t>(rg.consumed & 1);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_s(rg.bars + 8u * slot, static_cast<uint32_t>(rg.consumed >> 1) & 1u))) {
            if (lane == 0) give_up(p);
            return false;
        }
        const bool live = d0.j + tq < m.T;  // the lane's tile exists (else zeros from the copy)
        const uint32_t chunk_bytes = 2 * half;
        const size_t at = static_cast<size_t>(d0.j + tq) * 4 * chunk_bytes;
        const ptrdiff_t lo = PH == 2 ? p.lo - p.hi : 0;
        Desc d2;
        d2.live = false;
        auto multiply = [&](int c, const uint32_t (&wa)[8], const uint32_t (&wb)[8]) {
            uint32_t xw[8];
            const uint8_t *src = xl + at + c * chunk_bytes;
            load_x(xw, src, half, live);
            chunk_mma(acc, wa, wb, xw);
            if (PH == 2) {
                load_x(xw, src + lo, half, live);
                chunk_mma(acc, wa, wb, xw);
            }
        };
        auto refill = [&]() {
            // the stage is in registers: hand it back to the copy engine.  (It
            // was read only, which needs no proxy fence.)
            __syncwarp();
            d2 = feed.next(p, sm);
            if (d2.live) issue_at<PH>(p, rg, d2);
            read_ahead<V>(m, w1);
        };
        stage_products<V>(p, m, d0, w0, rg.base + slot * kStageBytes, multiply, refill);
        ++rg.consumed;
        fresh = d0.last;
        if (fresh) {
            // lane (g, q) holds rows g and g + 8 of pairs 2q and 2q + 1
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (2 * q + i < pairs) {
                    __stcg(to + i * rows, acc[0][i] + acc[1][i] + acc[2][i] + acc[3][i]);
                    __stcg(to + i * rows + 8, acc[0][2 + i] + acc[1][2 + i] + acc[2][2 + i] + acc[3][2 + i]);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
        }
        d0 = d1;
        d1 = d2;
        w0 = w1;
    }
    return true;
}

__device__ __forceinline__ float4 shfl4(const float4 &v, int from_xor) {
    return make_float4(__shfl_xor_sync(0xFFFFFFFFu, v.x, from_xor), __shfl_xor_sync(0xFFFFFFFFu, v.y, from_xor),
                       __shfl_xor_sync(0xFFFFFFFFu, v.z, from_xor), __shfl_xor_sync(0xFFFFFFFFu, v.w, from_xor));
}

// Four sums over the ranges of their row group, in order.
__device__ __forceinline__ float4 sum_ranges(const float *src, size_t plane, uint32_t ranges) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (uint32_t c = 0; c < ranges; ++c) {
        const float4 t = __ldcg(reinterpret_cast<const float4 *>(src + c * plane));
        v = make_float4(v.x + t.x, v.y + t.y, v.z + t.z, v.w + t.w);
    }
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Pairs of the list (the slots that are left out are not in it).
__device__ __forceinline__ int used_pairs(const Shared *sm) {
    const int last = sm->n_segs - 1;
    return sm->seg_first[last] + sm->seg_n[last];
}

// h from the sums of step 1: two lanes for a pair's row group (8 f, one piece).
template <bool LARGE>
__device__ __forceinline__ void make_hidden(const Params &p, const Shared *sm, uint32_t ranges) {
    const int slots = p.tokens * p.top_k;
    const uint32_t G = static_cast<uint32_t>(p.up.G), n = used_pairs(sm) * G, half = threadIdx.x & 1;
    const size_t rows = static_cast<size_t>(G) * kRowsPerGroup, plane = static_cast<size_t>(slots) * rows;
    const uint32_t per = blockDim.x / 2;
    for (uint32_t u0 = blockIdx.x * per; u0 < n; u0 += gridDim.x * per) {
        const uint32_t u = min(u0 + threadIdx.x / 2, n - 1);  // (lanes past the end do the last one again)
        const uint32_t pos = u / G, grp = u - pos * G;
        const float *src = p.gu + pos * rows + static_cast<size_t>(grp) * kRowsPerGroup + 4 * half;
        const float4 gt = sum_ranges(src, plane, ranges), up = sum_ranges(src + 8, plane, ranges);
        auto h = [](float g, float t) { return g / (1.f + expf(-g)) * t; };
        const float4 a = make_float4(h(gt.x, up.x), h(gt.y, up.y), h(gt.z, up.z), h(gt.w, up.w));
        const float4 b = shfl4(a, 1);
        // one piece, in the order 0 4 1 5 2 6 3 7; the first lane stores the
        // high parts, the second the low ones
        const float4 l = half ? b : a, r = half ? a : b;
        const float f[8] = {l.x, r.x, l.y, r.y, l.z, r.z, l.w, r.w};
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
            if (half) {
                const float r0 = f[2 * i] - __uint_as_float(v[i] << 16);
                const float r1 = f[2 * i + 1] - __uint_as_float(v[i] & 0xFFFF0000u);
                // (an infinite h has no rest)
                v[i] = pack_bf16(fabsf(r0) < 3.4e38f ? r0 : 0.f, fabsf(r1) < 3.4e38f ? r1 : 0.f);
            }
        }
        const int seg = sm->segment[pos], first = sm->seg_first[seg];
        const size_t o = static_cast<size_t>(first) * p.F * 2 +
                         piece_of<LARGE>(static_cast<int>(grp), sm->seg_n[seg], static_cast<int>(pos) - first);
        *reinterpret_cast<uint4 *>((half ? p.lo : p.hi) + o) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// y from the sums of step 2: a lane for four values of a token.
__device__ __forceinline__ void make_y(const Params &p, const Shared *sm, uint32_t ranges) {
    const int slots = p.tokens * p.top_k;
    const uint32_t per = static_cast<uint32_t>(p.H) / 4, n = p.tokens * per;
    const size_t rows = static_cast<size_t>(p.H), plane = static_cast<size_t>(slots) * rows;
    for (uint32_t u = blockIdx.x * blockDim.x + threadIdx.x; u < n; u += gridDim.x * blockDim.x) {
        const uint32_t t = u / per, c = (u - t * per) * 4;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.top_k; ++s) {
            const int i = static_cast<int>(t) * p.top_k + s;
            if (sm->expert[i] < 0) continue;
            const float4 v = sum_ranges(p.d + sm->place[i] * rows + c, plane, ranges);
            const float w = sm->weight[i];
            y = make_float4(fmaf(w, v.x, y.x), fmaf(w, v.y, y.y), fmaf(w, v.z, y.z), fmaf(w, v.w, y.w));
        }
        const size_t o = static_cast<size_t>(t) * p.H + c;
        put_y(p, o, y.x);
        put_y(p, o + 1, y.y);
        put_y(p, o + 2, y.z);
        put_y(p, o + 3, y.w);
    }
}

template <int V>
__global__ void __launch_bounds__(kThreads, 1) moe_small_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    SmallShared *sm = reinterpret_cast<SmallShared *>(base + kRingBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Ring rg;
    rg.bars = smem_addr(sm->bars) + static_cast<uint32_t>(warp) * kStages * 8u;
    rg.base = smem_addr(base) + static_cast<uint32_t>(warp) * kStages * kStageBytes;
    rg.issued = rg.consumed = 0;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init_s(rg.bars + 8u * s, 1);
        fence_barrier_init();
    }
    // x and the scores: a few tokens by every CTA for itself (x behind the
    // lists, the scores where the ring will be), more by the grid
    const uint8_t *x = p.xp;
    const double *scores = p.scores;
    bool ok = true;
    if (p.local) {
        uint8_t *xs = base + kRingBytes + ((sizeof(SmallShared) + 15) & ~size_t(15));
        double *own = reinterpret_cast<double *>(base);
        pack_x(p, xs, threadIdx.x, kThreads);
        if (!p.ids_in) score<1, 1>(p, own, warp, kWarps);
        x = xs;
        scores = own;
        __syncthreads();
    } else {
        pack_x(p, p.xp, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
        if (!p.ids_in) {
            const int u0 = warp * gridDim.x + blockIdx.x, step = gridDim.x * kWarps;
            if (p.tokens >= 8 && p.tokens * p.experts >= 1024)
                score<4, 4>(p, p.scores, u0, step);
            else
                score<1, 1>(p, p.scores, u0, step);
        }
        ok = grid_meet(p, &sm->s, kBarRoute);
    }
    if (ok) {
        route(p, &sm->s, scores);
        if (sm->s.n_segs == 0) {
            // no token goes anywhere
            const size_t n = static_cast<size_t>(p.tokens) * p.H;
            for (size_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) put_y(p, i, 0.f);
        } else {
            if (threadIdx.x == 0) sm->step[0] = plan_step<1>(p, &sm->s, 1);
            if (threadIdx.x == 32) sm->step[1] = plan_step<2>(p, &sm->s, 1);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the scores give way to copies
            __syncthreads();
            Feed<1> f1;
            f1.start(p, sm);
            Desc d0 = f1.next(p, sm);
            if (d0.live) issue_at<1>(p, rg, d0);
            Desc d1 = f1.next(p, sm);
            if (d1.live) issue_at<1>(p, rg, d1);
            ok = small_step<V, 1>(p, sm, x, rg, f1, d0, d1);
            // the first copies of step 2 run while the grid meets
            Feed<2> f2;
            f2.start(p, sm);
            if (ok) {
                d0 = f2.next(p, sm);
                if (d0.live) issue_at<2>(p, rg, d0);
                d1 = f2.next(p, sm);
                if (d1.live) issue_at<2>(p, rg, d1);
            }
            if (grid_meet(p, &sm->s, kBarSums)) {
                make_hidden<false>(p, &sm->s, sm->step[0].ranges);
                if (grid_meet(p, &sm->s, kBarHidden)) {
                    if (ok) small_step<V, 2>(p, sm, p.hi, rg, f2, d0, d1);
                    if (grid_meet(p, &sm->s, kBarDown)) make_y(p, &sm->s, sm->step[1].ranges);
                }
            }
        }
    }
    // copies that a wait left in flight land
    if (lane == 0)
        for (int k = rg.consumed; k < rg.issued; ++k)
            mbar_wait_s(rg.bars + 8u * (k & 1), static_cast<uint32_t>(k >> 1) & 1u);
    leave(p, &sm->s);
}

// ---------------------------------------------------------------------------
// Many pairs an expert: up to 64 share a read of its weights.
//
// A unit is a block of 128 rows of a segment's expert by a range of columns:
// D[row][pair] += W[row][k] * x[pair][k] on the tcgen05 tensor cores, 128 columns
// (a tile of each row) at a time.  W is the product's left side and is kept in
// TMEM, where the threads that decode it write it from registers: a row of the
// tile is a lane of TMEM.  (Through mma.sync, every warp reads all of x from
// shared memory for 16 rows of weights: 64 tokens of 8 experts of 14336 x 4096
// took 815 us, against 507.)  x and h are copied to shared memory as the product
// wants them (128-byte swizzle).  h's high and low parts are one product of twice
// the width, whose halves are added where the sums are stored: a product takes as
// long for 64 columns as for 32 (two in a row: 607 us, one: 573).
//
// Warp 0 claims units and copies weights and x into a ring of stages, a tile
// each; warp 1 issues the products; sixteen warps decode, eight to a tile, which
// holds a stage half as long as four do; two warps read a unit's metadata ahead,
// a row's tiles side by side (read by the thread that has the row, every word is
// a sector of its own, and the loads took a fifth of the decoding warps' time).
// The eight warps that had a unit's last tile store its sums, while the others
// decode the next unit's tiles (there are two places for sums).  Every wait is
// for something of an earlier tile, or of an earlier part of the same tile, so
// the tiles' order shows that all end.  Units come from a counter of the grid as
// items do above; the first weights of a step are copied while the grid meets.

constexpr int kGroups = 2, kGroupWarps = 8;  // warps that decode a tile: four, by rows, for each half of its columns
constexpr int kPlaces = 2 * kGroups;         // of decoded weights
constexpr int kDecodeWarps = kGroups * kGroupWarps, kMetaWarps = 2;
constexpr int kLargeThreads = 32 * (2 + kDecodeWarps + kMetaWarps);
constexpr int kUnitTiles = 16;   // tiles of a unit at most
constexpr int kAhead = 3;        // units that a CTA knows in advance
constexpr int kUnits = 24;       // the queue: no warp is more than 16 tiles behind the copies
constexpr int kMaxRing = 8;      // stages
constexpr int kBlockRows = 128;
constexpr uint32_t kTileRaw = kBlockRows * kTile, kTileBytes = kTileRaw + kTileRaw / 2;
constexpr uint32_t kSumCols = 2 * kSegLarge, kPlaceCols = kTile / 2;  // of TMEM: sums, decoded weights
constexpr uint32_t kTmemCols = 512;
static_assert(2 * kSumCols + kPlaces * kPlaceCols <= kTmemCols, "two places for sums, two for weights a group");

struct LargeShared {
    Shared s;
    Step step[2];
    unsigned long long queue[2][kUnits];  // ordinal << 32 | unit
    // mbarriers, by step
    unsigned long long weights[2][kMaxRing], x[2][kMaxRing], empty[2][kMaxRing];  // stages: copied, free
    unsigned long long decoded[2][kPlaces], used[2][kPlaces];                     // places of decoded weights
    unsigned long long sums[2][kGroups], stored[2][2];  // a group's last tile multiplied; places of sums free
    unsigned long long read[2][2], spent[2][2];          // a unit's metadata
    unsigned long long done[2];                          // all products of the step
    uint2 meta[2][kUnitTiles * (kBlockRows + 1)];        // of the tile rows of two units
    uint32_t tally[kPlaces][kBlockRows];                 // escapes found in a tile row by the half done first
    uint32_t tmem, abort;
};

struct Unit {
    uint32_t seg, range, block;
    int j, n;  // first tile; tiles (0: no more units)
};

// The CTA's unit `ord`; false when it is not known yet.
template <int PH>
__device__ __forceinline__ bool peek(const Params &p, const LargeShared *sm, uint32_t ord, Unit &u) {
    const Step &st = sm->step[PH - 1];
    const unsigned long long e = *const_cast<const volatile unsigned long long *>(&sm->queue[PH - 1][ord % kUnits]);
    if (e >> 32 != ord) return false;
    const uint32_t it = static_cast<uint32_t>(e);
    u = Unit{0u, 0u, 0u, 0, 0};
    if (it >= st.items) return true;
    const Item i = item_at<PH>(st, it);
    const int per = static_cast<int>(st.stages) * kNT;
    u.seg = i.seg;
    u.range = i.range;
    u.block = i.grp;
    u.j = static_cast<int>(i.range) * per;
    u.n = min(per, mat<PH>(p).T - u.j);
    return true;
}

// The same, waiting for it (with a limit; then there are no more units).
template <int PH>
__device__ __forceinline__ Unit unit_at(const Params &p, LargeShared *sm, uint32_t ord) {
    Unit u;
    if (peek<PH>(p, sm, ord, u)) return u;
    const long long t0 = clock64();
    while (!peek<PH>(p, sm, ord, u)) {
        const bool late = clock64() - t0 > kWaitCycles;
        if (late) {
            sm->abort = 1u;
            give_up(p);
        }
        if (late || *const_cast<volatile uint32_t *>(&sm->abort)) return Unit{0u, 0u, 0u, 0, 0};
    }
    return u;
}

__device__ __forceinline__ bool lost(const Params &p, LargeShared *sm) {
    sm->abort = 1u;
    give_up(p);
    return false;
}

// Pairs of a product for n that there are (its columns, two for each pair of h,
// are a multiple of 16); the rest are whatever shared memory holds, and their sums
// are not read.  Stages are as long as the largest segment needs, and their number
// tells: with h in eights, 33 to 40 pairs leave four stages instead of three (64
// tokens, one expert with 40 of the pairs: 509 us; with 41, and three stages, 554).
template <int PH>
__device__ __forceinline__ uint32_t product_pairs(uint32_t n) {
    constexpr uint32_t kUp = 16 / PH - 1;
    return (n + kUp) & ~kUp;
}

struct Stages {
    uint32_t base, bytes, n;
};

template <int PH>
__device__ __forceinline__ Stages stages_of(const Params &p, const LargeShared *sm, uint32_t base) {
    Stages s;
    s.base = base;
    s.bytes = kTileBytes + product_pairs<PH>(static_cast<uint32_t>(sm->s.most)) * 256u * PH;  // (h: two planes)
    s.n = min(static_cast<uint32_t>(kMaxRing), p.pool / s.bytes);
    return s;
}

template <int PH>
__device__ __forceinline__ uint32_t row_of(const Params &p, const LargeShared *sm, const Unit &u) {
    return sm->s.seg_expert[u.seg] * static_cast<uint32_t>(mat<PH>(p).G) * kRowsPerGroup + u.block * kBlockRows;
}

template <int PH>
__device__ __forceinline__ void copy_weights(const Params &p, LargeShared *sm, const Stages &rs, uint32_t slot,
                                             uint32_t row, int j) {
    const Mat &m = mat<PH>(p);
    const uint32_t st = rs.base + slot * rs.bytes, bar = smem_addr(&sm->weights[PH - 1][slot]);
    const uint64_t pol = policy_evict_first();
    mbar_expect_tx_s(bar, kTileBytes);
    tma3d(st, &m.tm_raw, 0, j, static_cast<int>(row), bar, pol);
    tma3d(st + kTileRaw, &m.tm_code, 0, j, static_cast<int>(row), bar, pol);
}

// What one thread of warp 0 has copied in a step: tiles of weights, of x.
struct Copied {
    uint32_t weights, x;
};

// Weights of the first tiles, as far as the ring goes.
template <int PH>
__device__ __forceinline__ Copied copy_first(const Params &p, LargeShared *sm, uint32_t base) {
    const Stages rs = stages_of<PH>(p, sm, base);
    Copied c = {0u, 0u};
    for (uint32_t ord = 0; ord < kAhead; ++ord) {
        const Unit u = unit_at<PH>(p, sm, ord);
        if (u.n == 0) break;
        const uint32_t row = row_of<PH>(p, sm, u);
        for (int t = 0; t < u.n && c.weights < rs.n; ++t) copy_weights<PH>(p, sm, rs, c.weights++, row, u.j + t);
    }
    return c;
}

template <int PH>
__device__ __forceinline__ void copy_step(const Params &p, LargeShared *sm, uint32_t base, Copied &c) {
    const Stages rs = stages_of<PH>(p, sm, base);
    const size_t line = static_cast<size_t>(mat<PH>(p).T) * kTile * 2;  // bytes of a pair's x
    uint32_t slot = 0, parity = 1;
    bool ok = true;
    for (uint32_t ord = 0; ok; ++ord) {
        const Unit u = unit_at<PH>(p, sm, ord);
        if (u.n == 0) break;
        const uint32_t claimed = atomicAdd(p.sync + (PH == 1 ? kNext1 : kNext2), 1u) + kAhead * gridDim.x;
        const uint32_t row = row_of<PH>(p, sm, u), n = sm->s.seg_n[u.seg], atom = product_pairs<PH>(n) * 128u;
        const size_t off = sm->s.seg_first[u.seg] * line;
        for (int t = 0; t < u.n; ++t) {
            ok = mbar_wait_s(smem_addr(&sm->empty[PH - 1][slot]), parity);
            if (!ok) break;
            if (c.x == c.weights) {
                copy_weights<PH>(p, sm, rs, slot, row, u.j + t);
                ++c.weights;
            }
            const uint32_t bar = smem_addr(&sm->x[PH - 1][slot]), dst = rs.base + slot * rs.bytes + kTileBytes;
            const size_t src = off + static_cast<size_t>(u.j + t) * n * 256u;
            mbar_expect_tx_s(bar, PH * n * 256u);
#pragma unroll
            for (int i = 0; i < 2 * PH; ++i)  // 64 columns of a plane
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                        dst + ((i & 1) * PH + (i >> 1)) * atom),
                    "l"((PH == 1 ? p.xp : i >= 2 ? p.lo : p.hi) + src + (i & 1) * n * 128u), "r"(n * 128u), "r"(bar)
                    : "memory");
            ++c.x;
            if (++slot == rs.n) {
                slot = 0;
                parity ^= 1u;
            }
        }
        const uint32_t next = ord + kAhead;
        *const_cast<volatile unsigned long long *>(&sm->queue[PH - 1][next % kUnits]) =
            (static_cast<unsigned long long>(next) << 32) | claimed;
    }
    // the stages are another step's next
    for (uint32_t i = c.x > rs.n ? c.x - rs.n : 0; ok && i < c.x; ++i)
        ok = mbar_wait_s(smem_addr(&sm->empty[PH - 1][i % rs.n]), (i / rs.n) & 1u);
    if (!ok) lost(p, sm);
}

// Every copy of a step lands (after a wait that gave up; else they have).
template <int PH>
__device__ __forceinline__ void land(const Params &p, LargeShared *sm, const Copied &c) {
    const uint32_t n = stages_of<PH>(p, sm, 0u).n;
    for (uint32_t i = c.weights > n ? c.weights - n : 0; i < c.weights; ++i)
        mbar_wait_s(smem_addr(&sm->weights[PH - 1][i % n]), (i / n) & 1u);
    for (uint32_t i = c.x > n ? c.x - n : 0; i < c.x; ++i)
        mbar_wait_s(smem_addr(&sm->x[PH - 1][i % n]), (i / n) & 1u);
}

// D[tmem] (+)= A[tmem] * B[smem] for one 128 x N x 16 step, BF16 -> FP32.
__device__ __forceinline__ void umma_weights(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// BF16 x BF16 -> FP32, both operands K-major, M = 128, N = n.
__device__ __forceinline__ uint32_t product_desc(uint32_t n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((kBlockRows >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// The value of lane 0, which makes it one for the warp in the compiler's eyes.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// A step by the warp that issues the products.  It goes through the step as a
// warp, and one lane issues: the operands of a product are then the warp's own
// (by one lane alone, each was handed over anew: 122 cycles a product).
template <int PH>
__device__ __forceinline__ void multiply_step(const Params &p, LargeShared *sm, uint32_t base, uint32_t tmem) {
    const Stages rs = stages_of<PH>(p, sm, base);
    const uint32_t stages = uniform(rs.n), bytes = uniform(rs.bytes), xs = uniform(rs.base) + kTileBytes;
    const uint32_t tm = uniform(tmem);
    uint32_t slot = 0, parity = 0, place = 0, pparity = 0;
    bool ok = true;
    for (uint32_t ord = 0; ok; ++ord) {
        const Unit u = unit_at<PH>(p, sm, ord);
        const uint32_t tiles = uniform(static_cast<uint32_t>(u.n));
        if (tiles == 0) break;
        const uint32_t n = PH * uniform(product_pairs<PH>(sm->s.seg_n[u.seg])), idesc = product_desc(n);
        const uint32_t sums = tm + (ord & 1u) * kSumCols;
        ok = mbar_wait_s(smem_addr(&sm->stored[PH - 1][ord & 1u]), ((ord >> 1) & 1u) ^ 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        for (uint32_t t = 0; ok && t < tiles; ++t) {
            ok = mbar_wait_s(smem_addr(&sm->x[PH - 1][slot]), parity) &&
                 mbar_wait_s(smem_addr(&sm->decoded[PH - 1][place]), pparity);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc::tc_fence_after();
            const uint64_t x = tc::smem_desc_sw128(xs + slot * bytes);
            const uint32_t wa = tm + 2u * kSumCols + place * kPlaceCols;
            if (elect_one()) {
#pragma unroll
                for (uint32_t k = 0; k < kTile / 16; ++k)  // (the descriptor's address is in 16 bytes)
                    umma_weights(sums, wa + k * 8, x + ((k >> 2) * n * 8u + (k & 3) * 2u), idesc,
                                 k == 0 ? t != 0 : 1u);
                tc::umma_commit(smem_addr(&sm->used[PH - 1][place]));
                tc::umma_commit(smem_addr(&sm->empty[PH - 1][slot]));
                if (t + 1 == tiles) tc::umma_commit(smem_addr(&sm->sums[PH - 1][place % kGroups]));
            }
            __syncwarp();
            if (++slot == stages) {
                slot = 0;
                parity ^= 1u;
            }
            if (++place == kPlaces) {
                place = 0;
                pparity ^= 1u;
            }
        }
    }
    if (!ok) lost(p, sm);
    // every product is over before its memory serves something else
    if (elect_one()) tc::umma_commit(smem_addr(&sm->done[PH - 1]));
    __syncwarp();
    mbar_wait_s(smem_addr(&sm->done[PH - 1]), 0);
}

// What decoding a tile row takes: x: its first escape's place; y: base | number
// of escapes << 8 | the first escape << 16.  (No tile row has more than 128;
// above 254 the metadata is wrong, as where it ends before it starts: 255.)
__device__ __forceinline__ uint2 meta_word(uint32_t base, uint32_t from, uint32_t end, uint32_t ev) {
    const uint32_t n = from <= end ? min(end - from, 254u) : 255u;
    return make_uint2(from, (base & 0xFFu) | (n << 8) | (ev << 16));
}

// A step by a warp that reads metadata: half of a unit's rows, two at a time, a
// lane for each of 16 tiles.
template <int V, int PH>
__device__ __forceinline__ void meta_step(const Params &p, LargeShared *sm) {
    constexpr int kRows = kBlockRows / kMetaWarps, kBatch = 8;
    const Mat &m = mat<PH>(p);
    const int lane = threadIdx.x & 31, t = lane & 15;
    const int r0 = (static_cast<int>(threadIdx.x >> 5) - 2 - kDecodeWarps) * kRows + (lane >> 4);
    for (uint32_t ord = 0;; ++ord) {
        const Unit u = unit_at<PH>(p, sm, ord);
        if (u.n == 0) break;
        const uint32_t d = ord & 1u;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_s(smem_addr(&sm->spent[PH - 1][d]), ((ord >> 1) & 1u) ^ 1u))) {
            lost(p, sm);
            return;
        }
        const size_t row = row_of<PH>(p, sm, u);
#pragma unroll 1
        for (int i0 = 0; i0 < kRows; i0 += 2 * kBatch) {
            uint32_t base[kBatch], from[kBatch], end[kBatch], ev[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const size_t r = row + r0 + i0 + 2 * b, at = r * m.T + u.j + t;
                base[b] = from[b] = end[b] = ev[b] = 0u;
                if (V == 1) {
                    if (t < u.n) {
                        base[b] = __ldg(static_cast<const uint8_t *>(m.meta) + at);
                        from[b] = __ldg(m.off + at);
                        end[b] = __ldg(m.off + at + 1);
                    }
                } else {
                    // row_esc and the counts of the row's earlier tiles
                    const uint16_t *tm = static_cast<const uint16_t *>(m.meta) + r * m.T;
                    for (int k = t; k < u.j; k += 16) from[b] += __ldg(tm + k) >> 8;
                    if (t < u.n) base[b] = __ldg(tm + u.j + t);
                    end[b] = __ldg(m.off + r);
                }
            }
            if (V == 2) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    uint32_t before = from[b], upto = base[b] >> 8;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) {
                        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o, 16);
                        if (t >= o) upto += v;
                    }
                    end[b] += before + upto;
                    from[b] = end[b] - (base[b] >> 8);
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (from[b] < end[b] && from[b] < m.n_esc) ev[b] = __ldg(m.esc + from[b]);
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                sm->meta[d][t * (kBlockRows + 1) + r0 + i0 + 2 * b] = meta_word(base[b], from[b], end[b], ev[b]);
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(smem_addr(&sm->read[PH - 1][d]));
    }
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[2][8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0][0]), "r"(v[0][1]), "r"(v[0][2]), "r"(v[0][3]), "r"(v[0][4]), "r"(v[0][5]), "r"(v[0][6]), "r"(v[0][7]),
        "r"(v[1][0]), "r"(v[1][1]), "r"(v[1][2]), "r"(v[1][3]), "r"(v[1][4]), "r"(v[1][5]), "r"(v[1][6]), "r"(v[1][7])
        : "memory");
}

// Half of the thread's row (r of the block) of a tile: 64 weights to its lane of
// TMEM.  The first half counts the row's escapes up from the first, the second
// down from the last; `tally` brings the two numbers together.
template <bool UP>
__device__ __forceinline__ void decode_half(const Params &p, const Mat &m, uint32_t st, uint32_t to, int r, uint2 w,
                                            uint32_t *tally) {
    const uint32_t base = w.y & 0xFFu, count = (w.y >> 8) & 0xFFu;
    if (p.err && base > static_cast<uint32_t>(kMaxBase)) raise_flag(p.err, S12_FLAG_BASE);
    const uint32_t raw = st + static_cast<uint32_t>(r) * 128u, rsw = static_cast<uint32_t>(r) & 7u;
    const uint32_t code = st + kTileRaw + static_cast<uint32_t>(r) * 64u, csw = (static_cast<uint32_t>(r) >> 1) & 3u;
    const uint32_t B2 = base * 0x00800080u, marks = count ? 0x88888888u : 0u;
    const uint32_t n = count == 255u ? 0u : count, limit = min(w.x + n, m.n_esc);
    const uint32_t first = UP ? w.x : w.x + n - 1u;
    uint32_t idx = first;
    // the exact values of a word's escapes (most rows with any have one)
    auto exact = [&](uint32_t mm, uint32_t *v) {
        while (mm) {
            const uint32_t j = static_cast<uint32_t>(UP ? __ffs(static_cast<int>(mm)) - 1 : 31 - __clz(mm)) >> 2;
            mm &= ~(8u << (4u * j));
            uint32_t value = 0;
            if (idx - w.x < n && idx < limit)
                value = idx == w.x ? w.y >> 16 : __ldg(m.esc + idx);
            else
                raise_flag(p.err, S12_FLAG_ESC_RANGE);
            idx += UP ? 1u : ~0u;
            const uint32_t sel = j & 4u ? 0x5410u : 0x3254u;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) v[i] = prmt(v[i], value, i == (j & 3u) ? sel : 0x3210u);
        }
    };
#pragma unroll 1
    for (uint32_t i = 0; i < 2; ++i) {  // 32 columns
        const uint32_t c = UP ? i : 3u - i;
        const uint4 k = lds128(code + ((c ^ csw) << 4));
        const uint4 a = lds128(raw + (((2u * c) ^ rsw) << 4)), b = lds128(raw + (((2u * c + 1u) ^ rsw) << 4));
        uint32_t v[2][8];
        decode_pairs(a.x, a.y, k.x, B2, v[0]);
        decode_pairs(a.z, a.w, k.y, B2, v[0] + 4);
        decode_pairs(b.x, b.y, k.z, B2, v[1]);
        decode_pairs(b.z, b.w, k.w, B2, v[1] + 4);
        const uint32_t m0 = escape_nibbles(k.x) & marks, m1 = escape_nibbles(k.y) & marks;
        const uint32_t m2 = escape_nibbles(k.z) & marks, m3 = escape_nibbles(k.w) & marks;
        if (m0 | m1 | m2 | m3) {
            if (UP) {
                exact(m0, v[0]);
                exact(m1, v[0] + 4);
                exact(m2, v[1]);
                exact(m3, v[1] + 4);
            } else {
                exact(m3, v[1] + 4);
                exact(m2, v[1]);
                exact(m1, v[0] + 4);
                exact(m0, v[0]);
            }
        }
        __syncwarp();
        tmem_st16(to + c * 16u, v);
    }
    if (count && p.err) {
        const uint32_t found = UP ? idx - first : first - idx;
        const uint32_t other = atomicAdd(tally, 0x10000u | found);
        if (other) {
            if ((other & 0xFFFFu) + found != count) raise_flag(p.err, S12_FLAG_ESC_COUNT);
            *tally = 0u;
        }
    }
}

// A step by one of the warps that decode: every other tile, across units.
template <int PH>
__device__ __forceinline__ void decode_step(const Params &p, LargeShared *sm, uint32_t base, uint32_t tmem) {
    const Mat &m = mat<PH>(p);
    const Stages rs = stages_of<PH>(p, sm, base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = (warp - 2) / kGroupWarps, quad = warp & 3;
    const int r = quad * 32 + lane, half = ((warp - 2) >> 2) & 1;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;  // TMEM lanes 32 quad on are this warp's
    uint32_t slot = static_cast<uint32_t>(group), parity = 0, sparity = 0;
    uint32_t place = static_cast<uint32_t>(group), pparity = 0;
    int k = group;  // the next tile, counted from the unit's first
    for (uint32_t ord = 0;; ++ord) {
        const Unit u = unit_at<PH>(p, sm, ord);
        if (u.n == 0) break;
        const uint32_t d = ord & 1u;
        bool ok = mbar_wait_s(smem_addr(&sm->read[PH - 1][d]), (ord >> 1) & 1u);
        for (; k < u.n; k += kGroups) {
            while (slot >= rs.n) {
                slot -= rs.n;
                parity ^= 1u;
            }
            // (a wait tells a phase from its neighbours only, and this group meets a
            // stage now and then: that its place was used shows that the stage's tile
            // before last is done, that the stage was free that the last one is)
            ok = ok && mbar_wait_s(smem_addr(&sm->used[PH - 1][place]), pparity ^ 1u) &&
                 mbar_wait_s(smem_addr(&sm->empty[PH - 1][slot]), parity ^ 1u) &&
                 mbar_wait_s(smem_addr(&sm->weights[PH - 1][slot]), parity);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                lost(p, sm);
                return;
            }
            tc::tc_fence_after();
            const uint2 w = sm->meta[d][k * (kBlockRows + 1) + r];
            const uint32_t st = rs.base + slot * rs.bytes, to = tmem + lanes + 2u * kSumCols + place * kPlaceCols;
            if (half)
                decode_half<false>(p, m, st, to, r, w, &sm->tally[place][r]);
            else
                decode_half<true>(p, m, st, to, r, w, &sm->tally[place][r]);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                tc::bar_arrive(smem_addr(&sm->decoded[PH - 1][place]));
                tc::bar_arrive(smem_addr(&sm->empty[PH - 1][slot]));
            }
            slot += kGroups;
            place += kGroups;
            if (place >= kPlaces) {
                place -= kPlaces;
                pparity ^= 1u;
            }
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            lost(p, sm);
            return;
        }
        if (lane == 0) tc::bar_arrive(smem_addr(&sm->spent[PH - 1][d]));
        k -= u.n;
        if (k == kGroups - 1) {
            // the unit's last tile was this group's: its sums, a lane of TMEM for each row
            const int pairs = sm->s.seg_n[u.seg];
            const size_t rows = static_cast<size_t>(m.G) * kRowsPerGroup;  // of an expert
            const uint32_t sums = tmem + lanes + d * kSumCols;
            float *to = (PH == 1 ? p.gu : p.d) +
                        (static_cast<size_t>(u.range) * (p.tokens * p.top_k) + sm->s.seg_first[u.seg]) * rows +
                        static_cast<size_t>(u.block) * kBlockRows + r;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_s(smem_addr(&sm->sums[PH - 1][group]), sparity))) {
                lost(p, sm);
                return;
            }
            sparity ^= 1u;
            tc::tc_fence_after();
            for (int c = 8 * half; c < pairs; c += 16) {
                uint32_t v[PH][2][4];  // (of the high and the low part of h)
#pragma unroll
                for (int i = 0; i < 2 * PH; ++i)
                    tc::tmem_ld4(sums + (i >> 1) * product_pairs<PH>(pairs) + c + 4 * (i & 1), v[i >> 1][i & 1]);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float sum = __uint_as_float(v[0][i >> 2][i & 3]);
                    if (PH == 2) sum += __uint_as_float(v[PH - 1][i >> 2][i & 3]);
                    if (c + i < pairs) __stcg(to + (c + i) * rows, sum);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(smem_addr(&sm->stored[PH - 1][d]));
        }
    }
}

// The x that this thread wrote goes to copies (by other SMs, after the grid met).
__device__ __forceinline__ void fence_for_copies() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <int V>
__global__ void __launch_bounds__(kLargeThreads, 1) moe_large_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    LargeShared *sm = reinterpret_cast<LargeShared *>(base);
    const uint32_t stages = smem_addr(base) + ((sizeof(LargeShared) + 1023) & ~size_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            for (int s = 0; s < kMaxRing; ++s) {
                mbar_init_s(smem_addr(&sm->weights[i][s]), 1);
                mbar_init_s(smem_addr(&sm->x[i][s]), 1);
                mbar_init_s(smem_addr(&sm->empty[i][s]), kGroupWarps + 1);  // the warps that decode it, the products
            }
            for (int k = 0; k < kPlaces; ++k) {
                mbar_init_s(smem_addr(&sm->decoded[i][k]), kGroupWarps);
                mbar_init_s(smem_addr(&sm->used[i][k]), 1);
            }
            for (int g = 0; g < kGroups; ++g) mbar_init_s(smem_addr(&sm->sums[i][g]), 1);
            for (int d = 0; d < 2; ++d) {
                mbar_init_s(smem_addr(&sm->stored[i][d]), kGroupWarps);
                mbar_init_s(smem_addr(&sm->read[i][d]), kMetaWarps);
                mbar_init_s(smem_addr(&sm->spent[i][d]), kDecodeWarps);
            }
            mbar_init_s(smem_addr(&sm->done[i]), 1);
        }
        sm->abort = 0u;
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i < kPlaces * kBlockRows; i += blockDim.x) (&sm->tally[0][0])[i] = 0u;
    if (warp == 1) {
        tc::tmem_alloc(smem_addr(&sm->tmem), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sm->tmem;
    bool ok = true;
    if (!p.ids_in) {
        constexpr int kWarpsHere = kLargeThreads / 32;
        const int u0 = warp * gridDim.x + blockIdx.x, step = gridDim.x * kWarpsHere;
        if (p.tokens * p.experts >= 1024)
            score<4, 4>(p, p.scores, u0, step);
        else
            score<1, 1>(p, p.scores, u0, step);
        ok = grid_meet(p, &sm->s, kBarRoute);
    }
    if (ok) {
        route(p, &sm->s, p.scores);
        if (sm->s.n_segs == 0) {
            // no token goes anywhere
            const size_t n = static_cast<size_t>(p.tokens) * p.H;
            for (size_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) put_y(p, i, 0.f);
        } else {
            constexpr int kGroupsOfBlock = kBlockRows / kRowsPerGroup;
            if (threadIdx.x == 0) sm->step[0] = plan_step<1>(p, &sm->s, kGroupsOfBlock);
            if (threadIdx.x == 32) sm->step[1] = plan_step<2>(p, &sm->s, kGroupsOfBlock);
            if (threadIdx.x >= 64 && threadIdx.x < 64 + 2 * kUnits) {
                const uint32_t k = (threadIdx.x - 64) % kUnits;
                sm->queue[(threadIdx.x - 64) / kUnits][k] =
                    k < kAhead ? (static_cast<unsigned long long>(k) << 32) | (blockIdx.x + k * gridDim.x) : ~0ull;
            }
            pack_sorted(p, &sm->s, used_pairs(&sm->s));
            fence_for_copies();
            __syncthreads();
            Copied c1 = {0u, 0u}, c2 = {0u, 0u};
            const bool copies = warp == 0 && lane == 0, multiplies = warp == 1;
            // the first weights are copied while the grid meets
            if (copies) c1 = copy_first<1>(p, sm, stages);
            __syncwarp();
            if (grid_meet(p, &sm->s, kBarPack)) {
                fence_for_copies();
                if (copies) {
                    copy_step<1>(p, sm, stages, c1);
                    if (!*const_cast<volatile uint32_t *>(&sm->abort)) c2 = copy_first<2>(p, sm, stages);
                } else if (multiplies) {
                    multiply_step<1>(p, sm, stages, tmem);
                } else if (warp >= 2 + kDecodeWarps) {
                    meta_step<V, 1>(p, sm);
                } else if (warp >= 2) {
                    decode_step<1>(p, sm, stages, tmem);
                }
                __syncwarp();
                if (grid_meet(p, &sm->s, kBarSums)) {
                    make_hidden<true>(p, &sm->s, sm->step[0].ranges);
                    fence_for_copies();
                    if (grid_meet(p, &sm->s, kBarHidden)) {
                        fence_for_copies();
                        const bool on = *const_cast<volatile uint32_t *>(&sm->abort) == 0u;
                        __syncthreads();
                        if (on) {
                            if (copies) {
                                copy_step<2>(p, sm, stages, c2);
                            } else if (multiplies) {
                                multiply_step<2>(p, sm, stages, tmem);
                            } else if (warp >= 2 + kDecodeWarps) {
                                meta_step<V, 2>(p, sm);
                            } else if (warp >= 2) {
                                decode_step<2>(p, sm, stages, tmem);
                            }
                        }
                        __syncwarp();
                        if (grid_meet(p, &sm->s, kBarDown)) make_y(p, &sm->s, sm->step[1].ranges);
                    }
                }
            }
            if (copies) {
                land<1>(p, sm, c1);
                land<2>(p, sm, c2);
            }
            __syncwarp();
        }
    }
    leave(p, &sm->s);
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace moe

// ---------------------------------------------------------------------------
// Host side.

namespace {

constexpr uint32_t kSmemLimit = 227 * 1024;

// Stages of an item.  Shorter ones cost more work an item, longer ones leave SMs
// idle at a step's end.  Small kernel: 2, 4 and 8 took 139, 129 and 133 us for a
// layer of 8 experts of 14336 x 4096 without escapes and one token.  Large: units
// of 8, 16 and 32 tiles took 550, 528 and 533 us for 64 tokens.
constexpr uint32_t kRangeSmall = 4, kRangeLarge = moe::kUnitTiles / stage::kNT;

struct MoePlan {
    bool small, local;
    int seg;
    uint32_t range, pool, smem;
    size_t sync, scores, xp, hi, lo, gu, d, total;
};

// Workspace parts; the words that have to be zero between calls are its head.
MoePlan plan(const MoeCall &c) {
    MoePlan pl = {};
    const uint64_t slots = static_cast<uint64_t>(c.tokens) * c.top_k;
    const uint64_t H = c.up->cols, F = c.down->cols;
    // by the products' multiply-adds, which is what the mma.sync kernel is slow
    // at; the other one costs 10 to 20 us more to begin with.  Here and there, us:
    // 8 experts of 14336 x 4096, top 2: 4 tokens (1.4e9) 373 and 364, 8 tokens
    // (2.8e9) 437 and 420, 64 tokens 1251 and 507; 32 of 1408 x 2176, top 4: 48
    // tokens (1.8e9) 170 and 186, 64 tokens (2.4e9) 208 and 187; 64 of 1024 x
    // 2048, top 8: 16 tokens (0.8e9) 165 and 169, 64 tokens (3.2e9) 245 and 192
    pl.small = slots * 3 * H * F <= 1ull << 31;
    pl.seg = pl.small ? moe::kSegSmall : moe::kSegLarge;
    pl.range = pl.small ? kRangeSmall : kRangeLarge;
    if (pl.small) {
        const uint32_t fixed = 1024 + moe::kRingBytes + align_up(sizeof(moe::SmallShared), 16);
        const uint64_t x_bytes = 2ull * c.tokens * H;
        // little enough for every CTA to do alone: less time than a meeting of the grid
        // (one token, alone and by the grid, us: 8 experts of 4096 columns 48.1 and
        // 51.2, of 1024 43.9 and 44.1, 32 of 1024 46.1 and 45.2, 16 of 4096 50.6 and 50.8,
        // 64 of 1024 48.5 and 44.6; 8 tokens, 16 experts of 1024 49.5 and 39.9)
        pl.local = fixed + x_bytes <= kSmemLimit && c.tokens * c.experts <= 512 &&
                   (c.ids_in || static_cast<uint64_t>(c.tokens) * c.experts * H <= (1u << 15));
        pl.smem = fixed + static_cast<uint32_t>(pl.local ? x_bytes : 0);
    } else {
        const uint32_t fixed = 1024 + align_up(sizeof(moe::LargeShared), 1024);
        pl.pool = kSmemLimit - fixed;
        pl.smem = kSmemLimit;
        static_assert(kSmemLimit - 2048 - sizeof(moe::LargeShared) >= 3 * (moe::kTileBytes + 2 * 256 * moe::kSegLarge),
                      "three stages at least");
    }
    // (by the shorter ranges always: a call of fewer tokens never needs more)
    const auto ranges = [](uint64_t cols) {
        const uint64_t stages = (cols / kTile + stage::kNT - 1) / stage::kNT;
        return (stages + kRangeSmall - 1) / kRangeSmall;
    };
    size_t at = 0;
    auto take = [&](uint64_t bytes) {
        const size_t o = at;
        at += align_up(bytes, kAlign);
        return o;
    };
    pl.sync = take(S12_WS_HEAD);
    pl.scores = take(8ull * c.tokens * c.experts);
    pl.xp = take(2 * slots * H);
    pl.hi = take(2 * slots * F);
    pl.lo = take(2 * slots * F);
    pl.gu = take(4 * slots * 2 * F * ranges(H));
    pl.d = take(4 * slots * H * ranges(F));
    pl.total = at;
    return pl;
}

int fill_mat(moe::Mat &m, const s12_view *v, int rows_e, int box_tiles, int box_rows) {
    const uint64_t R = v->rows, K = v->cols, T = K / kTile;
    if (make_tmap_u8_3d(&m.tm_raw, v->raw, 128, T, R, 128, K, 128, box_tiles, box_rows, 128) != S12_OK ||
        make_tmap_u8_3d(&m.tm_code, v->code, 64, T, R, 64, K / 2, 64, box_tiles, box_rows, 64) != S12_OK)
        return S12_ERR_CUDA;
    m.meta = v->version == 1 ? static_cast<const void *>(v->base) : static_cast<const void *>(v->tmeta);
    m.off = v->version == 1 ? v->esc_off : v->row_esc;
    m.esc = v->esc;
    m.n_esc = static_cast<uint32_t>(v->n_esc);
    m.R = static_cast<int>(R);
    m.T = static_cast<int>(T);
    m.G = rows_e / stage::kRowsPerGroup;
    m.S = static_cast<uint32_t>((T + stage::kNT - 1) / stage::kNT);
    return S12_OK;
}

}  // namespace

size_t moe_ws_bytes(const MoeCall &c) { return plan(c).total; }

int launch_moe(const MoeCall &c, void *ws, size_t ws_bytes, cudaStream_t stream) {
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return S12_ERR_CUDA;
    const MoePlan pl = plan(c);
    if (ws_bytes < pl.total) return S12_ERR_CAPACITY;
    moe::Params p = {};
    p.H = static_cast<int>(c.up->cols);
    p.F = static_cast<int>(c.down->cols);
    const int box_tiles = pl.small ? stage::kNT : 1, box_rows = pl.small ? stage::kRowsPerGroup : moe::kBlockRows;
    int rc = fill_mat(p.up, c.up, 2 * p.F, box_tiles, box_rows);
    if (rc == S12_OK) rc = fill_mat(p.down, c.down, p.H, box_tiles, box_rows);
    if (rc != S12_OK) return rc;
    p.x = c.x;
    p.router = c.router;
    p.ids_in = c.ids_in;
    p.weights_in = c.weights_in;
    p.ids = c.ids;
    p.weights = c.weights;
    p.y = c.y;
    p.err = c.err;
    p.tokens = c.tokens;
    p.experts = c.experts;
    p.top_k = c.top_k;
    p.renorm = c.renorm;
    p.y_f32 = c.y_type == S12_TYPE_F32;
    p.seg = pl.seg;
    p.local = pl.local;
    p.range = pl.range;
    p.pool = pl.pool;
    uint8_t *w = static_cast<uint8_t *>(ws);
    p.sync = reinterpret_cast<uint32_t *>(w + pl.sync);
    p.scores = reinterpret_cast<double *>(w + pl.scores);
    p.xp = w + pl.xp;
    p.hi = w + pl.hi;
    p.lo = w + pl.lo;
    p.gu = reinterpret_cast<float *>(w + pl.gu);
    p.d = reinterpret_cast<float *>(w + pl.d);
    const bool v1 = c.up->version == 1;
    auto kern = pl.small ? (v1 ? moe::moe_small_kernel<1> : moe::moe_small_kernel<2>)
                         : (v1 ? moe::moe_large_kernel<1> : moe::moe_large_kernel<2>);
    // (always the same limit: another thread's call may be between this line and its launch)
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
        return S12_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(pl.small ? moe::kThreads : moe::kLargeThreads);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs meet, so all have to be resident
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? S12_OK : S12_ERR_CUDA;
}

}  // namespace s12
