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
//   0. x is rewritten in the order the products read it; the scores are
//      summed; grid barrier; every CTA selects the experts and sorts the
//      (token, slot) pairs by expert by itself.
//   1. gate/up products and the SwiGLU, into the workspace (h).
//   2. grid barrier; down products (d); the last of a row group's experts adds
//      them by token, in slot order, and stores y.
// The first copies of step 2 are issued before the barrier: weights do not
// depend on it, so the copy engines run on while the grid meets.
//
// Products.  As in the GEMV, a warp takes 16 rows x 2 tiles of weights a stage
// from its own ring of two, decodes them in registers into the A operand of
// mma.m16n8k16, and multiplies 8 tokens at a time.  (The tensor cores' own
// kind of product reads its weights from shared memory, which the registers
// would have to write first; at a few tokens its rate is not what is missing.)
// Weights i and i + 4 of eight share a register, because their code nibbles
// are 16 bits apart: a pair's exponents are one mask and one multiply-add of
// the code word, its signs and mantissas one byte permute, and one bit select
// joins them: 17 instructions for 8 weights.  x and h are kept with the same
// pairs in a register.  h is kept as the sum of two BF16 values, so that it
// carries 16 bits of mantissa and y is rounded once, where it is stored.
//
// Work split (stream-K).  The stages of all active experts are numbered row
// group after row group and dealt to the grid's warps in equal ranges.  A row
// group that several warps share is added up as in the GEMV: through the
// CTA's parts, and across CTAs by the last to arrive.  All sums have a fixed
// order, so y is the same on every call.
//
// Every wait is bounded.  One that gives up raises S12_FLAG_TIMEOUT and a word
// that the other waits watch; the CTAs then leave, and the last one clears
// the counters.
#include <algorithm>

#include <cuda_bf16.h>

#include "s12_device.cuh"
#include "s12_launch.h"
#include "s12_stage.cuh"

namespace s12 {
namespace moe {

using namespace stage;

constexpr int kWarps = 16;   // warps per CTA, one CTA per SM
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;   // stages per warp ring
constexpr int kSegSmall = 8, kSegLarge = 64;  // (token, slot) pairs that share one read of an expert's weights
constexpr int kMaxSlots = S12_MOE_MAX_TOKENS * S12_MOE_MAX_TOP_K;
constexpr int kMaxSegs = S12_MOE_MAX_EXPERTS + kMaxSlots / kSegSmall;
constexpr uint32_t kPartBytes = 512;  // one warp's sums of 16 rows x 8 tokens
constexpr uint32_t kRingBytes = kWarps * kStages * kStageBytes;

// A matrix of all experts: expert after expert, rows_e rows each.
struct __align__(64) Mat {
    CUtensorMap tm_raw;   // u8 {128, T, R} (strides 128, K), box {128, 2, 16}, 128-byte swizzle
    CUtensorMap tm_code;  // u8 {64, T, R} (strides 64, K/2), box {64, 2, 16}, 64-byte swizzle
    const void *meta;     // version 1: base u8[n_tiles]; version 2: (base | count << 8) u16[n_tiles]
    const uint32_t *off;  // version 1: esc_off u32[n_tiles + 1]; version 2: row_esc u32[R + 1]
    const uint16_t *esc;
    uint32_t n_esc;
    int R, T;    // rows of all experts, tiles per row
    int G;       // 16-row groups per expert
    uint32_t S;  // stages per row group
};

// Words that the grid meets at.
enum { kBarRoute, kBarSums, kBarHidden, kBarDown, kNext1, kNext2, kExits, kAbort, kSyncWords };

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
    // the kernel for few tokens:
    int local;       // every CTA routes for itself, with x in shared memory
    uint32_t range_up, range_down;  // stages of an item
    // workspace
    uint32_t *sync;         // kSyncWords
    uint32_t *cnt;          // arrivals: [segs][G up], [segs][G down], [G down]
    uint32_t n_cnt, cnt_down, cnt_y;
    double *scores;         // [tokens][experts]
    uint8_t *xp, *hi, *lo;  // x, and h as two BF16 values, in the products' order
    float *gu;              // few tokens: [ranges][slots][2F]
    float *d;               // [slots][H], few tokens: [ranges][slots][H]
    float *warp_part;       // [CTAs * kWarps][2][NT][128] for more than 8 tokens an expert
    float *cta_part;        // [CTAs][2][NT][128]
};

struct Shared {
    unsigned long long bars[kWarps * kStages];
    float weight[kMaxSlots];
    int16_t expert[kMaxSlots];  // of each (token, slot), -1 for none
    uint16_t list[kMaxSlots];   // (token, slot) pairs by expert
    uint16_t token[kMaxSlots];  // of each of them
    uint16_t place[kMaxSlots];  // of each (token, slot) in the list
    int count[S12_MOE_MAX_EXPERTS], first[S12_MOE_MAX_EXPERTS];
    uint16_t seg_expert[kMaxSegs], seg_first[kMaxSegs];
    uint8_t seg_n[kMaxSegs];
    int n_segs, most;  // segments; pairs of the largest
    int ok, last;
};

// Order of x and h in the workspace, in 16-byte pieces of 8 values: tile,
// then 16-column chunk of a lane's 64, then half chunk, then token (of x) or
// sorted pair (of h), then which 64 columns of the tile.  A warp's load of
// one half chunk is then contiguous over tokens.  Inside a piece the values
// come as 0 4 1 5 2 6 3 7.
__device__ __forceinline__ size_t piece_at(int tile, int chunk, int half, int n, int i, int qh) {
    return ((((static_cast<size_t>(tile) * 4 + chunk) * 2 + half) * n + i) * 2 + qh) * 16;
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

__device__ __forceinline__ void pack_x(const Params &p, uint8_t *to, int i0, int step) {
    const int per_row = p.H / 8;
    const int n = p.tokens * per_row;
    for (int i = i0; i < n; i += step) {
        const int t = i / per_row, c8 = i - t * per_row;  // piece c8 of token t
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p.x) + i);
        const int in = c8 & 15;  // piece of the tile: 64 columns, chunk, half
        uint4 *dst = reinterpret_cast<uint4 *>(to + piece_at(c8 >> 4, (in >> 1) & 3, in & 1, p.tokens, t, in >> 3));
        *dst = make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u),
                          prmt(v.y, v.w, 0x7632u));
    }
}

__device__ __forceinline__ void unpack8(const uint4 &a, float (&v)[8]) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

// Scores of TT tokens and TE experts to a warp.  The products of BF16 values
// are exact in FP32; eight of them are added in FP32, the rest in 64 bits,
// because the choice of experts hangs on the order of the scores.
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
#pragma unroll(TT == 1 ? 8 : 1)
        for (int k = lane * 8; k < p.H; k += 256) {
            float xv[TT][8];
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                const size_t t = min(t0 + i, p.tokens - 1);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(p.x + t * p.H + k)), xv[i]);
            }
#pragma unroll
            for (int j = 0; j < TE; ++j) {
                const size_t e = min(e0 + j, p.experts - 1);
                float rv[8];
                unpack8(__ldg(reinterpret_cast<const uint4 *>(p.router + e * p.H + k)), rv);
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    float s = xv[i][0] * rv[0];
#pragma unroll
                    for (int c = 1; c < 8; ++c) s = fmaf(xv[i][c], rv[c], s);
                    acc[i][j] += static_cast<double>(s);
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
// the lower index first where two are equal (a NaN counts as -infinity, and
// makes the token's weights NaN).
__device__ __forceinline__ void select_experts(const Params &p, Shared *sm, const double *scores, int t) {
    constexpr int kPer = S12_MOE_MAX_EXPERTS / 32;
    const int lane = threadIdx.x & 31;
    const double *row = scores + static_cast<size_t>(t) * p.experts;
    const double low = -__longlong_as_double(0x7FF0000000000000ll);
    double v[kPer];
    uint32_t left = 0u;  // bit i: expert lane + 32 i is not chosen yet
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        v[i] = low;
        if (e < p.experts) {
            v[i] = row[e];
            if (v[i] != v[i]) v[i] = low;
            left |= 1u << i;
        }
    }
    double top = 0.0;
    float mine = 0.f;  // lane s < top_k: the weight of slot s before its division
    int chosen = -1;
    for (int s = 0; s < p.top_k; ++s) {
        double best = low;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if ((left >> i & 1u) && (at == 0x7FFFFFFF || v[i] > best)) {
                best = v[i];
                at = lane + 32 * i;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            const int a = __shfl_xor_sync(0xFFFFFFFFu, at, o);
            if (a != 0x7FFFFFFF && (at == 0x7FFFFFFF || b > best || (b == best && a < at))) {
                best = b;
                at = a;
            }
        }
        if ((at & 31) == lane) left &= ~(1u << (at >> 5));
        if (s == 0) top = best;
        if (lane == s) {
            chosen = at;
            mine = expf(static_cast<float>(best - top));
        }
    }
    float sum = 0.f;
    if (p.renorm) {
        sum = mine;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < p.experts) sum += expf(static_cast<float>(v[i] - top));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < p.top_k) {
        const int i = t * p.top_k + lane;
        sm->expert[i] = static_cast<int16_t>(chosen);
        sm->weight[i] = mine / sum;
        if (blockIdx.x == 0) {
            if (p.ids) p.ids[i] = chosen;
            if (p.weights) p.weights[i] = mine / sum;
        }
    }
}

// Every CTA for itself: the (token, slot) pairs sorted by expert (by index
// inside one), cut into segments of at most p.seg.
__device__ __forceinline__ void route(const Params &p, Shared *sm, const double *scores) {
    const int slots = p.tokens * p.top_k, tid = threadIdx.x;
    if (p.ids_in) {
        if (tid < slots) {
            const int e = __ldg(p.ids_in + tid);
            sm->expert[tid] = static_cast<int16_t>(e >= 0 && e < p.experts ? e : -1);
            sm->weight[tid] = __ldg(p.weights_in + tid);
        }
    } else {
        for (int t = tid >> 5; t < p.tokens; t += kWarps) select_experts(p, sm, scores, t);
    }
    __syncthreads();
    if (tid < p.experts) {
        int n = 0;
        for (int i = 0; i < slots; ++i) n += sm->expert[i] == tid;
        sm->count[tid] = n;
    }
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
            if (e < p.experts) sm->first[e] = at;
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
    if (tid < p.experts && sm->count[tid]) {
        int at = sm->first[tid];
        for (int i = 0; i < slots; ++i)
            if (sm->expert[i] == tid) {
                sm->place[i] = static_cast<uint16_t>(at);
                sm->token[at] = static_cast<uint16_t>(i / p.top_k);
                sm->list[at++] = static_cast<uint16_t>(i);
            }
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Positions.  PH 1: row groups by segment, then row; PH 2: by row, then
// segment (all of a row's experts end close together).

template <int PH>
__device__ __forceinline__ const Mat &mat(const Params &p) {
    return PH == 1 ? p.up : p.down;
}

template <int PH>
__device__ __forceinline__ void split(const Params &p, const Shared *sm, uint32_t gi, uint32_t &seg, uint32_t &grp) {
    if (PH == 1) {
        seg = gi / static_cast<uint32_t>(p.up.G);
        grp = gi - seg * static_cast<uint32_t>(p.up.G);
    } else {
        grp = gi / static_cast<uint32_t>(sm->n_segs);
        seg = gi - grp * static_cast<uint32_t>(sm->n_segs);
    }
}

// A stage: row group gi of the step, first tile j, `left` stages of the
// warp's range from here on; row16: its 16-row group in the matrix.
struct Cur {
    uint32_t gi;
    int j, left;
    uint32_t row16;
};

template <int PH>
__device__ __forceinline__ uint32_t row16_of(const Params &p, const Shared *sm, uint32_t gi) {
    uint32_t seg, grp;
    split<PH>(p, sm, gi, seg, grp);
    return sm->seg_expert[seg] * static_cast<uint32_t>(mat<PH>(p).G) + grp;
}

template <int PH>
__device__ __forceinline__ Cur locate(const Params &p, const Shared *sm, uint32_t s, int left) {
    const uint32_t S = mat<PH>(p).S;
    Cur c;
    c.gi = s / S;
    c.j = static_cast<int>(s - c.gi * S) * kNT;
    c.left = left;
    c.row16 = left > 0 ? row16_of<PH>(p, sm, c.gi) : 0u;
    return c;
}

template <int PH>
__device__ __forceinline__ void advance(const Params &p, const Shared *sm, Cur &c) {
    --c.left;
    c.j += kNT;
    if (c.j >= mat<PH>(p).T) {
        c.j = 0;
        ++c.gi;
        if (c.left > 0) c.row16 = row16_of<PH>(p, sm, c.gi);
    }
}

// The warp's ring: stages issued and consumed so far, over both steps.
struct Ring {
    uint32_t bars, base;
    int issued, consumed;
};

// Copy the stage at c into the ring's next place (lane 0 issues).
template <int PH>
__device__ __forceinline__ void issue(const Params &p, const Shared *sm, Ring &r, Cur &c) {
    if ((threadIdx.x & 31) == 0) {
        const uint32_t s = static_cast<uint32_t>(r.issued & 1), st = r.base + s * kStageBytes, bar = r.bars + 8u * s;
        const uint64_t pol = policy_evict_first();
        const Mat &m = mat<PH>(p);
        mbar_expect_tx_s(bar, kStageBytes);
        tma3d(st, &m.tm_raw, 0, c.j, static_cast<int>(c.row16) * kRowsPerGroup, bar, pol);
        tma3d(st + kRawStage, &m.tm_code, 0, c.j, static_cast<int>(c.row16) * kRowsPerGroup, bar, pol);
    }
    ++r.issued;
    advance<PH>(p, sm, c);
}

// The end of a CTA: copies that a wait left in flight land, and the last CTA
// leaves the workspace's words at zero.
__device__ __forceinline__ void finish(const Params &p, Shared *sm, const Ring &rg) {
    if ((threadIdx.x & 31) == 0)
        for (int k = rg.consumed; k < rg.issued; ++k)
            mbar_wait_s(rg.bars + 8u * (k & 1), static_cast<uint32_t>(k >> 1) & 1u);
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        sm->last = atomicAdd(p.sync + kExits, 1u) + 1 == gridDim.x;
    }
    __syncthreads();
    if (sm->last) {
        __threadfence();
        if (ld_acquire(p.sync + kAbort))
            for (uint32_t i = threadIdx.x; i < p.n_cnt; i += kThreads) p.cnt[i] = 0u;
        __syncthreads();
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
// stream index idx on; reads at or past `limit` are skipped and flagged.
__device__ __forceinline__ void patch(uint32_t (&w)[8], uint2 C, uint32_t idx, uint32_t limit,
                                      const uint16_t *__restrict__ esc, uint32_t *err) {
    uint64_t mm = (static_cast<uint64_t>(escape_nibbles(C.y)) << 32) | escape_nibbles(C.x);
    while (mm) {
        const int j = (__ffsll(static_cast<long long>(mm)) - 1) >> 2;
        mm &= mm - 1;
        uint32_t v = 0;
        if (idx < limit)
            v = __ldg(esc + idx);
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

// h of row group (seg, grp): lane (g, q) holds gate row f and up row f
// (f = 8 grp + g) of pairs 2q, 2q+1 of each eight.
template <int NT>
__device__ __forceinline__ void store_hidden(const Params &p, const Shared *sm, const float (&a)[NT][4], uint32_t seg,
                                             uint32_t grp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int n = sm->seg_n[seg], first = sm->seg_first[seg], slots = p.tokens * p.top_k;
    // the eight f of a row group are one piece; this lane's place in it
    const int c8 = static_cast<int>(grp), in = c8 & 15;
    const size_t base = piece_at(c8 >> 4, (in >> 1) & 3, in & 1, slots, first, in >> 3) +
                        2 * (g < 4 ? 2 * g : 2 * (g - 4) + 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int b = nt * 8 + 2 * q + i;
            if (b < n) {
                const float gt = a[nt][i], hv = gt / (1.f + expf(-gt)) * a[nt][2 + i];
                const __nv_bfloat16 hi = __float2bfloat16_rn(hv);
                const float rest = hv - __bfloat162float(hi);
                // (an infinite h has no rest)
                const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(rest) < 3.4e38f ? rest : 0.f);
                const size_t o = base + static_cast<size_t>(b) * 32;
                *reinterpret_cast<uint16_t *>(p.hi + o) = __bfloat16_as_ushort(hi);
                *reinterpret_cast<uint16_t *>(p.lo + o) = __bfloat16_as_ushort(lo);
            }
        }
}

__device__ __forceinline__ void put_y(const Params &p, size_t o, float v) {
    if (p.y_f32)
        static_cast<float *>(p.y)[o] = v;
    else
        static_cast<uint16_t *>(p.y)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// d of row group (seg, grp); the last segment of the row group adds up y.
template <int NT>
__device__ __forceinline__ void store_down(const Params &p, const Shared *sm, const float (&a)[NT][4], uint32_t seg,
                                           uint32_t grp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int n = sm->seg_n[seg], first = sm->seg_first[seg];
    const size_t r = static_cast<size_t>(grp) * kRowsPerGroup + g;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = nt * 8 + 2 * q + (i & 1);
            if (b < n) __stcg(p.d + static_cast<size_t>(sm->list[first + b]) * p.H + r + (i >= 2 ? 8 : 0), a[nt][i]);
        }
    __threadfence();
    __syncwarp();
    uint32_t prev = 0;
    if (lane == 0) prev = atomicAdd(p.cnt + p.cnt_y + grp, 1u);
    prev = __shfl_sync(0xFFFFFFFFu, prev, 0);
    if (prev + 1 != static_cast<uint32_t>(sm->n_segs)) return;
    __threadfence();
    if (lane == 0) atomicExch(p.cnt + p.cnt_y + grp, 0u);
    const size_t col = static_cast<size_t>(grp) * kRowsPerGroup + (lane & 15);
    for (int t = lane >> 4; t < p.tokens; t += 2) {
        float y = 0.f;
        for (int s = 0; s < p.top_k; ++s) {
            const int i = t * p.top_k + s;
            if (sm->expert[i] >= 0) y = fmaf(sm->weight[i], __ldcg(p.d + static_cast<size_t>(i) * p.H + col), y);
        }
        put_y(p, static_cast<size_t>(t) * p.H + col, y);
    }
}

template <int NT, int PH>
__device__ __noinline__ void store_group(const Params &p, const Shared *sm, const float (&a)[NT][4], uint32_t gi) {
    uint32_t seg, grp;
    split<PH>(p, sm, gi, seg, grp);
    if (PH == 1)
        store_hidden<NT>(p, sm, a, seg, grp);
    else
        store_down<NT>(p, sm, a, seg, grp);
}

// ---------------------------------------------------------------------------
// Row groups shared by warps.  Slot 0 of a warp (or CTA): the group that its
// range starts in; slot 1: the one that it ends in.

template <int NT>
__device__ __forceinline__ float4 *warp_slot(const Params &p, float4 *parts, int warp, int slot) {
    if (NT == 1) return parts + (warp * 2 + slot) * 32;
    return reinterpret_cast<float4 *>(p.warp_part) +
           ((static_cast<size_t>(blockIdx.x) * kWarps + warp) * 2 + slot) * NT * 32;
}

template <int NT>
__device__ __forceinline__ float4 *cta_slot(const Params &p, size_t cta, int slot) {
    return reinterpret_cast<float4 *>(p.cta_part) + (cta * 2 + slot) * NT * 32;
}

// The deal of a step's stages.
struct Deal {
    long long n_stages;
    int n_units;
    uint32_t S;
    uint32_t cnt0;  // the step's first arrival counter

    __device__ __forceinline__ long long start(long long unit) const { return unit_start(unit, n_stages, n_units); }
};

// Parts of a group that crosses CTAs: this CTA's goes to its slot, the last
// CTA to arrive adds all in CTA order.
template <int NT, int PH>
__device__ __noinline__ void join_ctas(const Params &p, const Shared *sm, const Deal &dl, float (&a)[NT][4],
                                       uint32_t gi) {
    const int lane = threadIdx.x & 31, n_ctas = gridDim.x;
    const long long c = blockIdx.x, c0 = dl.start(c * kWarps);
    const long long g0 = static_cast<long long>(gi) * dl.S, g1 = g0 + dl.S;
    float4 *mine = cta_slot<NT>(p, c, g0 <= c0 ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        __stcg(mine + nt * 32 + lane, make_float4(a[nt][0], a[nt][1], a[nt][2], a[nt][3]));
    __threadfence();
    __syncwarp();
    long long cf = c, cl = c;
    while (cf > 0 && dl.start(cf * kWarps) > g0) --cf;
    while (cl + 1 < n_ctas && dl.start((cl + 1) * kWarps) < g1) ++cl;
    // (CTAs without a stage of their own hand in nothing)
    uint32_t want = 0;
    for (long long v = cf; v <= cl; ++v) want += dl.start(v * kWarps) < dl.start((v + 1) * kWarps) ? 1u : 0u;
    uint32_t prev = 0;
    if (lane == 0) prev = atomicAdd(p.cnt + dl.cnt0 + gi, 1u);
    prev = __shfl_sync(0xFFFFFFFFu, prev, 0);
    if (prev + 1 != want) return;
    __threadfence();
    if (lane == 0) atomicExch(p.cnt + dl.cnt0 + gi, 0u);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) a[nt][i] = 0.f;
    for (long long v = cf; v <= cl; ++v) {
        const long long vs = dl.start(v * kWarps);
        if (vs >= dl.start((v + 1) * kWarps)) continue;
        const float4 *src = cta_slot<NT>(p, v, g0 <= vs ? 0 : 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4 t = __ldcg(src + nt * 32 + lane);
            a[nt][0] += t.x;
            a[nt][1] += t.y;
            a[nt][2] += t.z;
            a[nt][3] += t.w;
        }
    }
    store_group<NT, PH>(p, sm, a, gi);
}

// After every warp's parts are in place: each shared group is completed by
// the warp that holds its first stage in this CTA.
template <int NT, int PH>
__device__ __noinline__ void join_warps(const Params &p, const Shared *sm, float4 *parts, const Deal &dl) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long u = static_cast<long long>(blockIdx.x) * kWarps;
    const long long bnd = dl.start(u + (lane <= kWarps ? lane : kWarps));
    auto boundary = [&](int i) { return static_cast<long long>(__shfl_sync(0xFFFFFFFFu, bnd, i)); };
    const long long c0 = boundary(0), c1 = boundary(kWarps);
    const long long wb = boundary(warp), we = boundary(warp + 1);
    if (wb >= we) return;
    const uint32_t first = static_cast<uint32_t>(wb) / dl.S, last = static_cast<uint32_t>(we - 1) / dl.S;
    for (int k = 0; k < 2; ++k) {
        const uint32_t gi = k ? last : first;
        if (k && last == first) break;
        const long long g0 = static_cast<long long>(gi) * dl.S, g1 = g0 + dl.S;
        if (g0 >= wb && g1 <= we) continue;        // whole in this warp: stored already
        if ((g0 > c0 ? g0 : c0) < wb) continue;    // an earlier warp completes it
        float a[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[nt][i] = 0.f;
        for (int v = warp; v < kWarps; ++v) {
            const long long vb = boundary(v), ve = boundary(v + 1);
            if (vb >= g1) break;
            if (vb >= ve) continue;
            const float4 *src = warp_slot<NT>(p, parts, v, g0 <= vb ? 0 : 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float4 t = src[nt * 32 + lane];
                a[nt][0] += t.x;
                a[nt][1] += t.y;
                a[nt][2] += t.z;
                a[nt][3] += t.w;
            }
        }
        if (g0 >= c0 && g1 <= c1)
            store_group<NT, PH>(p, sm, a, gi);
        else
            join_ctas<NT, PH>(p, sm, dl, a, gi);
    }
}

// ---------------------------------------------------------------------------
// One step's products by one warp.

template <int V, class M>
__device__ __forceinline__ Meta load_meta(const M &m, const Cur &c, int len, int g, int tq, bool row_start) {
    const int r = static_cast<int>(c.row16) * kRowsPerGroup + g;
    Meta o;
    load_row_meta<V>(m, r, c.j, len, tq, row_start, o.a0, o.a1, o.a2);
    load_row_meta<V>(m, r + 8, c.j, len, tq, row_start, o.b0, o.b1, o.b2);
    return o;
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

__device__ __forceinline__ void chunk_mma(float (&acc)[4], const uint32_t (&wa)[8], const uint32_t (&wb)[8],
                                          const uint32_t (&xw)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        mma16816(acc, wa[2 * i], wb[2 * i], wa[2 * i + 1], wb[2 * i + 1], xw[2 * i], xw[2 * i + 1]);
}

// The warp's range of step PH; `pc` is the next stage to copy (the first
// ones are in flight).  False when a wait gave up.
template <int V, int NT, int PH>
__device__ __forceinline__ bool products(const Params &p, const Shared *sm, float4 *parts, Ring &rg, Cur pc,
                                         const Deal &dl, long long s0, int n) {
    constexpr int kChains = NT == 1 ? 2 : 1;  // independent sums, so that products do not wait for one another
    const Mat &m = mat<PH>(p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3, tq = q >> 1, qh = q & 1;
    const int nx = PH == 1 ? p.tokens : p.tokens * p.top_k;  // rows of x or h
    const size_t half = static_cast<size_t>(nx) * 32, chunk_bytes = 2 * half;
    // the lane's places in a stage ([row][tile][bytes], swizzled by the copies)
    const uint32_t line = static_cast<uint32_t>(2 * g + tq), rsw = line & 7u, csw = static_cast<uint32_t>(g) & 3u;
    const uint32_t oR = line * 128u, oC = kRawStage + line * 64u;

    Cur cc = locate<PH>(p, sm, static_cast<uint32_t>(s0), n), cn = cc;
    int len = min(kNT, m.T - cc.j);
    Meta mc = load_meta<V>(m, cc, len, g, tq, true);
    uint32_t runA = 0, runB = 0;
    if (V == 2) {
        const int r = static_cast<int>(cc.row16) * kRowsPerGroup + g;
        runA = mc.a2 + prefix_count_v2(m, r, cc.j, q);
        runB = mc.b2 + prefix_count_v2(m, r + 8, cc.j, q);
    }
    advance<PH>(p, sm, cn);

    float acc[kChains][NT][4];
    uint32_t xoff[NT];
    int nts = 0;  // eights of pairs in the current segment
    bool fresh = true;
    while (cc.left > 0) {
        if (fresh) {
            fresh = false;
            uint32_t seg, grp;
            split<PH>(p, sm, cc.gi, seg, grp);
            const int pairs = sm->seg_n[seg], first = sm->seg_first[seg];
            nts = (pairs + 7) >> 3;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // (columns past the last pair repeat it; their results are dropped)
                const int at = first + min(nt * 8 + g, pairs - 1);
                xoff[nt] = static_cast<uint32_t>((PH == 1 ? sm->list[at] / p.top_k : at) * 32 + qh * 16);
#pragma unroll
                for (int k = 0; k < kChains; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[k][nt][i] = 0.f;
            }
        }
        int lenn = 0;
        Meta mn = {0u, 0u, 0u, 0u, 0u, 0u};
        if (cn.left > 0) {
            lenn = min(kNT, m.T - cn.j);
            mn = load_meta<V>(m, cn, lenn, g, tq, cn.j == 0);
        }
        const uint32_t slot = static_cast<uint32_t>(rg.consumed & 1), bar = rg.bars + 8u * slot;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_s(bar, static_cast<uint32_t>(rg.consumed >> 1) & 1u))) {
            if (lane == 0) give_up(p);
            return false;
        }
        const uint32_t st = rg.base + slot * kStageBytes;
        const bool live = tq < len;  // the lane's tile belongs to this stage (else zeros from the copy)
        uint32_t bA, sA, eA, bB, sB, eB;
        row_span<V>(mc.a0, mc.a1, mc.a2, tq, runA, bA, sA, eA);
        row_span<V>(mc.b0, mc.b1, mc.b2, tq, runB, bB, sB, eB);
        const uint4 cA0 = lds128(st + oC + (((2u * qh) ^ csw) << 4));
        const uint4 cA1 = lds128(st + oC + (((2u * qh + 1u) ^ csw) << 4));
        const uint4 cB0 = lds128(st + oC + (((2u * qh) ^ csw) << 4) + 1024);
        const uint4 cB1 = lds128(st + oC + (((2u * qh + 1u) ^ csw) << 4) + 1024);
        if (p.err && (bA > static_cast<uint32_t>(kMaxBase) || bB > static_cast<uint32_t>(kMaxBase)))
            raise_flag(p.err, S12_FLAG_BASE);
        const bool anyesc = __any_sync(0xFFFFFFFFu, eA != sA || eB != sB);
        const uint32_t B2A = bA * 0x00800080u, B2B = bB * 0x00800080u;
        const size_t at = static_cast<size_t>(cc.j + tq) * 4 * chunk_bytes;
        const uint8_t *x0 = (PH == 1 ? p.xp : p.hi) + at, *x1 = p.lo + at;

        auto multiply = [&](int c, const uint32_t (&wa)[8], const uint32_t (&wb)[8], float (&a)[NT][4]) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (NT == 1 || nt < nts) {
                    uint32_t xw[8];
                    load_x(xw, x0 + xoff[nt] + c * chunk_bytes, half, live);
                    chunk_mma(a[nt], wa, wb, xw);
                    if (PH == 2) {
                        load_x(xw, x1 + xoff[nt] + c * chunk_bytes, half, live);
                        chunk_mma(a[nt], wa, wb, xw);
                    }
                }
        };
        auto refill = [&]() {
            // the stage is in registers: hand it back to the copy engine
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (pc.left > 0) issue<PH>(p, sm, rg, pc);
        };
        if (!anyesc) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 rA = lds128(st + oR + (((4u * qh + c) ^ rsw) << 4));
                const uint4 rB = lds128(st + oR + (((4u * qh + c) ^ rsw) << 4) + 2048);
                if (c == 3) refill();
                const uint4 kA = c < 2 ? cA0 : cA1, kB = c < 2 ? cB0 : cB1;
                uint32_t wa[8], wb[8];
                decode_pairs(rA.x, rA.y, c & 1 ? kA.z : kA.x, B2A, wa);
                decode_pairs(rA.z, rA.w, c & 1 ? kA.w : kA.y, B2A, wa + 4);
                decode_pairs(rB.x, rB.y, c & 1 ? kB.z : kB.x, B2B, wb);
                decode_pairs(rB.z, rB.w, c & 1 ? kB.w : kB.y, B2B, wb + 4);
                multiply(c, wa, wb, acc[c & (kChains - 1)]);
            }
        } else {
            // some row of the stage has escapes: a compact loop (its first
            // half of a tile row counts from the span's start, the second
            // half back from its end)
            const uint32_t nA = chunk_counts(cA0, cA1), nB = chunk_counts(cB0, cB1);
            const uint32_t allA = (nA * 0x01010101u) >> 24, allB = (nB * 0x01010101u) >> 24;
            const uint32_t pairA = allA + __shfl_xor_sync(0xFFFFFFFFu, allA, 1);
            const uint32_t pairB = allB + __shfl_xor_sync(0xFFFFFFFFu, allB, 1);
            if (p.err && live && qh == 0 && (pairA != eA - sA || pairB != eB - sB))
                raise_flag(p.err, S12_FLAG_ESC_COUNT);
            uint32_t iA = qh ? eA - allA : sA, iB = qh ? eB - allB : sB;
            const uint32_t limA = sA <= eA ? min(eA, m.n_esc) : 0u, limB = sB <= eB ? min(eB, m.n_esc) : 0u;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const uint4 rA = lds128(st + oR + (((4u * qh + c) ^ rsw) << 4));
                const uint4 rB = lds128(st + oR + (((4u * qh + c) ^ rsw) << 4) + 2048);
                const uint32_t piece = st + oC + (((2u * qh + (c >> 1)) ^ csw) << 4) + 8u * (c & 1);
                const uint2 kA = lds64(piece), kB = lds64(piece + 1024);
                uint32_t wa[8], wb[8];
                decode_pairs(rA.x, rA.y, kA.x, B2A, wa);
                decode_pairs(rA.z, rA.w, kA.y, B2A, wa + 4);
                decode_pairs(rB.x, rB.y, kB.x, B2B, wb);
                decode_pairs(rB.z, rB.w, kB.y, B2B, wb + 4);
                const uint32_t hereA = (nA >> (8 * c)) & 0xFFu, hereB = (nB >> (8 * c)) & 0xFFu;
                if (hereA) patch(wa, kA, iA, limA, m.esc, p.err);
                if (hereB) patch(wb, kB, iB, limB, m.esc, p.err);
                iA += hereA;
                iB += hereB;
                multiply(c, wa, wb, acc[0]);
            }
            refill();
        }
        ++rg.consumed;
        if (cn.gi != cc.gi || cn.left == 0) {
            // the range leaves this row group
            if (kChains == 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][0][i] += acc[kChains - 1][0][i];
            const long long g0 = static_cast<long long>(cc.gi) * dl.S;
            if (g0 >= s0 && g0 + dl.S <= s0 + n) {
                // (a copy: only it has an address, the sums stay in registers)
                float a[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[nt][i] = acc[0][nt][i];
                store_group<NT, PH>(p, sm, a, cc.gi);
            } else {
                float4 *dst = warp_slot<NT>(p, parts, warp, g0 <= s0 ? 0 : 1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    dst[nt * 32 + lane] = make_float4(acc[0][nt][0], acc[0][nt][1], acc[0][nt][2], acc[0][nt][3]);
            }
            fresh = true;
            if (V == 2) {
                runA = mn.a2;
                runB = mn.b2;
            }
        }
        cc = cn;
        len = lenn;
        mc = mn;
        if (cn.left > 0) advance<PH>(p, sm, cn);
    }
    return true;
}

template <int PH>
__device__ __forceinline__ Deal deal(const Params &p, const Shared *sm) {
    const Mat &m = mat<PH>(p);
    Deal d;
    d.S = m.S;
    d.n_stages = static_cast<long long>(sm->n_segs) * m.G * m.S;
    d.n_units = static_cast<int>(gridDim.x) * kWarps;
    d.cnt0 = PH == 1 ? 0u : p.cnt_down;
    return d;
}

// Both steps with NT eights of pairs a segment at most.
template <int V, int NT>
__device__ __noinline__ Ring layer(const Params &p, Shared *sm, float4 *parts, Ring rg) {
    const long long u = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const Deal d1 = deal<1>(p, sm), d2 = deal<2>(p, sm);
    const long long s1 = d1.start(u), s2 = d2.start(u);
    const int n1 = static_cast<int>(d1.start(u + 1) - s1), n2 = static_cast<int>(d2.start(u + 1) - s2);
    Cur pc = locate<1>(p, sm, static_cast<uint32_t>(s1), n1);
    for (int k = 0; k < kStages && pc.left > 0; ++k) issue<1>(p, sm, rg, pc);
    bool ok = n1 == 0 || products<V, NT, 1>(p, sm, parts, rg, pc, d1, s1, n1);
    // the first copies of step 2 run while the grid meets
    pc = locate<2>(p, sm, static_cast<uint32_t>(s2), n2);
    if (ok)
        for (int k = 0; k < kStages && pc.left > 0; ++k) issue<2>(p, sm, rg, pc);
    __syncthreads();
    join_warps<NT, 1>(p, sm, parts, d1);
    if (!grid_meet(p, sm, kBarHidden)) return rg;
    if (ok && n2 > 0) products<V, NT, 2>(p, sm, parts, rg, pc, d2, s2, n2);
    __syncthreads();
    join_warps<NT, 2>(p, sm, parts, d2);
    return rg;
}

template <int V>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    float4 *parts = reinterpret_cast<float4 *>(base + kRingBytes);
    Shared *sm = reinterpret_cast<Shared *>(base + kRingBytes + kWarps * 2 * kPartBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Ring rg;
    rg.bars = smem_addr(sm->bars) + static_cast<uint32_t>(warp) * kStages * 8u;
    rg.base = smem_addr(base) + static_cast<uint32_t>(warp) * kStages * kStageBytes;
    rg.issued = rg.consumed = 0;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init_s(rg.bars + 8u * s, 1);
        fence_barrier_init();
    }
    pack_x(p, p.xp, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
    if (!p.ids_in) {
        // many scores: 4 x 4 to a warp, so that x and the router are read a quarter as often
        const int u0 = warp * gridDim.x + blockIdx.x, step = gridDim.x * kWarps;
        if (p.tokens >= 8 && p.tokens * p.experts >= 1024)
            score<4, 4>(p, p.scores, u0, step);
        else
            score<1, 1>(p, p.scores, u0, step);
    }
    if (grid_meet(p, sm, kBarRoute)) {
        route(p, sm, p.scores);
        if (sm->n_segs == 0) {
            // no token goes anywhere
            const size_t n = static_cast<size_t>(p.tokens) * p.H;
            for (size_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) put_y(p, i, 0.f);
        } else if (sm->most <= 8) {
            rg = layer<V, 1>(p, sm, parts, rg);
        } else if (sm->most <= 16) {
            rg = layer<V, 2>(p, sm, parts, rg);
        } else if (sm->most <= 32) {
            rg = layer<V, 4>(p, sm, parts, rg);
        } else {
            rg = layer<V, 8>(p, sm, parts, rg);
        }
    }
    finish(p, sm, rg);
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
    uint32_t m1, m2, d2;  // reciprocals of `ranges` and of d2, the row groups (step 1) or segments (step 2)
};

struct SmallShared {
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

template <int PH>
__device__ __forceinline__ void plan_step(const Params &p, SmallShared *sm) {
    const Mat &m = mat<PH>(p);
    Step st;
    const uint32_t groups = static_cast<uint32_t>(sm->s.n_segs) * m.G;
    st.stages = min(PH == 1 ? p.range_up : p.range_down, m.S);
    st.ranges = (m.S + st.stages - 1) / st.stages;
    st.items = groups * st.ranges;
    st.d2 = PH == 1 ? static_cast<uint32_t>(m.G) : static_cast<uint32_t>(sm->s.n_segs);
    st.m1 = reciprocal(st.ranges);
    st.m2 = reciprocal(st.d2);
    sm->step[PH - 1] = st;
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
};

template <int V>
__device__ __forceinline__ Words load_words(const Mat &m, const Desc &d) {
    const int lane = threadIdx.x & 31, t = d.j + (lane >> 4);
    Words w = {0u, 0u, 0u};
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
    if (!anyesc) {
        const uint4 cA0 = lds128(oC + (((2u * qh) ^ csw) << 4)), cA1 = lds128(oC + (((2u * qh + 1u) ^ csw) << 4));
        const uint4 cB0 = lds128(oC + (((2u * qh) ^ csw) << 4) + 1024);
        const uint4 cB1 = lds128(oC + (((2u * qh + 1u) ^ csw) << 4) + 1024);
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
            multiply(c, wa, wb);
        }
        return;
    }
    // some row of the stage has escapes: a compact loop.  A lane's first half of
    // a tile row counts from the span's start, the second half back from its end.
    uint32_t sA, eA, sB, eB;
    if (V == 1) {
        sA = __shfl_sync(0xFFFFFFFFu, wd.w1, src);
        eA = __shfl_sync(0xFFFFFFFFu, wd.w2, src);
        sB = __shfl_sync(0xFFFFFFFFu, wd.w1, src + 8);
        eB = __shfl_sync(0xFFFFFFFFu, wd.w2, src + 8);
    } else {
        // row_esc and the counts of the row's earlier tiles
        const int r = static_cast<int>(d.row16) * kRowsPerGroup + g;
        const uint32_t n = wd.w0 >> 8;
        sA = __ldg(m.off + r) + prefix_count_v2(m, r, d.j, q);
        sB = __ldg(m.off + r + 8) + prefix_count_v2(m, r + 8, d.j, q);
        const uint32_t nA = __shfl_sync(0xFFFFFFFFu, n, g), nB = __shfl_sync(0xFFFFFFFFu, n, g + 8);
        sA += tq ? nA : 0u;
        sB += tq ? nB : 0u;
        eA = sA + __shfl_sync(0xFFFFFFFFu, n, src);
        eB = sB + __shfl_sync(0xFFFFFFFFu, n, src + 8);
    }
    const uint32_t nA = chunk_counts(lds128(oC + (((2u * qh) ^ csw) << 4)), lds128(oC + (((2u * qh + 1u) ^ csw) << 4)));
    const uint32_t nB = chunk_counts(lds128(oC + (((2u * qh) ^ csw) << 4) + 1024),
                                     lds128(oC + (((2u * qh + 1u) ^ csw) << 4) + 1024));
    const uint32_t allA = (nA * 0x01010101u) >> 24, allB = (nB * 0x01010101u) >> 24;
    const uint32_t pairA = allA + __shfl_xor_sync(0xFFFFFFFFu, allA, 1);
    const uint32_t pairB = allB + __shfl_xor_sync(0xFFFFFFFFu, allB, 1);
    if (p.err && d.j + tq < m.T && qh == 0 && (pairA != eA - sA || pairB != eB - sB))
        raise_flag(p.err, S12_FLAG_ESC_COUNT);
    uint32_t iA = qh ? eA - allA : sA, iB = qh ? eB - allB : sB;
    const uint32_t limA = sA <= eA ? min(eA, m.n_esc) : 0u, limB = sB <= eB ? min(eB, m.n_esc) : 0u;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        const uint4 rA = lds128(oR + (((4u * qh + c) ^ rsw) << 4));
        const uint4 rB = lds128(oR + (((4u * qh + c) ^ rsw) << 4) + 2048);
        const uint32_t piece = oC + (((2u * qh + (c >> 1)) ^ csw) << 4) + 8u * (c & 1);
        const uint2 kA = lds64(piece), kB = lds64(piece + 1024);
        uint32_t wa[8], wb[8];
        decode_pairs(rA.x, rA.y, kA.x, B2A, wa);
        decode_pairs(rA.z, rA.w, kA.y, B2A, wa + 4);
        decode_pairs(rB.x, rB.y, kB.x, B2B, wb);
        decode_pairs(rB.z, rB.w, kB.y, B2B, wb + 4);
        const uint32_t hereA = (nA >> (8 * c)) & 0xFFu, hereB = (nB >> (8 * c)) & 0xFFu;
        if (hereA) patch(wa, kA, iA, limA, m.esc, p.err);
        if (hereB) patch(wb, kB, iB, limB, m.esc, p.err);
        iA += hereA;
        iB += hereB;
        multiply(c, wa, wb);
    }
    refill();
}

// One step by one warp.  d0 and d1 are its first stages (their copies are in
// flight).  False when a wait gave up.
template <int V, int PH>
__device__ __forceinline__ bool small_step(const Params &p, const SmallShared *sm, const uint8_t *x, Ring &rg,
                                           Feed<PH> &feed, Desc d0, Desc d1) {
    const Mat &m = mat<PH>(p);
    const Step &st = sm->step[PH - 1];
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, tq = q >> 1, qh = q & 1;
    const int slots = p.tokens * p.top_k, nx = PH == 1 ? p.tokens : slots;  // rows of x or h
    const uint32_t half = static_cast<uint32_t>(nx) * 32u, chunk_bytes = 2 * half;
    const size_t rows = static_cast<size_t>(m.G) * kRowsPerGroup;  // of an expert
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains of products
    Words w0 = load_words<V>(m, d0);
    const uint8_t *xl = nullptr;  // the lane's column of x or h
    float *to = nullptr;          // its places of the item's sums, for pairs 2q and 2q + 1
    int pairs = 0;
    bool fresh = true;
    while (d0.live) {
        const Words w1 = load_words<V>(m, d1);
        if (fresh) {
            const Item at = item_at<PH>(st, d0.it);
            const int first = sm->s.seg_first[at.seg];
            pairs = sm->s.seg_n[at.seg];
            // (columns past the last pair repeat it; their results are dropped)
            const int i = first + min(g, pairs - 1);
            xl = x + static_cast<size_t>(PH == 1 ? sm->s.token[i] : i) * 32 + qh * 16;
            to = (PH == 1 ? p.gu : p.d) + (static_cast<size_t>(at.range) * slots + first + 2 * q) * rows +
                 static_cast<size_t>(at.grp) * kRowsPerGroup + g;
        }
        const uint32_t slot = static_cast<uint32_t>(rg.consumed & 1);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_s(rg.bars + 8u * slot, static_cast<uint32_t>(rg.consumed >> 1) & 1u))) {
            if (lane == 0) give_up(p);
            return false;
        }
        const bool live = d0.j + tq < m.T;  // the lane's tile exists (else zeros from the copy)
        const size_t at = static_cast<size_t>(d0.j + tq) * 4 * chunk_bytes;
        const ptrdiff_t lo = PH == 2 ? p.lo - p.hi : 0;
        Desc d2;
        d2.live = false;
        auto multiply = [&](int c, const uint32_t (&wa)[8], const uint32_t (&wb)[8]) {
            uint32_t xw[8];
            const uint8_t *src = xl + at + c * chunk_bytes;
            load_x(xw, src, half, live);
            chunk_mma(acc[c & 1], wa, wb, xw);
            if (PH == 2) {
                load_x(xw, src + lo, half, live);
                chunk_mma(acc[c & 1], wa, wb, xw);
            }
        };
        auto refill = [&]() {
            // the stage is in registers: hand it back to the copy engine.  (It
            // was read only, which needs no proxy fence.)
            __syncwarp();
            d2 = feed.next(p, sm);
            if (d2.live) issue_at<PH>(p, rg, d2);
        };
        stage_products<V>(p, m, d0, w0, rg.base + slot * kStageBytes, multiply, refill);
        ++rg.consumed;
        fresh = d0.last;
        if (fresh) {
            // lane (g, q) holds rows g and g + 8 of pairs 2q and 2q + 1
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (2 * q + i < pairs) {
                    __stcg(to + i * rows, acc[0][i] + acc[1][i]);
                    __stcg(to + i * rows + 8, acc[0][2 + i] + acc[1][2 + i]);
                }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
        }
        d0 = d1;
        d1 = d2;
        w0 = w1;
    }
    return true;
}

__device__ __forceinline__ void add4(float4 &a, const float4 &b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}

__device__ __forceinline__ float4 shfl4(const float4 &v, int from_xor) {
    return make_float4(__shfl_xor_sync(0xFFFFFFFFu, v.x, from_xor), __shfl_xor_sync(0xFFFFFFFFu, v.y, from_xor),
                       __shfl_xor_sync(0xFFFFFFFFu, v.z, from_xor), __shfl_xor_sync(0xFFFFFFFFu, v.w, from_xor));
}

// The 16 sums of a pair's row group over its ranges, 4 to a lane (lane & 3);
// lanes 4 apart add every eighth range, then one another: a fixed order.
__device__ __forceinline__ float4 sum_ranges(const float *src, size_t plane, uint32_t ranges) {
    const int lane = threadIdx.x & 31;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t c = lane >> 2; c < ranges; c += 8)
        add4(v, __ldcg(reinterpret_cast<const float4 *>(src + c * plane) + (lane & 3)));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) add4(v, shfl4(v, o));
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// h from the sums of step 1: a warp takes one pair's row group at a time.
__device__ __forceinline__ void make_hidden(const Params &p, const SmallShared *sm) {
    const int lane = threadIdx.x & 31, slots = p.tokens * p.top_k;
    const uint32_t G = static_cast<uint32_t>(p.up.G), ranges = sm->step[0].ranges;
    const int last = sm->s.n_segs - 1, pairs = sm->s.seg_first[last] + sm->s.seg_n[last];  // that are in use
    const size_t rows = static_cast<size_t>(G) * kRowsPerGroup, plane = static_cast<size_t>(slots) * rows;
    for (uint32_t u = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; u < pairs * G; u += gridDim.x * kWarps) {
        const uint32_t pos = u / G, grp = u - pos * G;
        const float4 v = sum_ranges(p.gu + pos * rows + static_cast<size_t>(grp) * kRowsPerGroup, plane, ranges);
        // lanes 0 and 1: gate rows 0-3 and 4-7; lanes 2 and 3: the up rows
        const float4 up = shfl4(v, 2);
        auto h = [](float g, float t) { return g / (1.f + expf(-g)) * t; };
        const float4 a = make_float4(h(v.x, up.x), h(v.y, up.y), h(v.z, up.z), h(v.w, up.w));
        const float4 b = shfl4(a, 1);
        if (lane == 0) {
            // one piece, in the order 0 4 1 5 2 6 3 7
            const float f[8] = {a.x, b.x, a.y, b.y, a.z, b.z, a.w, b.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
                const float r0 = f[2 * i] - __uint_as_float(hi[i] << 16);
                const float r1 = f[2 * i + 1] - __uint_as_float(hi[i] & 0xFFFF0000u);
                // (an infinite h has no rest)
                lo[i] = pack_bf16(fabsf(r0) < 3.4e38f ? r0 : 0.f, fabsf(r1) < 3.4e38f ? r1 : 0.f);
            }
            const int in = static_cast<int>(grp & 15u);
            const size_t o = piece_at(static_cast<int>(grp >> 4), (in >> 1) & 3, in & 1, slots, static_cast<int>(pos),
                                      in >> 3);
            *reinterpret_cast<uint4 *>(p.hi + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(p.lo + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// y from the sums of step 2: a warp takes 16 values of a token at a time.
__device__ __forceinline__ void make_y(const Params &p, const SmallShared *sm) {
    const int lane = threadIdx.x & 31, slots = p.tokens * p.top_k;
    const uint32_t G = static_cast<uint32_t>(p.down.G), ranges = sm->step[1].ranges;
    const size_t rows = static_cast<size_t>(G) * kRowsPerGroup, plane = static_cast<size_t>(slots) * rows;
    for (uint32_t u = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; u < p.tokens * G; u += gridDim.x * kWarps) {
        const uint32_t t = u / G, grp = u - t * G;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.top_k; ++s) {
            const int i = static_cast<int>(t) * p.top_k + s;
            if (sm->s.expert[i] < 0) continue;
            const float4 v = sum_ranges(p.d + sm->s.place[i] * rows + static_cast<size_t>(grp) * kRowsPerGroup, plane,
                                        ranges);
            const float w = sm->s.weight[i];
            y = make_float4(fmaf(w, v.x, y.x), fmaf(w, v.y, y.y), fmaf(w, v.z, y.z), fmaf(w, v.w, y.w));
        }
        if (lane < 4) {
            const size_t o = static_cast<size_t>(t) * p.H + static_cast<size_t>(grp) * kRowsPerGroup + 4 * lane;
            put_y(p, o, y.x);
            put_y(p, o + 1, y.y);
            put_y(p, o + 2, y.z);
            put_y(p, o + 3, y.w);
        }
    }
}

template <int V>
__global__ void __launch_bounds__(kThreads, 1) moe_small_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    SmallShared *sm = reinterpret_cast<SmallShared *>(base + kRingBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Ring rg;
    rg.bars = smem_addr(sm->s.bars) + static_cast<uint32_t>(warp) * kStages * 8u;
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
            if (threadIdx.x == 0) plan_step<1>(p, sm);
            if (threadIdx.x == 32) plan_step<2>(p, sm);
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
                make_hidden(p, sm);
                if (grid_meet(p, &sm->s, kBarHidden)) {
                    if (ok) small_step<V, 2>(p, sm, p.hi, rg, f2, d0, d1);
                    if (grid_meet(p, &sm->s, kBarDown)) make_y(p, sm);
                }
            }
        }
    }
    finish(p, &sm->s, rg);
}

}  // namespace moe

// ---------------------------------------------------------------------------
// Host side.

namespace {

constexpr uint32_t kSmemLimit = 227 * 1024;

struct MoePlan {
    int sms, segs, nt;
    bool small, local;
    int seg;
    uint32_t range_up, range_down, smem;
    uint64_t n_cnt, cnt_down, cnt_y;
    size_t sync, cnt, scores, xp, hi, lo, gu, d, warp_part, cta_part, total;
};

// Workspace parts; the words that have to be zero between calls come first.
MoePlan plan(const MoeCall &c, int sms) {
    MoePlan pl = {};
    const uint64_t slots = static_cast<uint64_t>(c.tokens) * c.top_k;
    const uint64_t H = c.up->cols, F = c.down->cols;
    pl.sms = sms;
    // (not by this call's tokens: the counters then lie in the same place for
    // every call with these containers, and what another call left there is zero)
    pl.segs = c.experts + moe::kMaxSlots / moe::kSegSmall;
    // few pairs an expert on average: warps share a row group's columns (one
    // with more than eight pairs is read once for every eight)
    pl.small = slots <= 4ull * c.experts || c.tokens <= 8;
    pl.seg = pl.small ? moe::kSegSmall : moe::kSegLarge;
    const uint32_t fixed = 1024 + moe::kRingBytes + align_up(sizeof(moe::SmallShared), 16);
    const uint64_t x_bytes = 2ull * c.tokens * H;
    // little enough for every CTA to do alone: less time than a meeting of the grid
    pl.local = pl.small && fixed + x_bytes <= kSmemLimit && c.tokens * c.experts <= 512 &&
               (c.ids_in || static_cast<uint64_t>(c.tokens) * c.experts * H <= (1u << 18));
    pl.smem = pl.small ? fixed + static_cast<uint32_t>(pl.local ? x_bytes : 0)
                       : 1024 + moe::kRingBytes + moe::kWarps * 2 * moe::kPartBytes + sizeof(moe::Shared);
    pl.range_up = pl.range_down = 4;
    const uint64_t g_up = 2 * F / 16, g_down = H / 16;
    pl.cnt_down = pl.segs * g_up;
    pl.cnt_y = pl.cnt_down + pl.segs * g_down;
    pl.n_cnt = pl.cnt_y + g_down;
    const int most = static_cast<int>(std::min<uint64_t>(slots, pl.seg));  // pairs of a segment
    pl.nt = most <= 8 ? 1 : most <= 16 ? 2 : most <= 32 ? 4 : 8;
    size_t at = 0;
    auto take = [&](uint64_t bytes) {
        const size_t o = at;
        at += align_up(bytes, kAlign);
        return o;
    };
    pl.sync = take(moe::kSyncWords * 4);
    pl.cnt = take(pl.n_cnt * 4);
    pl.scores = take(8ull * c.tokens * c.experts);
    pl.xp = take(2ull * c.tokens * H);
    pl.hi = take(2 * slots * F);
    pl.lo = take(2 * slots * F);
    const auto ranges = [&](uint64_t cols, uint32_t stages) {
        return pl.small ? ((cols / kTile + stage::kNT - 1) / stage::kNT + stages - 1) / stages : 1;
    };
    pl.gu = take(pl.small ? 4 * slots * 2 * F * ranges(H, pl.range_up) : 0);
    pl.d = take(4 * slots * H * ranges(F, pl.range_down));
    pl.warp_part = take(pl.nt == 1 ? 0 : static_cast<uint64_t>(sms) * moe::kWarps * 2 * pl.nt * moe::kPartBytes);
    pl.cta_part = take(static_cast<uint64_t>(sms) * 2 * pl.nt * moe::kPartBytes);
    pl.total = at;
    return pl;
}

int fill_mat(moe::Mat &m, const s12_view *v, int rows_e) {
    const uint64_t R = v->rows, K = v->cols, T = K / kTile;
    if (make_tmap_u8_3d(&m.tm_raw, v->raw, 128, T, R, 128, K, 128, stage::kNT, stage::kRowsPerGroup, 128) != S12_OK ||
        make_tmap_u8_3d(&m.tm_code, v->code, 64, T, R, 64, K / 2, 64, stage::kNT, stage::kRowsPerGroup, 64) != S12_OK)
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

size_t moe_ws_bytes(const MoeCall &c) {
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return 0;
    return plan(c, sms).total;
}

int launch_moe(const MoeCall &c, void *ws, size_t ws_bytes, cudaStream_t stream) {
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return S12_ERR_CUDA;
    const MoePlan pl = plan(c, sms);
    if (ws_bytes < pl.total) return S12_ERR_CAPACITY;
    moe::Params p = {};
    p.H = static_cast<int>(c.up->cols);
    p.F = static_cast<int>(c.down->cols);
    int rc = fill_mat(p.up, c.up, 2 * p.F);
    if (rc == S12_OK) rc = fill_mat(p.down, c.down, p.H);
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
    uint8_t *w = static_cast<uint8_t *>(ws);
    p.sync = reinterpret_cast<uint32_t *>(w + pl.sync);
    p.cnt = reinterpret_cast<uint32_t *>(w + pl.cnt);
    p.n_cnt = static_cast<uint32_t>(pl.n_cnt);
    p.cnt_down = static_cast<uint32_t>(pl.cnt_down);
    p.cnt_y = static_cast<uint32_t>(pl.cnt_y);
    p.scores = reinterpret_cast<double *>(w + pl.scores);
    p.xp = w + pl.xp;
    p.hi = w + pl.hi;
    p.lo = w + pl.lo;
    p.gu = reinterpret_cast<float *>(w + pl.gu);
    p.d = reinterpret_cast<float *>(w + pl.d);
    p.warp_part = reinterpret_cast<float *>(w + pl.warp_part);
    p.cta_part = reinterpret_cast<float *>(w + pl.cta_part);
    p.local = pl.local;
    p.seg = pl.seg;
    p.range_up = pl.range_up;
    p.range_down = pl.range_down;
    const uint32_t smem = pl.smem;
    auto kern = pl.small ? (c.up->version == 1 ? moe::moe_small_kernel<1> : moe::moe_small_kernel<2>)
                         : (c.up->version == 1 ? moe::moe_kernel<1> : moe::moe_kernel<2>);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return S12_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(moe::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs meet, so all have to be resident
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? S12_OK : S12_ERR_CUDA;
}

}  // namespace s12
