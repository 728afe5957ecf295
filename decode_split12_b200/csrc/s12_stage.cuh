// s12_stage.cuh -- the per-warp building blocks of the fused decode-GEMV and
// the mixture-of-experts layer: a stage of two tiles of a 16-row group in
// shared memory, its copies and metadata, the warp-level product, and the
// deal of blocks to warps.
#pragma once

#include <cuda.h>

#include "s12_device.cuh"

namespace s12 {
namespace stage {

constexpr int kRowsPerGroup = 16;
constexpr int kNT = 2;       // tiles per stage
constexpr uint32_t kRawTile = kRowsPerGroup * 128;   // raw plane of one block
constexpr uint32_t kCodeTile = kRowsPerGroup * 64;   // code plane of one block
constexpr uint32_t kRawStage = kNT * kRawTile;
constexpr uint32_t kStageBytes = kNT * (kRawTile + kCodeTile);
static_assert(kStageBytes % 1024 == 0, "stages keep the swizzle atom alignment");

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// d += A * B for one m16n8k16 product, BF16 operands, FP32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mbar_init_s(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx_s(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Wait for phase `parity` of the barrier; false after about a second.
__device__ __forceinline__ bool mbar_wait_s(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kWaitCycles) return false;
    return true;
}

// 3-D TMA copy of one box into this CTA's shared memory, completing on bar.
__device__ __forceinline__ void tma3d(uint32_t dst, const CUtensorMap *tm, int c0, int c1, int c2, uint32_t bar,
                                      uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

// First block of warp unit u's range: floor(u * n_blocks / n_units), from a
// double-precision quotient (the product is below 2^53) corrected to the
// exact floor; cheaper than a 64-bit integer division.
__device__ __forceinline__ long long unit_start(long long u, long long n_blocks, int n_units) {
    const long long x = u * n_blocks;
    long long q = static_cast<long long>(static_cast<double>(x) / static_cast<double>(n_units));
    if (q * n_units > x)
        --q;
    else if ((q + 1) * n_units <= x)
        ++q;
    return q;
}

// ---------------------------------------------------------------------------
// Metadata.  Lane (g, q) of a stage works on tile tq = q / 2 of the stage
// (its columns 64 (q % 2) .. +63 of that tile) for rows g and g+8, so it needs
// per row one base and the tile row's escape span [s, e).  They are loaded a
// stage ahead into a Meta (rows past the end and lanes past the stage's last
// tile read as base 0 with an empty span):
//   version 1:  base[t], esc_off[t], esc_off[t+1]     (t = r*T + j + tq)
//   version 2:  tmeta of the stage's two tiles, and the row's escape offset
//               row_esc[r] when the stage starts a row group; the spans
//               follow from a running offset per row.
struct Meta {
    uint32_t a0, a1, a2;  // row g
    uint32_t b0, b1, b2;  // row g + 8
};

// (M: any description of a matrix with its tile metadata `meta` and `off`,
// rows R and tiles per row T; the loaded words are kept as they are: any arithmetic on them here would
// make the warp wait for the loads a stage early)
template <int V, class M>
__device__ __forceinline__ void load_row_meta(const M &m, int r, int j, int len, int tq, bool seg_start,
                                              uint32_t &w0, uint32_t &w1, uint32_t &w2) {
    w0 = w1 = w2 = 0u;
    if (r >= m.R) return;
    const size_t t0 = static_cast<size_t>(r) * m.T + j;
    if (V == 1) {
        if (tq < len) {
            w0 = __ldg(static_cast<const uint8_t *>(m.meta) + t0 + tq);
            w1 = __ldg(m.off + t0 + tq);
            w2 = __ldg(m.off + t0 + tq + 1);
        }
    } else {
        const uint16_t *tm = static_cast<const uint16_t *>(m.meta) + t0;
        w0 = __ldg(tm);
        if (len > 1) w1 = __ldg(tm + 1);
        if (seg_start) w2 = __ldg(m.off + r);
    }
}

// Escape counts of tiles 0 .. j-1 of row r (version 2), summed across the
// quad (every lane of the warp calls it; lane q takes tiles q, q+4, ...).
template <class M>
__device__ __forceinline__ uint32_t prefix_count_v2(const M &m, int r, int j, int q) {
    uint32_t s = 0;
    if (r < m.R) {
        const uint16_t *tm = static_cast<const uint16_t *>(m.meta) + static_cast<size_t>(r) * m.T;
        for (int k = q; k < j; k += 4) s += __ldg(tm + k) >> 8;
    }
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
    return s;
}

// A row's base and escape span [s, e) for the lane's tile; `run` is the
// row's escape offset at the stage's first tile (version 2), advanced past
// the stage.
template <int V>
__device__ __forceinline__ void row_span(uint32_t w0, uint32_t w1, uint32_t w2, int tq, uint32_t &run, uint32_t &base,
                                         uint32_t &s, uint32_t &e) {
    if (V == 1) {
        base = w0;
        s = w1;
        e = w2;
    } else {
        const uint32_t c0 = w0 >> 8, c1 = w1 >> 8;
        base = (tq ? w1 : w0) & 0xFFu;
        s = run + (tq ? c0 : 0u);
        e = s + (tq ? c1 : c0);
        run += c0 + c1;
    }
}

// Escape-nibble counts of the lane's four 16-weight chunks of one row, one
// byte each (code words cw[0..3]: chunk c is cw[c/2].{x,y} or .{z,w}).
__device__ __forceinline__ uint32_t chunk_counts(uint4 c01, uint4 c23) {
    return __popc(escape_nibbles(c01.x) | (escape_nibbles(c01.y) >> 1)) |
           (__popc(escape_nibbles(c01.z) | (escape_nibbles(c01.w) >> 1)) << 8) |
           (__popc(escape_nibbles(c23.x) | (escape_nibbles(c23.y) >> 1)) << 16) |
           (__popc(escape_nibbles(c23.z) | (escape_nibbles(c23.w) >> 1)) << 24);
}

}  // namespace stage
}  // namespace s12
