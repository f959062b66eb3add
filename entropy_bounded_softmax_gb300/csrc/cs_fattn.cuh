// Device helpers shared by the fused attention kernels (k_fattn_fwd.cu,
// k_fattn_bwd.cu) and the one of several new tokens over a paged cache
// (k_tree.cu): bounded waits of a warp, operand tiles in shared memory and the
// products on them, kept keys, and row stores.
//
// Operand tiles.  R rows of DP (64, 128 or 256) bf16 or fp16, as the tensor
// copies write them with 128-byte swizzling: DP / 64 panels of R rows x 128
// bytes, head elements past D and rows past the sequence filled with zeros.  The
// same tile serves as a K-major operand (rows along M or N, the head along K:
// Q K^T) and, by its descriptor alone, as an MN-major one (the head along N,
// rows along K: P V), so nothing is ever transposed.
#pragma once

#include "cs_tcgen05.cuh"

namespace csd {

// Shared abort flag and limit of a CTA's bounded waits.
struct WaitLimit {
    volatile uint32_t* abort_flag;
    uint64_t cycles;
};

// Waits, as a whole warp, for the barrier's phase of index `phase`; false in
// every lane when any gave up (an abort raised elsewhere, or the limit,
// which raises it), so that the warp's control flow stays uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase, const WaitLimit& w) {
    const uint32_t a = smem_addr(bar);
    const uint32_t parity = static_cast<uint32_t>(phase & 1);
    bool ok = mbar_try_wait<false>(a, parity);
    if (!ok) {
        const long long c0 = clock64();
        for (uint32_t i = 0; i < (1u << 31); ++i) {
            ok = mbar_try_wait<false>(a, parity);
            if (ok || *w.abort_flag) break;
            if (clock64() - c0 > static_cast<long long>(w.cycles)) break;
        }
        if (!ok) *w.abort_flag = 1u;
    }
    return __all_sync(0xffffffffu, ok);
}

// The key head of query head h (an integer division costs the start of a CTA
// a hundred cycles): exact for h < 2^20, whose (h + 1/2) / group lies at least
// 1 / (2 group) from an integer, further than the roundings reach.
__device__ __forceinline__ int head_of(int h, float inv_group) {
    return static_cast<int>((static_cast<float>(h) + 0.5f) * inv_group);
}

// Raises, or lowers, the registers of every thread of this warpgroup (four
// warps, all of which call it) to N, a multiple of 8.  Raising waits for
// registers that the block was launched with and has given up.
template <int N>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}

// The box copies of one R x DP tile whose first row is `row` (BOX: rows of the
// map's box, a divisor of R).
template <int R, int DP, int BOX = R>
__device__ __forceinline__ void load_tile(unsigned char* dst, const void* tmap, int row,
                                          int head, int batch, uint64_t* bar) {
#pragma unroll
    for (int p = 0; p < DP / 64; ++p)
#pragma unroll
        for (int r = 0; r < R; r += BOX)
            tma_load_4d(dst + (p * R + r) * 128, tmap, 64 * p, row + r, head, batch, bar);
}

// The largest of three (NaN operands are passed over, as by fmaxf).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// What 16 rows of a panel add to a descriptor's address.
constexpr uint32_t kDescRows16 = 16 * 128 / 16;

// D[128 x N] = A . B^T on a tile of 128 rows and one of N (their low descriptor
// words), over the first 16 `steps` head elements: those past d_head are
// zeros, and products with them would cost as much as others.
template <int N, int DP, bool FP16 = false>
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b, int steps,
                                          bool leader) {
    constexpr uint32_t idesc = idesc_half(128, N, false, FP16);
    auto one = [&](int ks) {
        mma_bf16_ss(d, a + (ks >> 2) * (128 * 128 / 16) + (ks & 3) * (32 / 16),
                    b + (ks >> 2) * (N * 128 / 16) + (ks & 3) * (32 / 16), idesc, ks > 0, leader);
    };
    if (steps == DP / 16) {
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) one(ks);
    } else {
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks) one(ks);
    }
}

// D[128 x 16 steps] (+)= W[128 x N] . B[N x 16 steps] (N a multiple of 16), W
// bf16 in tensor memory from column w, B from the row of a tile that b, its
// low descriptor word as MN-major operand, names; idesc: of that shape.
// (Columns past 16 steps keep what they held.)
template <int N>
__device__ __forceinline__ void mma_weights(uint32_t d, uint32_t w, uint32_t b, uint32_t idesc,
                                            bool accumulate, bool leader) {
#pragma unroll
    for (int ks = 0; ks < N / 16; ++ks)
        mma_bf16_ts(d, w + 8 * ks, b + ks * kDescRows16, idesc, accumulate || ks > 0, leader);
}

// The low descriptor words of a tile at shared address a: as an operand of
// mma_tiles, and, of R rows, as B of mma_weights.
__device__ __forceinline__ uint32_t tile_desc(uint32_t a) { return desc_low(a, 0); }
template <int R>
__device__ __forceinline__ uint32_t weights_desc(uint32_t a) {
    return desc_low(a, R * 128);
}

// Bits of the 32 columns from `base` that lie below `limit`.
__device__ __forceinline__ uint32_t bits_below(int limit, int base) {
    const int n = limit - base;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// The first and one past the last nonzero byte of row[0, n), by one warp; an
// empty row gives lo >= hi.
__device__ __forceinline__ void warp_nonzero_range(const uint8_t* row, int n, int lane, int& lo,
                                                   int& hi) {
    // Fewer than 16 bytes before and after the aligned 16-byte units; all
    // loads of a round are under way before the first is used.
    const int lead = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15);
    const int h = lead < n ? lead : n;
    const int vecs = (n - h) >> 4;
    const int tail = h + 16 * vecs;
    const uint8_t before = lane < h ? row[lane] : 0;
    const uint8_t after = tail + lane < n ? row[tail + lane] : 0;
    int first = n, past = 0;
    const uint4* units = reinterpret_cast<const uint4*>(row + h);
    for (int v0 = 0; v0 < vecs; v0 += 4 * 32) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int v = v0 + 32 * k + lane;
            x[k] = v < vecs ? __ldg(units + v) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (v0 + 32 * k >= vecs) break;
            // The lowest and the highest word that is not zero.
            const uint32_t low = x[k].x ? x[k].x : x[k].y ? x[k].y : x[k].z ? x[k].z : x[k].w;
            const uint32_t high = x[k].w ? x[k].w : x[k].z ? x[k].z : x[k].y ? x[k].y : x[k].x;
            const int low_at = x[k].x ? 0 : x[k].y ? 4 : x[k].z ? 8 : 12;
            const int high_at = x[k].w ? 12 : x[k].z ? 8 : x[k].y ? 4 : 0;
            const int at = h + 16 * (v0 + 32 * k + lane);
            if (low) {
                first = min(first, at + low_at + ((__ffs(static_cast<int>(low)) - 1) >> 3));
                past = max(past, at + high_at + 4 - (__clz(static_cast<int>(high)) >> 3));
            }
        }
    }
    if (before) {
        first = min(first, lane);
        past = max(past, lane + 1);
    }
    if (after) {
        first = min(first, tail + lane);
        past = max(past, tail + lane + 1);
    }
    lo = __reduce_min_sync(0xffffffffu, first);
    hi = __reduce_max_sync(0xffffffffu, past);
}

// The kept keys among the R (a multiple of 32) from `key`, one bit each, and
// the rows of the tile whose key is removed set to zero: a removed key's
// weight is exactly 0, but 0 times the NaN or infinity that padding may hold
// is not.  By one warp; the caller makes the words and the tile visible.
template <int R, int DP>
__device__ __forceinline__ void mask_tile(const uint8_t* row, int keys, int key,
                                          unsigned char* tile, uint32_t* words, int lane) {
#pragma unroll
    for (int w = 0; w < R / 32; ++w) {
        const int j = key + 32 * w + lane;
        const bool kept = j < keys && row[j] != 0;
        const uint32_t bits = __ballot_sync(0xffffffffu, kept);
        if (lane == 0) words[w] = bits;
        if (!kept) {
#pragma unroll
            for (int p = 0; p < DP / 64; ++p)
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4*>(tile + p * R * 128 + (32 * w + lane) * 128 +
                                              16 * u) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    fence_proxy_async_smem();
}

// 32 fp32 columns c0 .. c0 + 31 times f, rounded to bf16, into row r of a
// 128-row tile as the tensor copies lay it out (so that the 32 lanes' 16-byte
// stores, each to a row of its own, fall in different banks).
__device__ __forceinline__ void stage_row32(unsigned char* tile, int r, int c0,
                                            const uint32_t* v, float f) {
    unsigned char* row = tile + (c0 >> 6) * (128 * 128) + r * 128;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16(__uint_as_float(v[8 * u + 2 * i]) * f,
                             __uint_as_float(v[8 * u + 2 * i + 1]) * f);
        *reinterpret_cast<uint4*>(row + ((((c0 >> 3) & 7) + u) ^ (r & 7)) * 16) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Copies panels P0 .. P0 + N - 1 of rows r0 .. r0 + 31 of a staged tile, which
// this warp has written, to 32 rows of the tensor, whole rows a few lanes at a
// time: `out` its first row, `stride` elements from row to row, `rows` of them
// there, d elements each.  (Tensor copies of the same rows took 1900 cycles a
// panel, 128 bytes at a time.)
template <int N>
__device__ __forceinline__ void store_rows32(const unsigned char* tile, int r0, int p0,
                                             uint16_t* out, int64_t stride, int rows, int d,
                                             int lane) {
    __syncwarp();
#pragma unroll 8
    for (int e = lane; e < 32 * 8 * N; e += 32) {
        const int r = e / (8 * N), u = e % (8 * N);
        const int p = p0 + u / 8, at = 64 * p + 8 * (u % 8);
        const uint4 v = *reinterpret_cast<const uint4*>(
            tile + p * (128 * 128) + (r0 + r) * 128 + (((u % 8) ^ ((r0 + r) & 7)) << 4));
        if (r < rows && at < d) *reinterpret_cast<uint4*>(out + r * stride + at) = v;
    }
}

// The same with zeros, without a tile.
template <int N>
__device__ __forceinline__ void zero_rows32(int p0, uint16_t* out, int64_t stride, int rows,
                                            int d, int lane) {
#pragma unroll 1
    for (int e = lane; e < 32 * 8 * N; e += 32) {
        const int r = e / (8 * N), at = 64 * p0 + 8 * (e % (8 * N));
        if (r < rows && at < d)
            *reinterpret_cast<uint4*>(out + r * stride + at) = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace csd
