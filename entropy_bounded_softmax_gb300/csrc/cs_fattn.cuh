// Device helpers shared by the fused attention kernels (k_fattn_fwd.cu,
// k_fattn_bwd.cu): bounded waits of a warp, operand tiles in shared memory
// and the products on them, kept keys, and row stores.
//
// Operand tiles.  R rows of DP (64 or 128) bf16, as the tensor copies write
// them with 128-byte swizzling: DP / 64 panels of R rows x 128 bytes, head
// elements past D and rows past the sequence filled with zeros.  The same
// tile serves as a K-major operand (rows along M or N, the head along K:
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

// The box copies of one R x DP tile whose first row is `row` (R: rows of the
// map's box).
template <int R, int DP>
__device__ __forceinline__ void load_tile(unsigned char* dst, const void* tmap, int row,
                                          int head, int batch, uint64_t* bar) {
#pragma unroll
    for (int p = 0; p < DP / 64; ++p)
        tma_load_4d(dst + p * R * 128, tmap, 64 * p, row, head, batch, bar);
}

// D[128 x N] = A[128 x DP] . B[N x DP]^T on two tiles.
template <int N, int DP>
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b) {
    constexpr uint32_t idesc = idesc_bf16(128, N, false);
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks)
        mma_bf16_ss(d, smem_desc_sw128(a + (ks >> 2) * (128 * 128) + (ks & 3) * 32, 1024),
                    smem_desc_sw128(b + (ks >> 2) * (N * 128) + (ks & 3) * 32, 1024),
                    idesc, ks > 0);
}

// Bits of the 32 columns from `base` that lie below `limit`.
__device__ __forceinline__ uint32_t bits_below(int limit, int base) {
    const int n = limit - base;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// The first and one past the last nonzero byte of row[0, n), by the whole
// CTA; an empty row gives lo >= hi.  lo_hi: two shared ints; includes two
// __syncthreads.
__device__ __forceinline__ void block_nonzero_range(const uint8_t* row, int n, int* lo_hi,
                                                    int& lo, int& hi) {
    if (threadIdx.x == 0) {
        lo_hi[0] = n;
        lo_hi[1] = 0;
    }
    __syncthreads();
    int first = n, past = 0;
    const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15);
    const int h = head < n ? head : n;
    const int vecs = (n - h) >> 4;
    auto one = [&](int i) {
        if (row[i]) {
            first = min(first, i);
            past = max(past, i + 1);
        }
    };
    for (int i = threadIdx.x; i < h; i += blockDim.x) one(i);
    for (int i = h + 16 * vecs + threadIdx.x; i < n; i += blockDim.x) one(i);
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + h) + v);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (w[i]) {
                const int at = h + 16 * v + 4 * i;
                first = min(first, at + ((__ffs(static_cast<int>(w[i])) - 1) >> 3));
                past = max(past, at + 4 - (__clz(static_cast<int>(w[i])) >> 3));
            }
        }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    past = __reduce_max_sync(0xffffffffu, past);
    if ((threadIdx.x & 31) == 0) {
        atomicMin(&lo_hi[0], first);
        atomicMax(&lo_hi[1], past);
    }
    __syncthreads();
    lo = lo_hi[0];
    hi = lo_hi[1];
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

// 32 fp32 columns c0 .. c0 + 31 times f, rounded to bf16, into a row of d
// elements (d % 8 == 0, the row 16-byte aligned).
__device__ __forceinline__ void store_row32(uint16_t* row, int d, int c0, const uint32_t* v,
                                            float f) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (c0 + 8 * u < d) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16(__uint_as_float(v[8 * u + 2 * i]) * f,
                                 __uint_as_float(v[8 * u + 2 * i + 1]) * f);
            *reinterpret_cast<uint4*>(row + c0 + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace csd
