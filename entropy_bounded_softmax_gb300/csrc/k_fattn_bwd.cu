// Fused attention, backward.  With P_ij = e^(s_ij - lse_i) recomputed from
// the forward's lse, g the gradient of out and delta_i = <g_i, out_i>:
//   dv_j = sum_i P_ij g_i
//   dS_ij = P_ij (<g_i, v_j> - delta_i)
//   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,
// dk and dv summed over the query heads that share a key head.
//
// Two launches of one kernel, so that every sum stays in one CTA's tensor
// memory: no atomics, the same bits every time, no fp32 copy of a gradient
// in memory.  They recompute P twice (seven products instead of five).
//   queries (KV = false)  128 query rows a CTA, over blocks of 64 keys:
//       S = Q K^T, G V^T, dq += dS K.  Before its blocks it takes delta of
//       its rows and leaves delta and lse, in base 2 and padded to whole
//       tiles, in the workspace for the second launch;
//   keys (KV = true)      128 key rows a CTA, over blocks of 64 queries of
//       every head of its group: S^T = K Q^T, V G^T, dv += P^T G,
//       dk += dS^T Q.
// In both the fixed tiles' rows are the lanes of tensor memory, and the
// weights, rounded to bf16 in the columns their scores had, are the next
// product's A operand there.  Roles:
//   warps 0-3, 4-7  the elementwise part of even and odd blocks, one row a
//                   thread, 64 columns of S and of G V^T in registers;
//   warp 8          issues the products: block i's sums, then block i + 2's
//                   scores into the columns that block i has left, so that
//                   the products of one block run under the elementwise
//                   part of the other;
//   warp 9          tensor copies: the two fixed tiles, then the blocks;
//   warp 10         queries with a key mask only: a block's kept keys as
//                   bits, and zeros over the removed keys' rows of K.
//
// P and dS are rounded to bf16, the operand type next to bf16 values (a sum
// over many rows averages those roundings); everything else stays fp32.
#include <math.h>

#include "cs_fattn.cuh"
#include "cs_tensormap.h"

namespace cs {
namespace {

using namespace csd;

constexpr int kBwdThreads = 352;
constexpr int kBwdMmaWarp = 8;
constexpr int kBwdLoadWarp = 9;
constexpr int kBwdMaskWarp = 10;
constexpr uint32_t kBwdTmemCols = 512;
constexpr uint32_t kBarCompute = 1;
constexpr int kBlk = 64;                       // rows of a streamed block

template <int DP>
struct BwdSmem {
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int kBlock = kBlk * DP * 2;
    static constexpr int kStages = 4;
    static constexpr int kA1 = 0;              // Q, or K
    static constexpr int kA2 = kA1 + kTile;    // G, or V
    static constexpr int kB = kA2 + kTile;     // [kStages] of K, V or of Q, G
    static constexpr int kStage = 2 * kBlock;
    static constexpr int kRows = kB + kStages * kStage;   // [kStages][2][64] lse, delta
    static constexpr int kDelta = kRows + kStages * 2 * kBlk * 4;   // [128]
    static constexpr int kBars = kDelta + 128 * 4;
    static constexpr int kNumBars = 1 + 3 * kStages + 2 + 2 + 1 + 1;
    static constexpr int kWords = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [kStages][2]
    static constexpr int kFlags = kWords + kStages * 8;
    static constexpr int kBytes = kFlags + 16 + 1024;
};

template <int DP, bool KV>
__global__ void __launch_bounds__(kBwdThreads, 1)
fattn_bwd_kernel(const FattnTask t, const __grid_constant__ CUtensorMap map_a1,
                 const __grid_constant__ CUtensorMap map_a2,
                 const __grid_constant__ CUtensorMap map_b1,
                 const __grid_constant__ CUtensorMap map_b2) {
    using L = BwdSmem<DP>;
    constexpr int NS = L::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* a_full = bars;                   // the fixed tiles landed
    uint64_t* b_full = a_full + 1;             // [NS] ring stage landed
    uint64_t* b_empty = b_full + NS;           // [NS] products that read it completed
    uint64_t* b_masked = b_empty + NS;         // [NS] removed rows zeroed, bits written
    uint64_t* s_full = b_masked + NS;          // [2] scores of an even, odd block
    uint64_t* w_full = s_full + 2;             // [2] its weights
    uint64_t* sums_full = w_full + 2;          // every sum completed
    uint64_t* drained = sums_full + 1;
    float* rows_s = reinterpret_cast<float*>(smem + L::kRows);
    float* delta_s = reinterpret_cast<float*>(smem + L::kDelta);
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kWords);
    volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags);
    const WaitLimit limit{flags, t.wait_limit_cycles};

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int group = t.heads / t.kv_heads;
    const int fixed_len = KV ? t.key_len : t.query_len;
    const int fixed_heads = KV ? t.kv_heads : t.heads;
    const int BH = t.batch * fixed_heads;
    const int tiles = (fixed_len + 127) / 128;
    // Under the causal mask late queries keep the most keys and early keys
    // have the most queries: longest first in both.
    const int order = static_cast<int>(blockIdx.x / BH);
    const int a0 = 128 * (!KV && t.causal ? tiles - 1 - order : order);
    const int bh = static_cast<int>(blockIdx.x % BH);
    const int b = bh / fixed_heads, ha = bh - b * fixed_heads;
    const int off = t.key_len - t.query_len;   // query i keeps keys j <= i + off
    const int64_t padded = (static_cast<int64_t>(t.query_len) + 127) / 128 * 128;
    float* ws_lse = t.rows;
    float* ws_delta = t.rows + static_cast<int64_t>(t.batch) * t.heads * padded;

    if (threadIdx.x == 0) {
        mbar_init(a_full, 1u);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&b_full[i], 1u);
            mbar_init(&b_empty[i], 1u);
            mbar_init(&b_masked[i], 1u);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1u);
            mbar_init(&w_full[i], 4u);
        }
        mbar_init(sums_full, 1u);
        mbar_init(drained, 1u);
        flags[0] = 0u;
        fence_mbar_init();
    }
    if (warp == kBwdMmaWarp)
        tmem_alloc(const_cast<uint32_t*>(flags) + 1, kBwdTmemCols);
    const uint8_t* mask = t.mask ? t.mask + b * t.mask_stride : nullptr;
    int key_lo = 0, key_hi = t.key_len;
    if (mask)
        block_nonzero_range(mask, t.key_len,
                            reinterpret_cast<int*>(smem + L::kFlags) + 2, key_lo, key_hi);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = flags[1];

    // Blocks first .. first + per - 1 of the streamed side, for each head.
    int first = 0, per = 0;
    const int last = min(a0 + 128, fixed_len) - 1;
    if (KV) {
        // Queries with a kept key in the tile: i >= a0 - off under causal.
        const int lo = t.causal ? max(0, a0 - off) : 0;
        first = lo / kBlk;
        if (lo < t.query_len && a0 < key_hi && last >= key_lo)
            per = (t.query_len + kBlk - 1) / kBlk - first;
    } else {
        const int hi = t.causal ? min(key_hi, last + off + 1) : key_hi;
        first = key_lo / kBlk;
        if (hi > key_lo) per = (hi + kBlk - 1) / kBlk - first;
    }
    const int blocks = KV ? per * group : per;
    // Block i's head on the streamed side and its first row there.
    auto block_head = [&](int i) { return KV ? ha * group + i / per : ha / group; };
    auto block_row = [&](int i) { return kBlk * (first + (KV ? i % per : i)); };
    const uint32_t acc1 = tmem;                // dq, or dv
    const uint32_t acc2 = tmem + DP;           // dk
    auto t_scores = [&](int s) { return tmem + 256 + 128 * s; };
    auto t_grads = [&](int s) { return tmem + 256 + 128 * s + kBlk; };

    if (warp < 8) {
        // ----------------------------------------------------- elementwise
        const int wg = warp >> 2;
        const int quarter = warp & 3;
        const int a = a0 + 32 * quarter + lane;          // this thread's row
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const float c = t.scale * kLog2e;
        float row_lse = 0.0f, row_delta = 0.0f;
        if (!KV) {
            // delta: DP / 8 lanes a row, 16 bytes of out and of g each.
            constexpr int LR = DP / 8;
            const int u = lane % LR;
#pragma unroll 4
            for (int r = 16 * warp + lane / LR; r < 16 * warp + 16; r += 32 / LR) {
                const int i = a0 + r;
                float d = 0.0f;
                if (i < t.query_len && 8 * u < t.d_head) {
                    const uint4 x = *reinterpret_cast<const uint4*>(
                        t.out + b * t.o_stride[0] + ha * t.o_stride[1] + i * t.o_stride[2] + 8 * u);
                    const uint4 y = *reinterpret_cast<const uint4*>(
                        t.go + b * t.go_stride[0] + ha * t.go_stride[1] + i * t.go_stride[2] + 8 * u);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        d = fmaf(InBF16::lo(xs[k]), InBF16::lo(ys[k]), d);
                        d = fmaf(InBF16::hi(xs[k]), InBF16::hi(ys[k]), d);
                    }
                }
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                if (u == 0) delta_s[r] = d;
            }
            // An empty row, and a row past the last, gets lse = +inf: P = 0.
            row_lse = INFINITY;
            if (a < t.query_len) {
                const float x = t.lse[static_cast<int64_t>(bh) * t.query_len + a];
                if (x != -INFINITY) row_lse = x * kLog2e;
            }
            named_barrier(kBarCompute, 256);
            row_delta = delta_s[a - a0];
            if (wg == 0) {
                ws_lse[bh * padded + a] = row_lse;
                ws_delta[bh * padded + a] = row_delta;
            }
        }
        bool ok = true;
        for (int i = wg; i < blocks; i += 2) {
            const int st = i % NS;
            ok = warp_wait(&s_full[wg], i >> 1, limit);
            if (KV && ok) ok = warp_wait(&b_full[st], i / NS, limit);
            if (!KV && mask && ok) ok = warp_wait(&b_masked[st], i / NS, limit);
            if (!ok) break;
            tc_fence_after_sync();
            const int b0 = block_row(i);
            uint32_t s[64], g[64];
            tmem_ld32_async(t_scores(wg) + lanes, s);
            tmem_ld32_async(t_scores(wg) + lanes + 32, s + 32);
            tmem_ld32_async(t_grads(wg) + lanes, g);
            tmem_ld32_async(t_grads(wg) + lanes + 32, g + 32);
            tmem_wait_ld<64>(s);
            tmem_wait_ld<64>(g);
            if (KV) {
                // Columns are queries.  Rows of removed keys are not treated
                // here: their sums are replaced by zeros at the end.
                const float4* lse4 = reinterpret_cast<const float4*>(rows_s + 2 * kBlk * st);
                const float4* delta4 = lse4 + kBlk / 4;
                // Causal: query b0 + k keeps this key from column `from` on.
                const int from = t.causal ? a - off - b0 : 0;
                const bool edge = t.causal && a0 + 32 * quarter + 31 - off > b0;
#pragma unroll
                for (int k4 = 0; k4 < kBlk / 4; ++k4) {
                    const float4 le = lse4[k4], de = delta4[k4];
                    const float ls[4] = {le.x, le.y, le.z, le.w};
                    const float ds[4] = {de.x, de.y, de.z, de.w};
                    float p[4], d[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int k = 4 * k4 + x;
                        p[x] = ex2(fmaf(__uint_as_float(s[k]), c, -ls[x]));
                        d[x] = p[x] * (__uint_as_float(g[k]) - ds[x]);
                        if (edge && k < from) p[x] = d[x] = 0.0f;
                    }
                    s[2 * k4] = pack_bf16(p[0], p[1]);
                    s[2 * k4 + 1] = pack_bf16(p[2], p[3]);
                    g[2 * k4] = pack_bf16(d[0], d[1]);
                    g[2 * k4 + 1] = pack_bf16(d[2], d[3]);
                }
                tmem_st32(t_scores(wg) + lanes, s);
            } else {
                // Columns are keys.
                const int limit_row = t.causal ? min(t.key_len, a + off + 1) : t.key_len;
                const int limit_warp =
                    t.causal ? min(t.key_len, a0 + 32 * quarter + off + 1) : t.key_len;
                uint2 kept = make_uint2(~0u, ~0u);
                if (mask) kept = *reinterpret_cast<const uint2*>(words + 2 * st);
                const bool edge = limit_warp < b0 + kBlk || (kept.x & kept.y) != ~0u;
                const uint32_t bits[2] = {kept.x & bits_below(limit_row, b0),
                                          kept.y & bits_below(limit_row, b0 + 32)};
#pragma unroll
                for (int k2 = 0; k2 < kBlk / 2; ++k2) {
                    float d[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int k = 2 * k2 + x;
                        const float p = ex2(fmaf(__uint_as_float(s[k]), c, -row_lse));
                        d[x] = p * (__uint_as_float(g[k]) - row_delta);
                        if (edge && !((bits[k >> 5] >> (k & 31)) & 1u)) d[x] = 0.0f;
                    }
                    g[k2] = pack_bf16(d[0], d[1]);
                }
            }
            tmem_st32(t_grads(wg) + lanes, g);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_full[wg]);
        }
        if (ok && blocks > 0) ok = warp_wait(sums_full, 0, limit);
        if (ok) {
            tc_fence_after_sync();
            // The rows' sums: keys: dv by the first four warps, dk by the
            // others; queries: half of dq's columns each.
            constexpr int kCols = KV ? DP : DP / 2;
            const int c0 = KV ? 0 : wg * kCols;
            const uint32_t from = (KV && wg == 1 ? acc2 : acc1) + lanes + c0;
            uint16_t* row;
            if (KV && wg == 0)
                row = t.dv + b * t.dv_stride[0] + ha * t.dv_stride[1] + a * t.dv_stride[2];
            else if (KV)
                row = t.dk + b * t.dk_stride[0] + ha * t.dk_stride[1] + a * t.dk_stride[2];
            else
                row = t.dq + b * t.dq_stride[0] + ha * t.dq_stride[1] + a * t.dq_stride[2];
            const float f = KV && wg == 0 ? 1.0f : t.scale;
            const bool live = a < fixed_len;
            const bool zero = blocks == 0 || (KV && mask && live && mask[a] == 0);
#pragma unroll
            for (int u = 0; u < kCols / 32; ++u) {
                uint32_t x[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = 0u;
                if (blocks > 0) {
                    tmem_ld32_async(from + 32 * u, x);
                    tmem_wait_ld<32>(x);
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = zero ? 0u : x[k];
                if (live) store_row32(row, t.d_head, c0 + 32 * u, x, f);
            }
        }
    } else if (warp == kBwdMmaWarp) {
        // ----------------------------------------------------- MMA issuer
        const uint32_t a1 = smem_addr(smem + L::kA1), a2 = smem_addr(smem + L::kA2);
        const uint32_t b1 = smem_addr(smem + L::kB), b2 = b1 + L::kBlock;
        auto scores = [&](int i) {
            if (lane == 0) {
                const uint32_t st = (i % NS) * L::kStage;
                mma_tiles<kBlk, DP>(t_scores(i & 1), a1, b1 + st);
                mma_tiles<kBlk, DP>(t_grads(i & 1), a2, b2 + st);
                mma_commit(&s_full[i & 1]);
            }
            __syncwarp();
        };
        bool ok = blocks == 0 || warp_wait(a_full, 0, limit);
        uint64_t* ready = !KV && mask ? b_masked : b_full;
        for (int i = 0; i < 2 && i < blocks && ok; ++i) {
            ok = warp_wait(&ready[i % NS], i / NS, limit);
            if (ok) scores(i);
        }
        for (int i = 0; i < blocks && ok; ++i) {
            ok = warp_wait(&w_full[i & 1], i >> 1, limit);
            if (!ok) break;
            tc_fence_after_sync();
            if (lane == 0) {
                const uint32_t st = (i % NS) * L::kStage;
                if (KV) {
                    mma_weights<kBlk, DP>(acc1, t_scores(i & 1), b2 + st, i > 0);
                    mma_weights<kBlk, DP>(acc2, t_grads(i & 1), b1 + st, i > 0);
                } else {
                    mma_weights<kBlk, DP>(acc1, t_grads(i & 1), b1 + st, i > 0);
                }
                mma_commit(&b_empty[i % NS]);
                if (i == blocks - 1) mma_commit(sums_full);
            }
            __syncwarp();
            if (i + 2 < blocks) {
                ok = warp_wait(&ready[(i + 2) % NS], (i + 2) / NS, limit);
                if (ok) scores(i + 2);
            }
        }
        // No product may be in flight when the tensor memory is freed.
        if (lane == 0) {
            mma_commit(drained);
            mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
        }
        __syncwarp();
    } else if (warp == kBwdLoadWarp) {
        // --------------------------------------------------------- loader
        int issued = 0;
        for (int i = 0; i < blocks; ++i) {
            const int st = i % NS;
            if (i >= NS && !warp_wait(&b_empty[st], i / NS - 1, limit)) break;
            if (lane == 0) {
                if (i == 0) {
                    mbar_arrive_expect_tx(a_full, 2 * L::kTile);
                    load_tile<128, DP>(smem + L::kA1, &map_a1, a0, ha, b, a_full);
                    load_tile<128, DP>(smem + L::kA2, &map_a2, a0, ha, b, a_full);
                }
                unsigned char* at = smem + L::kB + st * L::kStage;
                const int hb = block_head(i), row = block_row(i);
                mbar_arrive_expect_tx(&b_full[st], L::kStage + (KV ? 2 * kBlk * 4 : 0));
                load_tile<kBlk, DP>(at, &map_b1, row, hb, b, &b_full[st]);
                load_tile<kBlk, DP>(at + L::kBlock, &map_b2, row, hb, b, &b_full[st]);
                if (KV) {
                    const int64_t r = (static_cast<int64_t>(b) * t.heads + hb) * padded + row;
                    bulk_load(rows_s + 2 * kBlk * st, ws_lse + r, kBlk * 4, &b_full[st]);
                    bulk_load(rows_s + 2 * kBlk * st + kBlk, ws_delta + r, kBlk * 4,
                              &b_full[st]);
                }
            }
            __syncwarp();
            issued = i + 1;
        }
        // After an abort copies may still be in flight: none may land in
        // shared memory after the CTA exits (bounded waits).
        if (*limit.abort_flag && lane == 0 && issued > 0) {
            mbar_wait<false>(a_full, 0u, t.wait_limit_cycles);
            for (int i = max(0, issued - NS); i < issued; ++i)
                mbar_wait<false>(&b_full[i % NS], (i / NS) & 1, t.wait_limit_cycles);
        }
        __syncwarp();
    } else if (!KV && warp == kBwdMaskWarp && mask) {
        // ------------------------------------------------------ key masks
        for (int i = 0; i < blocks; ++i) {
            const int st = i % NS;
            if (!warp_wait(&b_full[st], i / NS, limit)) break;
            mask_tile<kBlk, DP>(mask, t.key_len, block_row(i), smem + L::kB + st * L::kStage,
                                words + 2 * st, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_masked[st]);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kBwdMmaWarp) tmem_dealloc(tmem, kBwdTmemCols);
    if (threadIdx.x == 0 && flags[0]) raise_error(t.err, kBitTimeout);
}

template <int DP, bool KV>
cudaError_t launch_bwd(const FattnTask& t, int slot, cudaStream_t stream) {
    const void* kern = reinterpret_cast<const void*>(fattn_bwd_kernel<DP, KV>);
    const int smem = BwdSmem<DP>::kBytes;
    cudaError_t e = ensure_smem_attribute(kern, slot, smem, false);
    if (e != cudaSuccess) return e;
    constexpr int RQ = KV ? kBlk : 128, RK = KV ? 128 : kBlk;
    CUtensorMap mq, mg, mk, mv;
    if (!encode_heads_map(&mq, t.q, t, t.heads, t.query_len, t.q_stride, RQ) ||
        !encode_heads_map(&mg, t.go, t, t.heads, t.query_len, t.go_stride, RQ) ||
        !encode_heads_map(&mk, t.k, t, t.kv_heads, t.key_len, t.k_stride, RK) ||
        !encode_heads_map(&mv, t.v, t, t.kv_heads, t.key_len, t.v_stride, RK))
        return cudaErrorInvalidValue;
    const int64_t length = KV ? t.key_len : t.query_len;
    const int64_t heads = KV ? t.kv_heads : t.heads;
    const int64_t grid = (length + 127) / 128 * t.batch * heads;
    if (grid == 0) return cudaSuccess;
    fattn_bwd_kernel<DP, KV><<<static_cast<unsigned>(grid), kBwdThreads, smem, stream>>>(
        t, KV ? mk : mq, KV ? mv : mg, KV ? mq : mk, KV ? mg : mv);
    return cudaGetLastError();
}

template <int DP>
cudaError_t launch_both(const FattnTask& t, int slot, cudaStream_t stream) {
    const cudaError_t e = launch_bwd<DP, false>(t, slot, stream);
    return e == cudaSuccess ? launch_bwd<DP, true>(t, slot + 1, stream) : e;
}

}  // namespace

cudaError_t launch_fattn_backward(const FattnTask& task, cudaStream_t stream) {
    return task.d_head <= 64 ? launch_both<64>(task, 58, stream)
                             : launch_both<128>(task, 60, stream);
}

}  // namespace cs
