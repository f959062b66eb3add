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
//   queries (KV = false)  128 query rows a CTA, over blocks of 128 keys:
//       S = Q K^T, G V^T, dq += dS K.  Before its blocks it takes delta of
//       its rows and leaves delta and lse, in base 2 and padded to whole
//       tiles, in the workspace for the second launch;
//   keys (KV = true)      128 key rows a CTA, over blocks of 128 queries of
//       every head of its group: S^T = K Q^T, V G^T, dv += P^T G,
//       dk += dS^T Q.
// In both the fixed tiles' rows are the lanes of tensor memory, and the
// weights, rounded to bf16 in columns their scores had, are the next
// product's A operand there.  Products of 128 columns, because one of 64
// reads its A tile from shared memory twice as often and is bound by that.
//
// Tensor memory holds two sums, S and G V^T (keys), or one sum, S and two of
// G V^T (queries).  The elementwise part has two phases, P from S and dS from
// P and G V^T, and the products are issued so that each phase runs under
// products that do not wait for it:
//   keys     dv(i), S(i+1), dk(i), G V^T(i+1): P(i+1) under dk(i) and
//            G V^T(i+1), dS(i) under dv(i) and S(i+1);
//   queries  S(i+1), G V^T(i+1), dq(i): P(i) and dS(i) under the first two.
// Roles:
//   warps 0-7   the elementwise part, a row and 64 of its columns a thread
//               (warps w and w + 4 share the rows of lanes 32 (w % 4) ..);
//   warp 8      issues the products;
//   warp 9      tensor copies: the two fixed tiles, then the blocks;
//   warp 10     queries with a key mask only: a block's kept keys as bits,
//               and zeros over the removed keys' rows of K.
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
constexpr uint32_t kBarElementwise = 1;
constexpr uint32_t kElementwise = 256;         // threads

// The first streamed tensor (K, or Q) is read by a block's first and last
// product, the second (V, or G) by the ones between: three stages and two.
template <int DP>
struct BwdSmem {
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int kStages1 = 3, kStages2 = 2, kStagesR = 2;
    static constexpr int kA1 = 0;              // Q, or K
    static constexpr int kA2 = kA1 + kTile;    // G, or V
    static constexpr int kB1 = kA2 + kTile;
    static constexpr int kB2 = kB1 + kStages1 * kTile;
    static constexpr int kRows = kB2 + kStages2 * kTile;  // [kStagesR][2][128] lse, delta
    static constexpr int kBars = kRows + kStagesR * 2 * 128 * 4;
    static constexpr int kNumBars =
        1 + 3 * kStages1 + 2 * kStages2 + 2 * kStagesR + 6 + 2;
    static constexpr int kWords = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [kStages1][4]
    static constexpr int kFlags = kWords + kStages1 * 16;
    static constexpr int kBytes = kFlags + 16;
};

// D[128 x DP] (+)= W[128 x 128] . B[128 x DP], W bf16 in tensor memory, the
// two halves of its columns 64 columns of 32 bits apart; B a tile.
template <int DP>
__device__ __forceinline__ void mma_weights(uint32_t d, uint32_t w, uint32_t b,
                                            bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16(128, DP, true);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
        mma_bf16_ts(d, w + 64 * (ks >> 2) + 8 * (ks & 3),
                    smem_desc_mn_sw128(b + ks * 2048, 128 * 128, 1024), idesc,
                    accumulate || ks > 0);
}

template <int DP, bool KV>
__global__ void __launch_bounds__(kBwdThreads, 1)
fattn_bwd_kernel(const FattnTask t, const __grid_constant__ CUtensorMap map_a1,
                 const __grid_constant__ CUtensorMap map_a2,
                 const __grid_constant__ CUtensorMap map_b1,
                 const __grid_constant__ CUtensorMap map_b2) {
    using L = BwdSmem<DP>;
    constexpr int N1 = L::kStages1, N2 = L::kStages2, NR = L::kStagesR;
    // The tiles need 1024-byte alignment, and fill the shared memory that a
    // CTA can have up to a few hundred bytes; there are no static variables.
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* a_full = bars;                   // the fixed tiles landed
    uint64_t* b1_full = a_full + 1;            // [N1] ring stage landed
    uint64_t* b1_empty = b1_full + N1;         // [N1] products that read it completed
    uint64_t* b1_masked = b1_empty + N1;       // [N1] removed rows zeroed, bits written
    uint64_t* b2_full = b1_masked + N1;        // [N2]
    uint64_t* b2_empty = b2_full + N2;
    uint64_t* r_full = b2_empty + N2;          // [NR] keys: lse and delta landed
    uint64_t* r_empty = r_full + NR;
    uint64_t* s_full = r_empty + NR;           // a block's scores
    uint64_t* s_read = s_full + 1;             // queries: in registers
    uint64_t* g_full = s_read + 1;             // [2] its G V^T, by buffer
    uint64_t* p_full = g_full + 2;             // keys: its P
    uint64_t* d_full = p_full + 1;             // its dS
    uint64_t* sums_full = d_full + 1;          // every sum completed
    uint64_t* drained = sums_full + 1;
    float* rows_s = reinterpret_cast<float*>(smem + L::kRows);
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
        for (int i = 0; i < N1; ++i) {
            mbar_init(&b1_full[i], 1u);
            mbar_init(&b1_empty[i], 1u);
            mbar_init(&b1_masked[i], 1u);
        }
        for (int i = 0; i < N2; ++i) {
            mbar_init(&b2_full[i], 1u);
            mbar_init(&b2_empty[i], 1u);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&r_full[i], 1u);
            mbar_init(&r_empty[i], 8u);
        }
        mbar_init(s_full, 1u);
        mbar_init(s_read, 8u);
        mbar_init(&g_full[0], 1u);
        mbar_init(&g_full[1], 1u);
        mbar_init(p_full, 8u);
        mbar_init(d_full, 8u);
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
        first = lo >> 7;
        if (lo < t.query_len && a0 < key_hi && last >= key_lo)
            per = ((t.query_len + 127) >> 7) - first;
    } else {
        const int hi = t.causal ? min(key_hi, last + off + 1) : key_hi;
        first = key_lo >> 7;
        if (hi > key_lo) per = ((hi + 127) >> 7) - first;
    }
    const int blocks = KV ? per * group : per;
    // Block i's head on the streamed side and its first row there.
    auto block_head = [&](int i) { return KV ? ha * group + i / per : ha / group; };
    auto block_row = [&](int i) { return (first + (KV ? i % per : i)) << 7; };
    const uint32_t acc1 = tmem;                // dq, or dv
    const uint32_t acc2 = tmem + DP;           // keys: dk
    const uint32_t t_s = tmem + (KV ? 256 : 128);
    // G V^T of block i: keys: one buffer; queries: two, because a block's may
    // complete before every warp has waited for the one before.
    auto g_buf = [&](int i) { return KV ? 1 : i & 1; };
    auto g_phase = [&](int i) { return KV ? i : i >> 1; };
    auto t_g = [&](int i) { return tmem + 256 + 128 * g_buf(i); };

    if (warp < 8) {
        // ----------------------------------------------------- elementwise
        const int half = warp >> 2;
        const int quarter = warp & 3;
        const int a = a0 + 32 * quarter + lane;          // this thread's row
        const uint32_t at = (static_cast<uint32_t>(quarter * 32) << 16) + 64 * half;
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
                if (u == 0) rows_s[r] = d;
            }
            // An empty row, and a row past the last, gets lse = +inf: P = 0.
            row_lse = INFINITY;
            if (a < t.query_len) {
                const float x = t.lse[static_cast<int64_t>(bh) * t.query_len + a];
                if (x != -INFINITY) row_lse = x * kLog2e;
            }
            named_barrier(kBarElementwise, kElementwise);
            row_delta = rows_s[a - a0];
            if (half == 0) {
                ws_lse[bh * padded + a] = row_lse;
                ws_delta[bh * padded + a] = row_delta;
            }
        }
        bool ok = true;
        for (int i = 0; i < blocks; ++i) {
            const int st = i % NR;
            const int b0 = block_row(i) + 64 * half;     // first of this thread's columns
            const float4* lse4 = reinterpret_cast<const float4*>(rows_s + 256 * st + 64 * half);
            const float4* delta4 = lse4 + 32;
            if (KV) ok = warp_wait(&r_full[st], i / NR, limit);
            if (!KV && mask) ok = warp_wait(&b1_masked[i % N1], i / N1, limit);
            if (ok) ok = warp_wait(s_full, i, limit);
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t s[64];
            tmem_ld32_async(t_s + at, s);
            tmem_ld32_async(t_s + at + 32, s + 32);
            tmem_wait_ld<64>(s);
            if (!KV) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
            }
            if (KV) {
                // Columns are queries.  Rows of removed keys are not treated
                // here: their sums are replaced by zeros at the end.
                // Causal: query b0 + k keeps this key from column `from` on.
                const int from = t.causal ? a - off - b0 : 0;
                const bool edge = t.causal && a0 + 32 * quarter + 31 - off > b0;
                uint32_t w[32];
#pragma unroll
                for (int k4 = 0; k4 < 16; ++k4) {
                    const float4 le = lse4[k4];
                    const float ls[4] = {le.x, le.y, le.z, le.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int k = 4 * k4 + x;
                        float p = ex2(fmaf(__uint_as_float(s[k]), c, -ls[x]));
                        if (edge && k < from) p = 0.0f;
                        s[k] = __float_as_uint(p);
                    }
                    w[2 * k4] = pack_bf16(__uint_as_float(s[4 * k4]),
                                          __uint_as_float(s[4 * k4 + 1]));
                    w[2 * k4 + 1] = pack_bf16(__uint_as_float(s[4 * k4 + 2]),
                                              __uint_as_float(s[4 * k4 + 3]));
                }
                tmem_st32(t_s + at, w);
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            } else {
                // Columns are keys.
                const int limit_row = t.causal ? min(t.key_len, a + off + 1) : t.key_len;
                const int limit_warp =
                    t.causal ? min(t.key_len, a0 + 32 * quarter + off + 1) : t.key_len;
                uint2 kept = make_uint2(~0u, ~0u);
                if (mask) kept = *reinterpret_cast<const uint2*>(words + 4 * (i % N1) + 2 * half);
                const bool edge = limit_warp < b0 + 64 || (kept.x & kept.y) != ~0u;
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    s[k] = __float_as_uint(ex2(fmaf(__uint_as_float(s[k]), c, -row_lse)));
                if (edge) {
                    const uint32_t bits[2] = {kept.x & bits_below(limit_row, b0),
                                              kept.y & bits_below(limit_row, b0 + 32)};
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (!((bits[k >> 5] >> (k & 31)) & 1u)) s[k] = 0u;
                }
            }
            ok = warp_wait(&g_full[g_buf(i)], g_phase(i), limit);
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t g[64];
            tmem_ld32_async(t_g(i) + at, g);
            tmem_ld32_async(t_g(i) + at + 32, g + 32);
            tmem_wait_ld<64>(g);
            // dS; 0 where P is 0, whatever G V^T holds there (a removed
            // value's NaN, a causally removed query's infinity).
#pragma unroll
            for (int k4 = 0; k4 < 16; ++k4) {
                float4 de = make_float4(row_delta, row_delta, row_delta, row_delta);
                if (KV) de = delta4[k4];
                const float ds[4] = {de.x, de.y, de.z, de.w};
                float d[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = __uint_as_float(s[4 * k4 + x]);
                    d[x] = p * (__uint_as_float(g[4 * k4 + x]) - ds[x]);
                    if (p == 0.0f) d[x] = 0.0f;
                }
                g[2 * k4] = pack_bf16(d[0], d[1]);
                g[2 * k4 + 1] = pack_bf16(d[2], d[3]);
            }
            tmem_st32(t_g(i) + at, g);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(d_full);
                if (KV) mbar_arrive(&r_empty[st]);
            }
        }
        if (ok && blocks > 0) ok = warp_wait(sums_full, 0, limit);
        if (ok) {
            tc_fence_after_sync();
            // The rows' sums: keys: dv by the first four warps, dk by the
            // others; queries: half of dq's columns each.
            constexpr int kCols = KV ? DP : DP / 2;
            const int c0 = KV ? 0 : half * kCols;
            const uint32_t from = (KV && half == 1 ? acc2 : acc1) +
                                  (static_cast<uint32_t>(quarter * 32) << 16) + c0;
            uint16_t* row;
            if (KV && half == 0)
                row = t.dv + b * t.dv_stride[0] + ha * t.dv_stride[1] + a * t.dv_stride[2];
            else if (KV)
                row = t.dk + b * t.dk_stride[0] + ha * t.dk_stride[1] + a * t.dk_stride[2];
            else
                row = t.dq + b * t.dq_stride[0] + ha * t.dq_stride[1] + a * t.dq_stride[2];
            const float f = KV && half == 0 ? 1.0f : t.scale;
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
        const uint32_t b1 = smem_addr(smem + L::kB1), b2 = smem_addr(smem + L::kB2);
        auto tile1 = [&](int i) { return b1 + (i % N1) * L::kTile; };
        auto tile2 = [&](int i) { return b2 + (i % N2) * L::kTile; };
        uint64_t* ready1 = !KV && mask ? b1_masked : b1_full;
        // S of block i, G V^T of block i, once their tiles are there.
        auto scores = [&](int i) {
            if (!warp_wait(&ready1[i % N1], i / N1, limit)) return false;
            if (lane == 0) {
                mma_tiles<128, DP>(t_s, a1, tile1(i));
                mma_commit(s_full);
            }
            __syncwarp();
            return true;
        };
        auto grads = [&](int i) {
            if (!warp_wait(&b2_full[i % N2], i / N2, limit)) return false;
            if (lane == 0) {
                mma_tiles<128, DP>(t_g(i), a2, tile2(i));
                mma_commit(&g_full[g_buf(i)]);
                if (!KV) mma_commit(&b2_empty[i % N2]);
            }
            __syncwarp();
            return true;
        };
        bool ok = blocks == 0 ||
                  (warp_wait(a_full, 0, limit) && scores(0) && grads(0));
        for (int i = 0; i < blocks && ok; ++i) {
            const bool more = i + 1 < blocks;
            if (KV) {
                ok = warp_wait(p_full, i, limit);
                if (!ok) break;
                tc_fence_after_sync();
                if (lane == 0) {
                    mma_weights<DP>(acc1, t_s, tile2(i), i > 0);
                    mma_commit(&b2_empty[i % N2]);
                }
                __syncwarp();
                if (more) ok = scores(i + 1);
            } else if (more) {
                ok = warp_wait(s_read, i, limit);
                if (!ok) break;
                tc_fence_after_sync();
                ok = scores(i + 1) && grads(i + 1);
            }
            if (ok) ok = warp_wait(d_full, i, limit);
            if (!ok) break;
            tc_fence_after_sync();
            if (lane == 0) {
                mma_weights<DP>(KV ? acc2 : acc1, t_g(i), tile1(i), i > 0);
                mma_commit(&b1_empty[i % N1]);
                if (!more) mma_commit(sums_full);
            }
            __syncwarp();
            if (KV && more) ok = grads(i + 1);
        }
        // No product may be in flight when the tensor memory is freed.
        if (lane == 0) {
            mma_commit(drained);
            mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
        }
        __syncwarp();
    } else if (warp == kBwdLoadWarp) {
        // --------------------------------------------------------- loader
        int issued1 = 0, issued2 = 0;
        for (int i = 0; i < blocks; ++i) {
            const int s1 = i % N1, s2 = i % N2, sr = i % NR;
            const int hb = block_head(i), row = block_row(i);
            if (i >= N1 && !warp_wait(&b1_empty[s1], i / N1 - 1, limit)) break;
            if (lane == 0) {
                if (i == 0) {
                    mbar_arrive_expect_tx(a_full, 2 * L::kTile);
                    load_tile<128, DP>(smem + L::kA1, &map_a1, a0, ha, b, a_full);
                }
                mbar_arrive_expect_tx(&b1_full[s1], L::kTile);
                load_tile<128, DP>(smem + L::kB1 + s1 * L::kTile, &map_b1, row, hb, b,
                                   &b1_full[s1]);
                if (i == 0) load_tile<128, DP>(smem + L::kA2, &map_a2, a0, ha, b, a_full);
            }
            __syncwarp();
            issued1 = i + 1;
            if (KV && i >= NR && !warp_wait(&r_empty[sr], i / NR - 1, limit)) break;
            if (i >= N2 && !warp_wait(&b2_empty[s2], i / N2 - 1, limit)) break;
            if (lane == 0) {
                if (KV) {
                    const int64_t r = (static_cast<int64_t>(b) * t.heads + hb) * padded + row;
                    mbar_arrive_expect_tx(&r_full[sr], 2 * 128 * 4);
                    bulk_load(rows_s + 256 * sr, ws_lse + r, 128 * 4, &r_full[sr]);
                    bulk_load(rows_s + 256 * sr + 128, ws_delta + r, 128 * 4, &r_full[sr]);
                }
                mbar_arrive_expect_tx(&b2_full[s2], L::kTile);
                load_tile<128, DP>(smem + L::kB2 + s2 * L::kTile, &map_b2, row, hb, b,
                                   &b2_full[s2]);
            }
            __syncwarp();
            issued2 = i + 1;
        }
        // After an abort copies may still be in flight: none may land in
        // shared memory after the CTA exits (bounded waits).
        if (*limit.abort_flag && lane == 0 && issued1 > 0) {
            mbar_wait<false>(a_full, 0u, t.wait_limit_cycles);
            for (int i = max(0, issued1 - N1); i < issued1; ++i)
                mbar_wait<false>(&b1_full[i % N1], (i / N1) & 1, t.wait_limit_cycles);
            for (int i = max(0, issued2 - N2); i < issued2; ++i) {
                mbar_wait<false>(&b2_full[i % N2], (i / N2) & 1, t.wait_limit_cycles);
                if (KV) mbar_wait<false>(&r_full[i % NR], (i / NR) & 1, t.wait_limit_cycles);
            }
        }
        __syncwarp();
    } else if (!KV && warp == kBwdMaskWarp && mask) {
        // ------------------------------------------------------ key masks
        for (int i = 0; i < blocks; ++i) {
            const int st = i % N1;
            if (!warp_wait(&b1_full[st], i / N1, limit)) break;
            mask_tile<128, DP>(mask, t.key_len, block_row(i), smem + L::kB1 + st * L::kTile,
                               words + 4 * st, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&b1_masked[st]);
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
    constexpr int smem = BwdSmem<DP>::kBytes;
    static_assert(smem <= 232448, "the shared memory of a CTA");
    cudaError_t e = ensure_smem_attribute(kern, slot, smem, false);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mg, mk, mv;
    if (!encode_heads_map(&mq, t.q, t, t.heads, t.query_len, t.q_stride, 128) ||
        !encode_heads_map(&mg, t.go, t, t.heads, t.query_len, t.go_stride, 128) ||
        !encode_heads_map(&mk, t.k, t, t.kv_heads, t.key_len, t.k_stride, 128) ||
        !encode_heads_map(&mv, t.v, t, t.kv_heads, t.key_len, t.v_stride, 128))
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
