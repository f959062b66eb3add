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
//   queries (KV = false)  128 query rows a CTA, over blocks of keys:
//       S = Q K^T, G V^T, dq += dS K.  Before its blocks it takes delta of
//       its rows and leaves -delta and -lse, in base 2 and padded to whole
//       tiles, in the workspace for the second launch;
//   keys (KV = true)      128 key rows a CTA, over blocks of queries of
//       every head of its group: S^T = K Q^T, V G^T, dv += P^T G,
//       dk += dS^T Q.  It starts while the first still runs, and waits for it
//       where it needs the workspace: its start, and what is left of the
//       device's SMs at the first's end, cost nothing.
// Where the tiles of a launch are too few for the device (few key heads, short
// sequences against long ones), a tile's blocks are shared by a cluster of up
// to eight CTAs, which leave their sums in shared memory in fp32; each adds an
// equal share of the rows over the cluster, in the order of the ranks, so that
// these sums have a fixed order too.  8 query heads on one key head x 4096 of
// 128, causal: 351 us without, 126 with; 8 on 2 x 512 of 64: 39 and 26.
//
// In both the fixed tiles' rows are the lanes of tensor memory, and the
// weights, rounded to bf16 in columns their scores had, are the next
// product's A operand there.  Blocks are 128 rows for d_head > 64: a product
// of 64 columns reads its A tile from shared memory twice as often and is
// bound by that.  For d_head <= 64 they are 64 rows, so that two CTAs fit an
// SM and the start and the end of one run under the other's work.
//
// Tensor memory holds two sums, S and G V^T (keys), or one sum, S and two of
// G V^T (queries).  The elementwise part has two phases, P from S and dS from
// P and G V^T, and the products are issued so that each phase runs under
// products that do not wait for it:
//   keys     dv(i), S(i+1), dk(i), G V^T(i+1): P(i+1) under dk(i) and
//            G V^T(i+1), dS(i) under dv(i) and S(i+1);
//   queries  S(i+1), G V^T(i+1), dq(i): P(i) and dS(i) under the first two.
// Roles:
//   warps 0-7   the elementwise part, a row and half its columns a thread
//               (warps w and w + 4 share the rows of lanes 32 (w % 4) ..);
//   warp 8      issues the products;
//   warp 9      tensor copies: the two fixed tiles, then the blocks;
//   warp 10     queries with a key mask only: a block's kept keys as bits,
//               and zeros over the removed keys' rows of K.
//
// Measured, both launches: 2 x 8 heads x 4096 of 128, causal, 163 us (1.05
// PFLOP/s of the five products, 1.47 of the seven; the tensor pipe 60 and 69%
// busy, and what the rest goes to, as in the forward, not measured); 32 x 8
// heads x 512 of 64, 76 us (bound by the chain of each block's two elementwise
// phases and by the starts and ends of the CTAs: the tensor pipe 22 and 28%
// busy).
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
constexpr uint32_t kBarElementwise = 1;
constexpr uint32_t kElementwise = 256;         // threads

// The first streamed tensor (K, or Q) is read by a block's first and last
// product, the second (V, or G) by the ones between: three stages and two.
template <int DP>
struct BwdPlan {
    static constexpr int kBlk = DP == 64 ? 64 : 128;      // rows of a block
    static constexpr int kCtasPerSm = DP == 64 ? 2 : 1;
    static constexpr uint32_t kTmemCols = DP == 64 ? 256 : 512;
    static constexpr int kCols = kBlk / 2;                // columns of a thread
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int kBlock = kBlk * DP * 2;
    static constexpr int kStages1 = 3, kStages2 = 2, kStagesR = 2;
    static constexpr int kA1 = 0;              // Q, or K
    static constexpr int kA2 = kA1 + kTile;    // G, or V
    static constexpr int kB1 = kA2 + kTile;
    static constexpr int kB2 = kB1 + kStages1 * kBlock;
    // Queries: the tile of out, before the first blocks: where shared memory
    // is full, over the last stage of the first ring.
    static constexpr int kOut = DP == 64 ? kB2 + kStages2 * kBlock
                                         : kB1 + (kStages1 - 1) * kBlock;
    static constexpr int kRows = kB2 + kStages2 * kBlock + (DP == 64 ? kTile : 0);  // [kStagesR][2][128] lse, delta
    static constexpr int kBars = kRows + kStagesR * 2 * 128 * 4;
    static constexpr int kNumBars =
        3 + 3 * kStages1 + 2 * kStages2 + 2 * kStagesR + 8 + 2;
    static constexpr int kWords = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [kStages1][4]
    static constexpr int kFlags = kWords + kStages1 * 16;
    static constexpr int kBytes = kFlags + 16;
    // A cluster's sums, in fp32 from the start of shared memory on.
    static constexpr int kSums = 128 * DP * 4;
    static_assert(2 * kSums <= kB2 + kStages2 * kBlock, "dk and dv fit");
    static_assert(kSums <= kB1, "dq fits the fixed tiles");
};

__device__ __forceinline__ float2 pair(const uint32_t* x, int k) {
    return make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
}

// Zeros for the columns whose bit is not set.
template <int N>
__device__ __forceinline__ void clear_removed(uint32_t (&x)[N], const uint32_t (&kept)[N / 32]) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (!((kept[k >> 5] >> (k & 31)) & 1u)) x[k] = 0u;
}

__device__ __forceinline__ void store_weights(uint32_t at, const uint32_t (&w)[32]) {
    tmem_st32(at, w);
}
__device__ __forceinline__ void store_weights(uint32_t at, const uint32_t (&w)[16]) {
    tmem_st16(at, w);
}

// SPLIT: launched in clusters that share a tile (an instance of its own, so
// that its code does not cost the others registers: 2% of 32 x 8 x 512).
template <int DP, bool KV, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads, BwdPlan<DP>::kCtasPerSm)
fattn_bwd_kernel(const FattnTask t, const __grid_constant__ CUtensorMap map_a1,
                 const __grid_constant__ CUtensorMap map_a2,
                 const __grid_constant__ CUtensorMap map_b1,
                 const __grid_constant__ CUtensorMap map_b2,
                 const __grid_constant__ CUtensorMap map_o) {
    using L = BwdPlan<DP>;
    constexpr int N1 = L::kStages1, N2 = L::kStages2, NR = L::kStagesR;
    constexpr int BLK = L::kBlk, CO = L::kCols;
    // The tiles need 1024-byte alignment, and fill the shared memory that a
    // CTA can have up to a few hundred bytes; there are no static variables.
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* a_full = bars;                   // [2] a fixed tile landed
    uint64_t* o_full = a_full + 2;             // queries: the tile of out landed
    uint64_t* b1_full = o_full + 1;            // [N1] ring stage landed
    uint64_t* b1_empty = b1_full + N1;         // [N1] products that read it completed
    uint64_t* b1_masked = b1_empty + N1;       // [N1] removed rows zeroed, bits written
    uint64_t* b2_full = b1_masked + N1;        // [N2]
    uint64_t* b2_empty = b2_full + N2;
    uint64_t* r_full = b2_empty + N2;          // [NR] keys: lse and delta landed
    uint64_t* s_full = r_full + NR;            // a block's scores
    uint64_t* g_full = s_full + 1;             // [2] its G V^T, by buffer
    uint64_t* sums_full = g_full + 2;          // every sum completed
    uint64_t* drained = sums_full + 1;
    uint64_t* r_empty = drained + 1;           // [NR] from eight warps, as those below
    uint64_t* o_read = r_empty + NR;           // queries: the tile of out is read
    uint64_t* s_read = o_read + 1;             // queries: the scores are in registers
    uint64_t* p_full = s_read + 1;             // keys: the block's P
    uint64_t* d_full = p_full + 1;             // [2] its dS, by buffer
    float* rows_s = reinterpret_cast<float*>(smem + L::kRows);
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kWords);
    volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags);
    const WaitLimit limit{flags, t.wait_limit_cycles};
    if (!KV) allow_next_kernel();

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int fixed_len = KV ? t.key_len : t.query_len;
    // Under the causal mask late queries keep the most keys and early keys
    // have the most queries: longest first in both.
    // The fixed tiles' head, and this CTA's place among those of its cluster,
    // which share the tile's blocks.
    const int bits = SPLIT ? t.split_bits : 0;
    const int ha = blockIdx.x >> bits, rank = blockIdx.x & ((1 << bits) - 1), b = blockIdx.y;
    const int a0 = 128 * static_cast<int>(!KV && t.causal ? gridDim.z - 1 - blockIdx.z
                                                          : blockIdx.z);
    const int off = t.key_len - t.query_len;   // query i keeps keys j <= i + off
    const int group = KV ? t.heads / t.kv_heads : 1;
    const int hk = KV ? ha : head_of(ha, t.inv_group);
    const int64_t padded = (static_cast<int64_t>(t.query_len) + 127) / 128 * 128;
    float* ws_lse = t.rows;
    float* ws_delta = t.rows + static_cast<int64_t>(t.batch) * t.heads * padded;

    // Keys: the queries with a kept key in the tile, i >= a0 - off under causal.
    const int lo = KV && t.causal ? max(0, a0 - off) : 0;
    const int last = min(a0 + 128, fixed_len) - 1;
    // Blocks first .. first + per - 1 of the streamed side, for each head.
    int first = lo / BLK, per = 0;
    if (KV && lo < t.query_len) per = (t.query_len + BLK - 1) / BLK - first;
    // Of the tile's n blocks, head after head, this CTA takes from the first of
    // its share on.
    auto share = [&](int n, int r) {
        return static_cast<int>(static_cast<int64_t>(n) * r >> bits);
    };
    // A block's head on the streamed side and its first row there, walked in
    // order (each walker keeps its own: a division by `per` for every block
    // would cost more than its elementwise part's shorter phase).
    struct Place {
        int head, row;
    };
    int from = share(per * group, rank), blocks = share(per * group, rank + 1) - from;
    Place begin{KV ? ha * group : hk, BLK * (first + from)};
    if (KV && from > 0) {
        begin.head += from / per;
        begin.row = BLK * (first + from % per);
    }
    auto advance = [&](Place& x) {
        x.row += BLK;
        if (KV && x.row >= BLK * (first + per)) {
            x.row = BLK * first;
            ++x.head;
        }
    };
    auto load1 = [&](int i, Place& at) {
        uint64_t* bar = &b1_full[i % N1];
        mbar_arrive_expect_tx(bar, L::kBlock);
        load_tile<BLK, DP>(smem + L::kB1 + (i % N1) * L::kBlock, &map_b1, at.row, at.head, b,
                           bar);
        advance(at);
    };
    // Keys: lse and delta of a block's queries.
    auto load_rows = [&](int i, Place& at) {
        const int64_t r = (static_cast<int64_t>(b) * t.heads + at.head) * padded + at.row;
        uint64_t* bar = &r_full[i % NR];
        float* rows = rows_s + 2 * BLK * (i % NR);
        mbar_arrive_expect_tx(bar, 2 * BLK * 4);
        bulk_load(rows, ws_lse + r, BLK * 4, bar);
        bulk_load(rows + BLK, ws_delta + r, BLK * 4, bar);
        advance(at);
    };
    auto load2 = [&](int i, Place& at) {
        uint64_t* bar = &b2_full[i % N2];
        mbar_arrive_expect_tx(bar, L::kBlock);
        load_tile<BLK, DP>(smem + L::kB2 + (i % N2) * L::kBlock, &map_b2, at.row, at.head, b,
                           bar);
        advance(at);
    };
    Place at1 = begin, at2 = begin, at_r = begin;   // the loader's
    static_assert(N2 == NR, "the row values' ring is as deep as the second tensor's");

    // The loader initialises the barriers, and starts the copies that the mask
    // does not decide on before the others have set up and the mask is read
    // (1700 cycles), in the order of their use: the first S, the first G V^T.
    const bool any = KV && blocks > 0;   // if the tile's keys are kept
    if (warp == kBwdLoadWarp) {
        static_assert(L::kNumBars <= 32, "a lane a barrier");
        if (lane < L::kNumBars) mbar_init(bars + lane, bars + lane < r_empty ? 1u : 8u);
        if (lane == 0) flags[0] = 0u;
        fence_mbar_init();
        __syncwarp();
        if (lane == 0) {
            if (t.query_len > 0 && t.key_len > 0) {   // (an empty tensor has no map)
                prefetch_tmap(&map_b1);
                prefetch_tmap(&map_b2);
            }
            mbar_arrive_expect_tx(&a_full[0], L::kTile);
            load_tile<128, DP, BLK>(smem + L::kA1, &map_a1, a0, ha, b, &a_full[0]);
            if (any) load1(0, at1);
            mbar_arrive_expect_tx(&a_full[1], L::kTile);
            load_tile<128, DP, BLK>(smem + L::kA2, &map_a2, a0, ha, b, &a_full[1]);
            if (any) load2(0, at2);
            if (!KV) {
                mbar_arrive_expect_tx(o_full, L::kTile);
                load_tile<128, DP, BLK>(smem + L::kOut, &map_o, a0, ha, b, o_full);
            }
        }
        __syncwarp();
    } else if (warp == kBwdMmaWarp) {
        tmem_alloc(const_cast<uint32_t*>(flags) + 1, L::kTmemCols);
    }
    const uint8_t* mask = t.mask ? t.mask + b * t.mask_stride : nullptr;
    // An elementwise thread's row of the fixed tile, and what it needs from
    // memory for it, loaded before the set-up's waits: lse, or whether the key
    // is removed.
    const int a = a0 + 32 * (warp & 3) + lane;
    const int64_t row_of_head = static_cast<int64_t>(b) * t.heads + ha;
    float lse = -INFINITY;
    bool removed = false;
    if (warp < 8 && a < fixed_len) {
        if (!KV) lse = t.lse[row_of_head * t.query_len + a];
        if (KV && mask) removed = mask[a] == 0;
    }
    int key_lo = 0, key_hi = t.key_len;
    if (mask) warp_nonzero_range(mask, t.key_len, lane, key_lo, key_hi);

    if (KV) {
        if (a0 >= key_hi || last < key_lo) per = 0;
    } else {
        const int hi = t.causal ? min(key_hi, last + off + 1) : key_hi;
        first = key_lo / BLK;
        if (hi > key_lo) per = (hi + BLK - 1) / BLK - first;
        from = share(per, rank);
        begin.row = BLK * (first + from);
        at1 = at2 = begin;
    }
    blocks = per > 0 ? share(per * group, rank + 1) - from : 0;
    const bool joint = SPLIT && per > 0;   // the cluster's sums are added
    if (!KV && warp == kBwdLoadWarp && lane == 0 && blocks > 0) {
        load1(0, at1);
        load2(0, at2);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = flags[1];
    const uint32_t acc1 = tmem;                // dq, or dv
    const uint32_t acc2 = tmem + DP;           // keys: dk
    const uint32_t t_s = tmem + (KV ? 2 : 1) * DP;
    // G V^T of block i, and the dS over it: keys: one buffer; queries: two with
    // barriers of their own, because there a block's G V^T may complete, and a
    // fast warp's dS be written, before every warp is done with the block
    // before.
    auto g_buf = [&](int i) { return KV ? 0 : i & 1; };
    auto g_phase = [&](int i) { return KV ? i : i >> 1; };
    auto t_g = [&](int i) { return t_s + BLK * (KV ? 1 : 1 + (i & 1)); };

    if (warp < 8) {
        // ----------------------------------------------------- elementwise
        const int half = warp >> 2;
        const int quarter = warp & 3;
        const uint32_t at = (static_cast<uint32_t>(quarter * 32) << 16) + CO * half;
        const float c = t.scale * kLog2e;
        const float2 c2 = make_float2(c, c);
        float row_lse = 0.0f, row_delta = 0.0f;   // queries: -lse, -delta
        bool ok = true;
        if (!KV) {
            // delta: DP / 8 lanes a row, 16 bytes of out and of g each, 16 rows
            // a warp, from the tiles that the tensor copies brought.  (Loads of
            // out's rows took 2 to 10 thousand cycles, a third of a short
            // sequence's CTA.)  A wait that gives up leaves delta wrong and the
            // barrier below matched; the next wait gives up too.
            constexpr int LR = DP / 8, kSteps = 16 * LR / 32;
            warp_wait(&a_full[1], 0, limit);
            warp_wait(o_full, 0, limit);
            const int u = lane % LR, r0 = 16 * warp + lane / LR;
            float d[kSteps];
#pragma unroll
            for (int n = 0; n < kSteps; ++n) {
                const int r = r0 + n * (32 / LR);
                const int at = (u >> 3) * (128 * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
                const uint4 x = *reinterpret_cast<const uint4*>(smem + L::kOut + at);
                const uint4 y = *reinterpret_cast<const uint4*>(smem + L::kA2 + at);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                const uint32_t ys[4] = {y.x, y.y, y.z, y.w};
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sum = fma2(make_float2(InBF16::lo(xs[k]), InBF16::hi(xs[k])),
                               make_float2(InBF16::lo(ys[k]), InBF16::hi(ys[k])), sum);
                d[n] = sum.x + sum.y;
            }
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1)
#pragma unroll
                for (int n = 0; n < kSteps; ++n) d[n] += __shfl_xor_sync(0xffffffffu, d[n], o);
#pragma unroll
            for (int n = 0; n < kSteps; ++n)
                if (u == 0) rows_s[r0 + n * (32 / LR)] = d[n];
            __syncwarp();
            if (lane == 0) mbar_arrive(o_read);
            // An empty row, and a row past the last, gets -lse = -inf: P = 0.
            row_lse = lse == -INFINITY ? lse : -lse * kLog2e;
            named_barrier(kBarElementwise, kElementwise);
            row_delta = -rows_s[a - a0];
            if (half == 0 && rank == 0) {
                ws_lse[row_of_head * padded + a] = row_lse;
                ws_delta[row_of_head * padded + a] = row_delta;
            }
        }
        Place place = begin;
        for (int i = 0; i < blocks; ++i) {
            const int st = i % NR;
            const int b0 = place.row + CO * half;        // first of this thread's columns
            advance(place);
            // -lse and -delta of this thread's columns (keys).
            const float4* lse4 = reinterpret_cast<const float4*>(rows_s + 2 * BLK * st + CO * half);
            const float4* delta4 = lse4 + BLK / 4;
            if (KV) ok = warp_wait(&r_full[st], i / NR, limit);
            if (!KV && mask) ok = warp_wait(&b1_masked[i % N1], i / N1, limit);
            if (ok) ok = warp_wait(s_full, i, limit);
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t s[CO];
#pragma unroll
            for (int u = 0; u < CO / 32; ++u) tmem_ld32_async(t_s + at + 32 * u, s + 32 * u);
            tmem_wait_ld<CO>(s);
            if (!KV) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
            }
            // P from S: 2^(s c - lse), packed pairs.
            uint32_t kept[CO / 32];
#pragma unroll
            for (int u = 0; u < CO / 32; ++u) kept[u] = ~0u;
            bool edge;
            if (KV) {
                // Columns are queries.  Rows of removed keys are not treated
                // here: their sums are replaced by zeros at the end.
                // Causal: query b0 + k keeps this key from k = a - off - b0 on.
                edge = t.causal && a0 + 32 * quarter + 31 - off > b0;
                if (edge) {
#pragma unroll
                    for (int u = 0; u < CO / 32; ++u) kept[u] = ~bits_below(a - off, b0 + 32 * u);
                }
            } else {
                // Columns are keys.
                const int limit_warp =
                    t.causal ? min(t.key_len, a0 + 32 * quarter + off + 1) : t.key_len;
                edge = limit_warp < b0 + CO;
                if (mask) {
#pragma unroll
                    for (int u = 0; u < CO / 32; ++u) {
                        kept[u] = words[4 * (i % N1) + CO / 32 * half + u];
                        edge = edge || kept[u] != ~0u;
                    }
                }
                if (edge) {
                    const int limit_row = t.causal ? min(t.key_len, a + off + 1) : t.key_len;
#pragma unroll
                    for (int u = 0; u < CO / 32; ++u) kept[u] &= bits_below(limit_row, b0 + 32 * u);
                }
            }
#pragma unroll
            for (int k4 = 0; k4 < CO / 4; ++k4) {
                float4 le = make_float4(row_lse, row_lse, row_lse, row_lse);
                if (KV) le = lse4[k4];
                const float2 y0 = fma2(pair(s, 4 * k4), c2, make_float2(le.x, le.y));
                const float2 y1 = fma2(pair(s, 4 * k4 + 2), c2, make_float2(le.z, le.w));
                s[4 * k4] = __float_as_uint(ex2(y0.x));
                s[4 * k4 + 1] = __float_as_uint(ex2(y0.y));
                s[4 * k4 + 2] = __float_as_uint(ex2(y1.x));
                s[4 * k4 + 3] = __float_as_uint(ex2(y1.y));
            }
            if (edge) clear_removed(s, kept);
            if (KV) {
                uint32_t w[CO / 2];
#pragma unroll
                for (int k = 0; k < CO / 2; ++k) {
                    const float2 p = pair(s, 2 * k);
                    w[k] = pack_bf16(p.x, p.y);
                }
                store_weights(t_s + at, w);
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            ok = warp_wait(&g_full[g_buf(i)], g_phase(i), limit);
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t g[CO];
#pragma unroll
            for (int u = 0; u < CO / 32; ++u) tmem_ld32_async(t_g(i) + at + 32 * u, g + 32 * u);
            tmem_wait_ld<CO>(g);
            // dS = P (G V^T - delta), packed pairs; exactly 0 for removed
            // pairs, whatever G V^T holds there (padding's NaN).
#pragma unroll
            for (int k4 = 0; k4 < CO / 4; ++k4) {
                float4 de = make_float4(row_delta, row_delta, row_delta, row_delta);
                if (KV) de = delta4[k4];
                const float2 d0 = mul2(pair(s, 4 * k4),
                                       add2(pair(g, 4 * k4), make_float2(de.x, de.y)));
                const float2 d1 = mul2(pair(s, 4 * k4 + 2),
                                       add2(pair(g, 4 * k4 + 2), make_float2(de.z, de.w)));
                g[4 * k4] = __float_as_uint(d0.x);
                g[4 * k4 + 1] = __float_as_uint(d0.y);
                g[4 * k4 + 2] = __float_as_uint(d1.x);
                g[4 * k4 + 3] = __float_as_uint(d1.y);
            }
            if (edge) clear_removed(g, kept);
            uint32_t w[CO / 2];
#pragma unroll
            for (int k = 0; k < CO / 2; ++k) {
                const float2 d = pair(g, 2 * k);
                w[k] = pack_bf16(d.x, d.y);
            }
            store_weights(t_g(i) + at, w);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&d_full[g_buf(i)]);
                if (KV) mbar_arrive(&r_empty[st]);
            }
        }
        // The rows' sums, staged over the fixed tiles once those are read: keys:
        // dv by the first four warps, dk by the others; queries: a panel of 64
        // columns of dq each.
        if (ok && blocks > 0) ok = warp_wait(sums_full, 0, limit);
        const int row0 = a0 + 32 * quarter;
        constexpr int kPanels = DP / 64;
        const int p0 = KV || kPanels == 1 ? 0 : half, p1 = KV ? kPanels : p0 + 1;
        if (joint) {
            // In fp32, over the fixed tiles and the first ring, once all has
            // landed and is read: rows of DP floats, their 16-byte units
            // permuted by the row.
            if (ok && blocks == 0)
                ok = warp_wait(&a_full[0], 0, limit) && warp_wait(&a_full[1], 0, limit);
            if (ok && (KV || kPanels == 2 || half == 0)) {
                tc_fence_after_sync();
                const uint32_t sums = (KV && half == 1 ? acc2 : acc1) +
                                      (static_cast<uint32_t>(quarter * 32) << 16);
                const int r = 32 * quarter + lane;
                unsigned char* to = smem + (KV && half == 1 ? L::kSums : 0) + r * DP * 4;
#pragma unroll 1
                for (int c0 = 64 * p0; c0 < 64 * p1; c0 += 32) {
                    uint32_t x[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = 0u;
                    if (blocks > 0) {
                        tmem_ld32_async(sums + c0, x);
                        tmem_wait_ld<32>(x);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(to + (((c0 / 4 + k) ^ (r & 7)) << 4)) =
                            make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                }
            }
        } else if (ok && row0 < fixed_len && (KV || kPanels == 2 || half == 0)) {
            unsigned char* stage = smem + (KV && half == 1 ? L::kA2 : L::kA1);
            uint16_t* to = KV ? (half == 1 ? t.dk : t.dv) : t.dq;
            const int64_t* stride = KV ? (half == 1 ? t.dk_stride : t.dv_stride) : t.dq_stride;
            to += b * stride[0] + ha * stride[1] + row0 * stride[2];
            if (blocks > 0) {
                tc_fence_after_sync();
                const uint32_t sums = (KV && half == 1 ? acc2 : acc1) +
                                      (static_cast<uint32_t>(quarter * 32) << 16);
                const float f = KV && half == 0 ? 1.0f : t.scale;
                // Exactly 0 for removed keys and for queries without keys,
                // whatever the rows that they were multiplied with hold.
                const bool zero = KV ? removed : row_lse == -INFINITY;
#pragma unroll 1
                for (int c0 = 64 * p0; c0 < 64 * p1; c0 += 32) {
                    uint32_t x[32];
                    tmem_ld32_async(sums + c0, x);
                    tmem_wait_ld<32>(x);
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] = zero ? 0u : x[k];
                    stage_row32(stage, 32 * quarter + lane, c0, x, f);
                }
                store_rows32<KV ? kPanels : 1>(stage, 32 * quarter, p0, to, stride[2],
                                               fixed_len - row0, t.d_head, lane);
            } else {
                zero_rows32<KV ? kPanels : 1>(p0, to, stride[2], fixed_len - row0, t.d_head, lane);
            }
        }
    } else if (warp == kBwdMmaWarp) {
        // ----------------------------------------------------- MMA issuer
        const bool leader = elect_lane();
        constexpr uint32_t step = L::kBlock / 16;
        const int steps = (t.d_head + 15) / 16;
        const uint32_t idesc = idesc_bf16(128, 16 * steps, true);
        const uint32_t b1 = smem_addr(smem + L::kB1), b2 = smem_addr(smem + L::kB2);
        const uint32_t a1_t = tile_desc(smem_addr(smem + L::kA1));
        const uint32_t a2_t = tile_desc(smem_addr(smem + L::kA2));
        const uint32_t b1_t = tile_desc(b1), b1_w = weights_desc<BLK>(b1);
        const uint32_t b2_t = tile_desc(b2), b2_w = weights_desc<BLK>(b2);
        uint64_t* ready1 = !KV && mask ? b1_masked : b1_full;
        // S of block i, G V^T of block i, once their tiles are there.
        auto scores = [&](int i) {
            if (!warp_wait(&ready1[i % N1], i / N1, limit)) return false;
            mma_tiles<BLK, DP>(t_s, a1_t, b1_t + (i % N1) * step, steps, leader);
            mma_commit(s_full, leader);
            return true;
        };
        auto grads = [&](int i) {
            if (!warp_wait(&b2_full[i % N2], i / N2, limit)) return false;
            mma_tiles<BLK, DP>(t_g(i), a2_t, b2_t + (i % N2) * step, steps, leader);
            mma_commit(&g_full[g_buf(i)], leader);
            if (!KV) mma_commit(&b2_empty[i % N2], leader);
            return true;
        };
        // A sum's product; each half's weights are where its scores were.
        auto sums = [&](uint32_t d, uint32_t w, uint32_t b, bool accumulate) {
            mma_weights<CO>(d, w, b, idesc, accumulate, leader);
            mma_weights<CO>(d, w + CO, b + CO / 16 * kDescRows16, idesc, true, leader);
        };
        bool ok = blocks == 0 ||
                  (warp_wait(&a_full[0], 0, limit) && scores(0) &&
                   warp_wait(&a_full[1], 0, limit) && grads(0));
        for (int i = 0; i < blocks && ok; ++i) {
            const bool more = i + 1 < blocks;
            if (KV) {
                ok = warp_wait(p_full, i, limit);
                if (!ok) break;
                tc_fence_after_sync();
                sums(acc1, t_s, b2_w + (i % N2) * step, i > 0);
                mma_commit(&b2_empty[i % N2], leader);
                if (more) ok = scores(i + 1);
            } else if (more) {
                ok = warp_wait(s_read, i, limit);
                if (!ok) break;
                tc_fence_after_sync();
                ok = scores(i + 1) && grads(i + 1);
            }
            if (ok) ok = warp_wait(&d_full[g_buf(i)], g_phase(i), limit);
            if (!ok) break;
            tc_fence_after_sync();
            sums(KV ? acc2 : acc1, t_g(i), b1_w + (i % N1) * step, i > 0);
            mma_commit(&b1_empty[i % N1], leader);
            if (!more) mma_commit(sums_full, leader);
            if (KV && more) ok = grads(i + 1);
        }
        // No product may be in flight when the tensor memory is freed.
        mma_commit(drained, leader);
        mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
        __syncwarp();
    } else if (warp == kBwdLoadWarp) {
        // --------------------------------------------------------- loader
        if (KV && lane == 0) {
            wait_for_previous_kernel();   // it writes the workspace
            if (blocks > 0) load_rows(0, at_r);
        }
        __syncwarp();
        // The rest once the first blocks are there: while CTAs start together
        // L2 is what bounds them (288 KB each took 9000 cycles to come).
        int issued1 = min(blocks, 1), issued2 = issued1;
        if (blocks > 1) warp_wait(&b2_full[0], 0, limit);
        for (int i = 1; i < blocks; ++i) {
            if (i >= N1 && !warp_wait(&b1_empty[i % N1], i / N1 - 1, limit)) break;
            // The first copy over the tile of out.
            if (!KV && DP == 128 && i == N1 - 1 && !warp_wait(o_read, 0, limit)) break;
            if (lane == 0) load1(i, at1);
            issued1 = i + 1;
            if (i >= N2) {
                if (KV && !warp_wait(&r_empty[i % NR], i / NR - 1, limit)) break;
                if (!warp_wait(&b2_empty[i % N2], i / N2 - 1, limit)) break;
            }
            if (lane == 0) {
                if (KV) load_rows(i, at_r);
                load2(i, at2);
            }
            issued2 = i + 1;
        }
        // A copy may still be in flight after an abort, or the fixed tiles'
        // without blocks: none may land in shared memory after the CTA exits
        // (bounded waits).
        for (int i = 0; i < 2; ++i) mbar_wait<false>(&a_full[i], 0u, t.wait_limit_cycles);
        if (any && blocks == 0) {
            mbar_wait<false>(&b1_full[0], 0u, t.wait_limit_cycles);
            mbar_wait<false>(&b2_full[0], 0u, t.wait_limit_cycles);
        }
        if (!KV) mbar_wait<false>(o_full, 0u, t.wait_limit_cycles);
        if (*limit.abort_flag) {
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
            mask_tile<BLK, DP>(mask, t.key_len, begin.row + BLK * i, smem + L::kB1 + st * L::kBlock,
                               words + 4 * st, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&b1_masked[st]);
        }
    }
    if (joint) {
        // Each CTA adds its share of the rows over the cluster, in the order
        // of the ranks.
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        constexpr int kUnits = DP / 8;
        const int rows = 128 >> bits;
        for (int e = threadIdx.x; e < (KV ? 2 : 1) * rows * kUnits; e += kBwdThreads) {
            const int u = e % kUnits, x = e / kUnits / rows;
            const int r = rank * rows + (e / kUnits & (rows - 1)), i = a0 + r;
            if (i >= fixed_len || 8 * u >= t.d_head) continue;
            const bool zero = KV ? mask && mask[i] == 0
                                 : t.lse[row_of_head * t.query_len + i] == -INFINITY;
            const uint32_t at = smem_addr(smem) + x * L::kSums + r * DP * 4;
            float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
#pragma unroll 2
            for (int k = 0; k < 1 << bits; ++k) {
                const uint32_t there = map_to_rank(at, k);
                const float4 v0 = cluster_load(there + ((2 * u ^ (r & 7)) << 4));
                const float4 v1 = cluster_load(there + (((2 * u + 1) ^ (r & 7)) << 4));
                s0 = make_float4(s0.x + v0.x, s0.y + v0.y, s0.z + v0.z, s0.w + v0.w);
                s1 = make_float4(s1.x + v1.x, s1.y + v1.y, s1.z + v1.z, s1.w + v1.w);
            }
            const float f = KV && x == 0 ? 1.0f : t.scale;
            uint4 w = make_uint4(pack_bf16(s0.x * f, s0.y * f), pack_bf16(s0.z * f, s0.w * f),
                                 pack_bf16(s1.x * f, s1.y * f), pack_bf16(s1.z * f, s1.w * f));
            if (zero) w = make_uint4(0u, 0u, 0u, 0u);
            uint16_t* to = KV ? (x == 1 ? t.dk : t.dv) : t.dq;
            const int64_t* stride = KV ? (x == 1 ? t.dk_stride : t.dv_stride) : t.dq_stride;
            *reinterpret_cast<uint4*>(to + b * stride[0] + ha * stride[1] + i * stride[2] +
                                      8 * u) = w;
        }
        // No CTA ends while another reads its shared memory.
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kBwdMmaWarp) tmem_dealloc(tmem, L::kTmemCols);
    if (threadIdx.x == 0 && flags[0]) raise_error(t.err, kBitTimeout);
}

// One of the two launches: its tiles of `heads` heads of `length` rows, walked
// over up to `blocks` blocks; slots: two, for the kernel without and with
// clusters.
template <int DP, bool KV>
cudaError_t launch_one(FattnTask t, int heads, int length, int64_t blocks, bool overlapped,
                       int slot, cudaStream_t stream, const CUtensorMap& a1,
                       const CUtensorMap& a2, const CUtensorMap& b1, const CUtensorMap& b2,
                       const CUtensorMap& out) {
    using L = BwdPlan<DP>;
    static_assert(L::kBytes <= 232448, "the shared memory of a CTA");
    const int row_tiles = (length + 127) / 128;
    t.split_bits = split_bits(static_cast<int64_t>(heads) * t.batch * row_tiles, blocks, 4,
                              t.sm_count * L::kCtasPerSm);
    const auto kernel = t.split_bits > 0 ? fattn_bwd_kernel<DP, KV, true>
                                         : fattn_bwd_kernel<DP, KV, false>;
    const cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel),
                                                slot + (t.split_bits > 0), L::kBytes, false);
    if (e != cudaSuccess) return e;
    const dim3 grid(heads << t.split_bits, t.batch, row_tiles);
    return launch_shaped(
        kernel, {grid, kBwdThreads, L::kBytes, stream, overlapped, 1 << t.split_bits}, t, a1, a2,
        b1, b2, out);
}

template <int DP>
cudaError_t launch_both(const FattnTask& t, int slot, cudaStream_t stream) {
    using L = BwdPlan<DP>;
    // Boxes of a block's rows; fixed tiles of 128 rows are two of them where
    // blocks are 64.
    CUtensorMap q, g, k, v, out;
    constexpr int kBox = L::kBlk;
    if (!encode_heads_map(&q, t.q, t, t.heads, t.query_len, t.q_stride, kBox) ||
        !encode_heads_map(&g, t.go, t, t.heads, t.query_len, t.go_stride, kBox) ||
        !encode_heads_map(&k, t.k, t, t.kv_heads, t.key_len, t.k_stride, kBox) ||
        !encode_heads_map(&v, t.v, t, t.kv_heads, t.key_len, t.v_stride, kBox) ||
        !encode_heads_map(&out, t.out, t, t.heads, t.query_len, t.o_stride, kBox))
        return cudaErrorInvalidValue;
    const int64_t key_blocks = (t.key_len + kBox - 1) / kBox;
    const int64_t query_blocks = (t.query_len + kBox - 1) / kBox * (t.heads / t.kv_heads);
    cudaError_t e = cudaSuccess;
    if (t.query_len > 0)
        e = launch_one<DP, false>(t, t.heads, t.query_len, key_blocks, false, slot, stream, q, g,
                                  k, v, out);
    // The second overlaps the first only: without that one (no queries) it may
    // not start before the stream's own work, which may use the gradients'
    // memory, has ended.
    if (e == cudaSuccess && t.key_len > 0)
        e = launch_one<DP, true>(t, t.kv_heads, t.key_len, query_blocks, t.query_len > 0, slot + 2,
                                 stream, k, v, q, g, out);
    return e;
}

}  // namespace

cudaError_t launch_fattn_backward(const FattnTask& task, cudaStream_t stream) {
    return task.d_head <= 64 ? launch_both<64>(task, 58, stream)
                             : launch_both<128>(task, 68, stream);
}

}  // namespace cs
