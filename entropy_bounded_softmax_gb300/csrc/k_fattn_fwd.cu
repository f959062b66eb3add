// Fused attention, forward.  For every query row i of a head:
//   s_j = scale q_i . k_j over the kept keys, m = max s_j,
//   l = sum e^(s_j - m), out_i = sum e^(s_j - m) v_j / l, lse_i = m + ln l,
// in one pass over the keys with the running m and l of a softmax: the
// scores never leave the SM.
//
// A CTA takes two tiles of 128 query rows of one head and walks the keys in
// blocks, so that one tile's products run under the other's softmax and both
// use the same K and V.  Tensor memory holds each tile's scores (a block's
// columns) and output (DP columns); a tile's weights overwrite its scores as
// bf16 and are the next product's A operand there.
//   d_head > 64   blocks of 128 keys, one CTA an SM.  A pair of blocks takes
//                 3000 cycles: the tensor pipe needs 2048 of them for its four
//                 products, shared memory 2050 for the 192 KB that they read
//                 and the 64 that the copies write; what the other 950 go to
//                 is not measured (2 x 8 heads x 4096 of 128, causal: 52 us,
//                 1.3 PFLOP/s, tensor pipe 58% busy);
//   d_head <= 64  blocks of 64 keys, two CTAs an SM, which four tiles keep
//                 busier (32 x 8 heads x 512: 24.2 us; two CTAs of one tile
//                 with two score buffers 28.5, three of one tile 28.4, one of
//                 two tiles and blocks of 128 35).
// Where the pairs of tiles are too few for the device (one prompt of few heads,
// few queries over long keys), a cluster of up to eight CTAs shares a pair's
// keys, and joins: each leaves its unnormalised outputs, maxima and sums in
// shared memory, and works out an equal share of the rows over the cluster, in
// the order of the ranks.  2 heads x 4096 of 128: 52 us without, 27 with; 4
// heads, one query over 4096 keys: 47 and 12.
// Roles, one mbarrier hand-off each:
//   warps 0-3, 4-7  softmax of tile 0 and 1, one row a thread: the maximum of
//                   the row's scores, 2^(s c - m c) and the sum, the weights
//                   back to tensor memory; at the end the output, through
//                   shared memory;
//   warp 8          issues the products: for each block and tile P V, then the
//                   next block's Q K^T into the columns P V has read (the
//                   products of one thread execute in its order);
//   warp 9          tensor copies of Q, and of K and V into rings;
//   warp 10         with a key mask only: a block's kept keys as bits, and
//                   zeros over the removed keys' rows of V.
//
// The weights are rounded to bf16, the type the tensor cores take next to
// bf16 values; their sum is taken in fp32 before that.  m may lag the true
// maximum by up to a factor 2^8 in the weights (exact in fp32 and bf16: they
// share an exponent range) so that the outputs are rescaled, in tensor
// memory, only when a row's maximum grew by more than that.
#include <math.h>
#include <string.h>

#include "cs_fattn.cuh"
#include "cs_tensormap.h"

namespace cs {
namespace {

using namespace csd;

constexpr float kRescaleBits = 8.0f;

constexpr int kFwdThreads = 384;
constexpr int kFwdMmaWarp = 8;
constexpr int kFwdLoadWarp = 9;
constexpr int kFwdMaskWarp = 10;

template <int DP>
struct FwdPlan {
    static constexpr int kBlk = DP == 64 ? 64 : 128;      // keys of a block
    static constexpr int kCtasPerSm = DP == 64 ? 2 : 1;
    static constexpr uint32_t kTmemCols = DP == 64 ? 256 : 512;
    // Registers a thread: 168 or, with two CTAs an SM, 80 at launch; the
    // softmax warps take what the others give up: 256 x 208 + 128 x 72 <=
    // 384 x 168, and 256 x 88 + 128 x 56 <= 384 x 80.
    static constexpr int kRegsSoftmax = DP == 64 ? 88 : 208;
    static constexpr int kRegsOther = DP == 64 ? 56 : 72;
    // Scores a softmax thread holds: the whole row, or 32 at a time, read from
    // tensor memory once for the maximum and once for the weights.
    static constexpr int kChunk = DP == 64 ? 32 : 128;
    // Shared memory.
    static constexpr int kTile = 128 * DP * 2;            // of Q
    static constexpr int kBlock = kBlk * DP * 2;          // of K or V
    static constexpr int kStages = 2;                     // of K and of V
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kStages * kBlock;
    static constexpr int kBars = kV + kStages * kBlock;
    static constexpr int kNumBars = 5 * kStages + 4 * 2 + 1 + 2;
    static constexpr int kWords = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [kStages][4]
    static constexpr int kFlags = kWords + kStages * 16;  // abort, tmem
    static constexpr int kBytes = kFlags + 16 + 1024;     // and alignment slack
    // Clusters: both tiles' maxima and sums, and, in fp32 from the start on,
    // their outputs.
    static constexpr int kStats = kFlags + 16;            // [256] float2
    static constexpr int kSums = 128 * DP * 4;
    static_assert(2 * kSums <= kBars, "both tiles' outputs fit");
    static constexpr int kSplitBytes = kBytes + 256 * 8;
    // The blocks of keys from which on a join, about 4 us, is worth it.  D 64,
    // whole and in clusters: 512 keys (16 heads x 512, causal) 12.7 and 13.6 us,
    // 768 (8 heads x 64) 13.7 and 11.9.  D 128: 768 keys 12.8 and 13.2, 1024 (8
    // heads x 256, causal) 17.4 and 16.0.
    static constexpr int kSplitBlocks = DP == 64 ? 12 : 8;
};

// -inf for the columns whose bit is not set.
template <int N>
__device__ __forceinline__ void remove_columns(uint32_t (&s)[N], const uint32_t* kept) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (!((kept[k >> 5] >> (k & 31)) & 1u)) s[k] = __float_as_uint(-INFINITY);
}

// SPLIT: launched in clusters that share a pair of tiles.
template <int DP, bool SPLIT>
__global__ void __launch_bounds__(kFwdThreads, FwdPlan<DP>::kCtasPerSm)
fattn_fwd_kernel(const FattnTask t, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
    using L = FwdPlan<DP>;
    constexpr int NS = L::kStages, BLK = L::kBlk, CH = L::kChunk;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* k_full = bars;                  // [NS] ring stage landed
    uint64_t* k_empty = k_full + NS;          // [NS] products that read it completed
    uint64_t* v_full = k_empty + NS;
    uint64_t* v_empty = v_full + NS;
    uint64_t* v_masked = v_empty + NS;        // [NS] removed rows zeroed, bits written
    uint64_t* q_full = v_masked + NS;         // [2] a tile's queries landed
    uint64_t* s_full = q_full + 2;            // [2] its scores of a block
    uint64_t* o_full = s_full + 2;            // [2] the block's P V completed
    uint64_t* o_done = o_full + 2;            // [2] its last P V completed
    uint64_t* drained = o_done + 2;
    uint64_t* p_full = drained + 1;           // [2] its weights, from four warps
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kWords);
    volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags);
    const WaitLimit limit{flags, t.wait_limit_cycles};

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // Under the causal mask later rows keep more keys: longest first.
    const int bits = SPLIT ? t.split_bits : 0;
    const int h = blockIdx.x >> bits, rank = blockIdx.x & ((1 << bits) - 1), b = blockIdx.y;
    const int qt = t.causal ? static_cast<int>(gridDim.z - 1 - blockIdx.z)
                            : static_cast<int>(blockIdx.z);
    const int hk = head_of(h, t.inv_group);
    const int q0 = 256 * qt;
    const int off = t.key_len - t.query_len;   // row i keeps keys j <= i + off

    auto load_q = [&](int i) {
        if (q0 + 128 * i >= t.query_len) return;
        mbar_arrive_expect_tx(&q_full[i], L::kTile);
        load_tile<128, DP>(smem + L::kQ + i * L::kTile, &map_q, q0 + 128 * i, h, b, &q_full[i]);
    };

    // The loader initialises the barriers, and starts its first copies before
    // the others have set up.
    if (warp == kFwdLoadWarp) {
        if (lane < L::kNumBars) mbar_init(bars + lane, bars + lane < p_full ? 1u : 4u);
        if (lane == 0) flags[0] = 0u;
        static_assert(L::kNumBars <= 32, "a lane a barrier");
        fence_mbar_init();
        __syncwarp();
        if (lane == 0) {
            if (t.key_len > 0) {   // (an empty tensor has no map)
                prefetch_tmap(&map_k);
                prefetch_tmap(&map_v);
            }
            load_q(0);
        }
        __syncwarp();
    } else if (warp == kFwdMmaWarp) {
        tmem_alloc(const_cast<uint32_t*>(flags) + 1, L::kTmemCols);
    }
    const uint8_t* mask = t.mask ? t.mask + b * t.mask_stride : nullptr;
    int key_lo = 0, key_hi = t.key_len;
    if (mask) warp_nonzero_range(mask, t.key_len, lane, key_lo, key_hi);

    // Blocks first, first + 1, ..: n[i] of them for tile i, none for a tile without
    // rows or without kept keys.
    const int first = key_lo / BLK;
    int n[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int last = min(q0 + 128 * (i + 1), t.query_len) - 1;
        const int hi = t.causal ? min(key_hi, last + off + 1) : key_hi;
        n[i] = last >= q0 + 128 * i && hi > key_lo ? (hi + BLK - 1) / BLK - first : 0;
    }
    // A cluster's CTAs take equal shares of them, and join their outputs.
    const int all = max(n[0], n[1]);
    const bool joint = SPLIT && all > 0;
    const int from = SPLIT ? static_cast<int>(static_cast<int64_t>(all) * rank >> bits) : 0;
    if (SPLIT) {
        const int to = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) >> bits);
#pragma unroll
        for (int i = 0; i < 2; ++i) n[i] = max(0, min(n[i], to) - from);
    }
    const int j0 = first + from;
    const int blocks = max(n[0], n[1]);
    auto load_k = [&](int j) {
        const int st = j % NS;
        mbar_arrive_expect_tx(&k_full[st], L::kBlock);
        load_tile<BLK, DP>(smem + L::kK + st * L::kBlock, &map_k, (j0 + j) * BLK, hk, b,
                           &k_full[st]);
    };
    auto load_v = [&](int j) {
        const int st = j % NS;
        mbar_arrive_expect_tx(&v_full[st], L::kBlock);
        load_tile<BLK, DP>(smem + L::kV + st * L::kBlock, &map_v, (j0 + j) * BLK, hk, b,
                           &v_full[st]);
    };
    const int early = min(blocks, NS);
    if (warp == kFwdLoadWarp && lane == 0) {
        // In the order of their use.
        for (int j = 0; j < early; ++j) {
            load_k(j);
            if (j == 0) load_q(1);
            load_v(j);
        }
        if (early == 0) load_q(1);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = flags[1];

    if (warp < 8) {
        // -------------------------------------------------------- softmax
        take_registers<L::kRegsSoftmax>();
        const int tile = warp >> 2;
        const int row0 = q0 + 128 * tile + 32 * (warp & 3);
        const int i = row0 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + BLK * tile;
        const uint32_t to = tmem + lanes + 2 * BLK + DP * tile;
        const float c = t.scale * kLog2e;
        // Keys below these limits are kept in every row of the warp, and in
        // this thread's.
        const int warp_limit = t.causal ? min(t.key_len, row0 + off + 1) : t.key_len;
        const int row_limit = t.causal ? min(t.key_len, i + off + 1) : t.key_len;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        const int nt = n[tile];
        for (int j = 0; j < nt; ++j) {
            ok = warp_wait(&s_full[tile], j, limit);
            if (ok && mask) ok = warp_wait(&v_masked[j % NS], j / NS, limit);
            if (!ok) break;
            tc_fence_after_sync();
            const int key = (j0 + j) * BLK;
            bool edge = warp_limit < key + BLK;
            uint32_t kept[BLK / 32];
#pragma unroll
            for (int u = 0; u < BLK / 32; ++u) {
                kept[u] = mask ? words[4 * (j % NS) + u] : ~0u;
                edge = edge || kept[u] != ~0u;
            }
            if (edge) {
#pragma unroll
                for (int u = 0; u < BLK / 32; ++u) kept[u] &= bits_below(row_limit, key + 32 * u);
            }
            uint32_t s[CH];
            auto load = [&](int x) {
#pragma unroll
                for (int u = 0; u < CH / 32; ++u) tmem_ld32_async(ts + CH * x + 32 * u, s + 32 * u);
                tmem_wait_ld<CH>(s);
                if (edge) remove_columns(s, kept + CH / 32 * x);
            };
            float mx[4] = {m, m, m, m};
#pragma unroll
            for (int x = 0; x < BLK / CH; ++x) {
                load(x);
#pragma unroll
                for (int k = 0; k < CH; k += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        mx[y] = max3(mx[y], __uint_as_float(s[k + 2 * y]),
                                     __uint_as_float(s[k + 2 * y + 1]));
            }
            const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
            if (j == 0) {
                m = top;
            } else if (__any_sync(0xffffffffu, (top - m) * c > kRescaleBits)) {
                const float f = m == -INFINITY ? 0.0f : ex2((m - top) * c);
                m = top;
                l *= f;
                ok = warp_wait(&o_full[tile], j - 1, limit);
                if (!ok) break;
                tc_fence_after_sync();
#pragma unroll 1
                for (int u = 0; u < DP / 32; ++u) {
                    uint32_t o[32];
                    tmem_ld32_async(to + 32 * u, o);
                    tmem_wait_ld<32>(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st32(to + 32 * u, o);
                }
            }
            const float mc = m == -INFINITY ? 0.0f : m * c;
            const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int x = 0; x < BLK / CH; ++x) {
                if (CH < BLK) load(x);
#pragma unroll
                for (int k = 0; k < CH / 2; ++k) {
                    const float2 y = fma2(make_float2(__uint_as_float(s[2 * k]),
                                                      __uint_as_float(s[2 * k + 1])), c2, mc2);
                    const float2 e = make_float2(ex2(y.x), ex2(y.y));
                    sum[k & 1] = add2(sum[k & 1], e);
                    s[k] = pack_bf16(e.x, e.y);
                }
                // (Over columns that this thread has read for good.)
                if (CH == 32) tmem_st16(ts + 16 * x, s);
#pragma unroll
                for (int u = 0; u < CH / 64; ++u) tmem_st32(ts + CH / 2 * x + 32 * u, s + 32 * u);
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[tile]);
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
        }
        // The tile's queries are read (or, without blocks, have landed) before
        // the output is staged over them.
        if (joint) {
            // In fp32, over the queries, keys and values, once both tiles' are
            // read (or have landed): rows of DP floats, their 16-byte units
            // permuted by the row.
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (ok && n[x] > 0) ok = warp_wait(&o_done[x], 0, limit);
                if (ok && n[x] == 0 && q0 + 128 * x < t.query_len)
                    ok = warp_wait(&q_full[x], 0, limit);
            }
            float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
            const int r = 32 * (warp & 3) + lane;
            if (ok) {
                tc_fence_after_sync();
                stats[128 * tile + r] = make_float2(m == -INFINITY ? 0.0f : m * c, l);
                unsigned char* row = smem + tile * L::kSums + r * DP * 4;
#pragma unroll 1
                for (int u = 0; u < DP / 32; ++u) {
                    uint32_t o[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                    if (nt > 0) {
                        tmem_ld32_async(to + 32 * u, o);
                        tmem_wait_ld<32>(o);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(row + (((8 * u + k) ^ (r & 7)) << 4)) =
                            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            // Each CTA joins its share of the rows, rank after rank: the
            // largest maximum M, the sums and outputs times 2^(m - M).
            constexpr int kUnits = DP / 8;
            const int rows = 256 >> bits;
            for (int e = threadIdx.x; e < rows * kUnits; e += 256) {
                const int u = e % kUnits, at = rank * rows + e / kUnits, qi = q0 + at;
                if (qi >= t.query_len || 8 * u >= t.d_head) continue;
                const uint32_t stat = smem_addr(smem + L::kStats) + at * 8;
                float top = -INFINITY, sum = 0.0f;
                for (int k = 0; k < 1 << bits; ++k) {
                    const float2 s = cluster_load2(map_to_rank(stat, k));
                    if (s.y != 0.0f) top = fmaxf(top, s.x);
                }
                const uint32_t line = smem_addr(smem) + (at >> 7) * L::kSums + (at & 127) * DP * 4;
                float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                for (int k = 0; k < 1 << bits; ++k) {
                    const float2 s = cluster_load2(map_to_rank(stat, k));
                    if (s.y == 0.0f) continue;   // no keys there
                    const float f = ex2(s.x - top);
                    sum = fmaf(s.y, f, sum);
                    const uint32_t there = map_to_rank(line, k);
                    const float4 v0 = cluster_load(there + ((2 * u ^ (at & 7)) << 4));
                    const float4 v1 = cluster_load(there + (((2 * u + 1) ^ (at & 7)) << 4));
                    const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                    for (int y = 0; y < 8; ++y) acc[y] = fmaf(v[y], f, acc[y]);
                }
                const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
                *reinterpret_cast<uint4*>(t.out + b * t.o_stride[0] + h * t.o_stride[1] +
                                          qi * t.o_stride[2] + 8 * u) =
                    make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv),
                               pack_bf16(acc[2] * inv, acc[3] * inv),
                               pack_bf16(acc[4] * inv, acc[5] * inv),
                               pack_bf16(acc[6] * inv, acc[7] * inv));
                if (u == 0) {
                    if (t.lse)
                        t.lse[(static_cast<int64_t>(b) * t.heads + h) * t.query_len + qi] =
                            sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
                    if (!isfinite(sum)) raise_error(t.err, kBitNan);
                }
            }
            // No CTA ends while another reads its shared memory.
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            ok = false;   // nothing is left to write
        }
        if (ok && nt > 0) ok = warp_wait(&o_done[tile], 0, limit);
        if (ok && nt == 0 && row0 < t.query_len) ok = warp_wait(&q_full[tile], 0, limit);
        if (ok && row0 < t.query_len) {
            tc_fence_after_sync();
            const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
            const bool some_empty = __any_sync(0xffffffffu, l == 0.0f);
            unsigned char* stage = smem + L::kQ + tile * L::kTile;
            const int r = 32 * (warp & 3);
            const int64_t row = (static_cast<int64_t>(b) * t.heads + h) * t.query_len + i;
#pragma unroll 1
            for (int u = 0; u < DP / 32; ++u) {
                uint32_t o[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
                if (nt > 0) {
                    tmem_ld32_async(to + 32 * u, o);
                    tmem_wait_ld<32>(o);
                }
                // Exactly 0 without kept keys, whatever a value that only
                // `causal` removes holds (0 times its NaN is NaN).
                if (some_empty) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = l == 0.0f ? 0u : o[k];
                }
                stage_row32(stage, r + lane, 32 * u, o, inv);
            }
            store_rows32<DP / 64>(
                stage, r, 0,
                t.out + b * t.o_stride[0] + h * t.o_stride[1] + row0 * t.o_stride[2],
                t.o_stride[2], t.query_len - row0, t.d_head, lane);
            if (i < t.query_len) {
                if (t.lse)
                    t.lse[row] =
                        l == 0.0f ? -INFINITY : (m * c + log2f(l)) * kLn2;
                if (!isfinite(l)) raise_error(t.err, kBitNan);
            }
        }
    } else {
        give_registers<L::kRegsOther>();
        if (warp == kFwdMmaWarp) {
            // ------------------------------------------------- MMA issuer
            const bool leader = elect_lane();
            const uint32_t q = tile_desc(smem_addr(smem + L::kQ));
            const uint32_t k = tile_desc(smem_addr(smem + L::kK));
            const uint32_t v = weights_desc<BLK>(smem_addr(smem + L::kV));
            constexpr uint32_t tile = L::kTile / 16, step = L::kBlock / 16;
            const int steps = (t.d_head + 15) / 16;
            const uint32_t idesc = idesc_bf16(128, 16 * steps, true);
            auto scores = [&](int i, int j) {
                mma_tiles<BLK, DP>(tmem + BLK * i, q + i * tile, k + (j % NS) * step, steps, leader);
                mma_commit(&s_full[i], leader);
            };
            bool ok = true;
            if (blocks > 0) {
                ok = warp_wait(&k_full[0], 0, limit);
                for (int i = 0; i < 2 && ok; ++i) {
                    if (n[i] == 0) continue;
                    ok = warp_wait(&q_full[i], 0, limit);
                    if (ok) scores(i, 0);
                }
                if (ok) mma_commit(&k_empty[0], leader);
            }
            uint64_t* v_ready = mask ? v_masked : v_full;
            for (int j = 0; j < blocks && ok; ++j) {
                const int st = j % NS, next = (j + 1) % NS;
                ok = warp_wait(&v_ready[st], j / NS, limit);
                for (int i = 0; i < 2 && ok; ++i) {
                    if (j >= n[i]) continue;
                    ok = warp_wait(&p_full[i], j, limit);
                    if (!ok) break;
                    tc_fence_after_sync();
                    mma_weights<BLK>(tmem + 2 * BLK + DP * i, tmem + BLK * i, v + st * step,
                                     idesc, j > 0, leader);
                    mma_commit(&o_full[i], leader);
                    if (j + 1 == n[i]) {
                        mma_commit(&o_done[i], leader);
                    } else {
                        ok = warp_wait(&k_full[next], (j + 1) / NS, limit);
                        if (ok) scores(i, j + 1);
                    }
                }
                if (ok) {
                    mma_commit(&v_empty[st], leader);
                    if (j + 1 < blocks) mma_commit(&k_empty[next], leader);
                }
            }
            // No product may be in flight when the tensor memory is freed.
            mma_commit(drained, leader);
            mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
            __syncwarp();
        } else if (warp == kFwdLoadWarp) {
            // ----------------------------------------------------- loader
            int k_issued = early, v_issued = early;
            for (int j = early; j < blocks; ++j) {
                if (!warp_wait(&k_empty[j % NS], j / NS - 1, limit)) break;
                if (lane == 0) load_k(j);
                k_issued = j + 1;
                if (!warp_wait(&v_empty[j % NS], j / NS - 1, limit)) break;
                if (lane == 0) load_v(j);
                v_issued = j + 1;
            }
            // A copy may still be in flight after an abort, or that of a tile
            // without blocks: none may land in shared memory after the CTA
            // exits (bounded waits).
            for (int i = 0; i < 2; ++i)
                if (q0 + 128 * i < t.query_len) mbar_wait<false>(&q_full[i], 0u, t.wait_limit_cycles);
            if (*limit.abort_flag) {
                for (int j = max(0, k_issued - NS); j < k_issued; ++j)
                    mbar_wait<false>(&k_full[j % NS], (j / NS) & 1, t.wait_limit_cycles);
                for (int j = max(0, v_issued - NS); j < v_issued; ++j)
                    mbar_wait<false>(&v_full[j % NS], (j / NS) & 1, t.wait_limit_cycles);
            }
            __syncwarp();
        } else if (warp == kFwdMaskWarp && mask) {
            // -------------------------------------------------- key masks
            for (int j = 0; j < blocks; ++j) {
                const int st = j % NS;
                if (!warp_wait(&v_full[st], j / NS, limit)) break;
                mask_tile<BLK, DP>(mask, t.key_len, (j0 + j) * BLK, smem + L::kV + st * L::kBlock,
                                   words + 4 * st, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_masked[st]);
            }
        }
        if (joint) {   // the softmax warps' two
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kFwdMmaWarp) tmem_dealloc(tmem, L::kTmemCols);
    if (threadIdx.x == 0 && flags[0]) raise_error(t.err, kBitTimeout);
}

// slots: two, for the kernel without and with clusters.
template <int DP>
cudaError_t launch_fwd(FattnTask t, int slot, int split_slot, cudaStream_t stream) {
    using L = FwdPlan<DP>;
    const int row_tiles = (t.query_len + 255) / 256;
    const int64_t blocks = (t.key_len + L::kBlk - 1) / L::kBlk;
    t.split_bits = blocks < L::kSplitBlocks
                       ? 0
                       : split_bits(static_cast<int64_t>(t.heads) * t.batch * row_tiles, blocks,
                                    256 / L::kBlk, t.sm_count * L::kCtasPerSm);
    const bool split = t.split_bits > 0;
    const auto kernel = split ? fattn_fwd_kernel<DP, true> : fattn_fwd_kernel<DP, false>;
    const int bytes = split ? L::kSplitBytes : L::kBytes;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel),
                                          split ? split_slot : slot, bytes, false);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv;
    if (!encode_heads_map(&mq, t.q, t, t.heads, t.query_len, t.q_stride, 128) ||
        !encode_heads_map(&mk, t.k, t, t.kv_heads, t.key_len, t.k_stride, L::kBlk) ||
        !encode_heads_map(&mv, t.v, t, t.kv_heads, t.key_len, t.v_stride, L::kBlk))
        return cudaErrorInvalidValue;
    const dim3 grid(t.heads << t.split_bits, t.batch, row_tiles);
    return launch_shaped(kernel,
                         {grid, kFwdThreads, bytes, stream, false, 1 << t.split_bits}, t, mq,
                         mk, mv);
}

}  // namespace

cudaError_t launch_fattn_forward(const FattnTask& task, cudaStream_t stream) {
    return task.d_head <= 64 ? launch_fwd<64>(task, 56, 72, stream)
                             : launch_fwd<128>(task, 57, 73, stream);
}

}  // namespace cs
