// Attention of several new tokens per sequence over a paged key-value cache:
// a tree of drafted tokens, or a prompt's next chunk.  Sequence b has n =
// lengths[b] tokens in its pages, the last w of them new.  New token i attends
// the n - w before all new ones and those new ones, j, that mask[i][j] (or
// j <= i) keeps.  For its head h and key head hk:
//   s_j = scale q . k_j,  out = sum e^(s_j - m) v_j / sum e^(s_j - m).
//
// The rows of a key head, (new token, query head) with the heads side by side,
// make tiles of 128; a unit is one tile or, where there are more, a pair.  Its
// keys and values are walked once, in blocks, by one CTA:
//   one tile   even blocks belong to the first softmax warpgroup, odd blocks to
//              the second, each with scores, weights and an output of its own
//              in tensor memory, so that one's products run under the other's
//              softmax; the two are joined at the end (d_head > 128, whose
//              outputs fill tensor memory: one warpgroup, all blocks);
//   a pair     each warpgroup has a tile and all blocks.
// The blocks of the batch's units are dealt in equal shares to one wave of CTA
// groups, as paged_attention deals its steps: `width` CTAs of a group walk the
// same pages for as many key heads at the same time.  A unit that lies in one
// share is finished there; parts of the others (maximum, sum, unnormalised
// output) go to the workspace, and a second small kernel joins them.
//
// Roles, one mbarrier hand-off each:
//   warps 0-3, 4-7  softmax, one row a thread;
//   warp 8          issues the products (tcgen05, operands in shared memory,
//                   weights in tensor memory);
//   warps 12-15     look pages up and keep the rings of K and V full by
//                   asynchronous copies of 16 bytes, whatever a page's size and
//                   its strides are; queries too.
//
// The weights are rounded to the cache's type, the one the tensor cores take
// beside its values; their sum is taken in fp32 before that.  They carry a
// factor 2^8, and their maximum may lag by 2^6: fp16 has no exponents below
// 2^-24, and the largest weight, 2^8 to 2^14, leaves 2^-32 of it.
#include <cuda_fp16.h>
#include <math.h>

#include "cs_fattn.cuh"

namespace cs {
namespace {

using namespace csd;

constexpr int kTrThreads = 512;
constexpr int kTrMmaWarp = 8;
constexpr int kTrCopyWarp = 12;
constexpr float kTrWeightBits = 8.0f;  // log2 of the weights' common factor
constexpr float kTrLagBits = 6.0f;     // how far the maximum may lag
constexpr int kTrWords = 8;            // blocks whose kept tokens are noted

struct TrBF16 {
    static constexpr bool kFp16 = false;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        return pack_bf16(lo, hi);
    }
};
struct TrFP16 {
    static constexpr bool kFp16 = true;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// DP: d_head rounded up to 64, 128 or 256; NQ: tiles of a unit.
template <int DP, int NQ>
struct TreePlan {
    static constexpr int kBlk = tree_block(DP);            // tokens of a block
    static constexpr int kTiles = DP == 256 ? 1 : 2;       // accumulators
    static constexpr int kTile = 128 * DP * 2;             // of Q
    static constexpr int kBlock = kBlk * DP * 2;           // of K or V
    static constexpr int kStages = DP == 64 ? 6 - (NQ - 1) : DP == 128 ? 4 - NQ : 2;
    // Registers a thread: 128 at launch; the softmax warps take what the others
    // give up: 256 x 192 + 256 x 64 = 512 x 128.
    static constexpr int kRegsSoftmax = 192;
    static constexpr int kRegsOther = 64;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kOut = kTiles * kBlk;             // first column of the outputs
    static_assert(kOut + kTiles * DP <= 512, "tensor memory");
    // Shared memory.
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + NQ * kTile;
    static constexpr int kV = kK + kStages * kBlock;
    static constexpr int kBars = kV + kStages * kBlock;
    static constexpr int kNumBars = 4 * kStages + 11;
    static constexpr int kWords = kBars + (8 * kNumBars + 15) / 16 * 16;  // [kTrWords][4]
    static constexpr int kScan = kWords + kTrWords * 16;   // [18] ints
    static constexpr int kFlags = kScan + 80;              // abort, tmem
    static constexpr int kStats = kFlags + 16;             // [2][128] float2 (one tile)
    static constexpr int kBytes = kStats + (NQ == 1 ? 2 * 128 * 8 : 0);
    static_assert(kBytes <= 232448, "shared memory of a CTA");
    static_assert(kStages + 2 <= kTrWords, "a block's words outlive its keys' stage");
};

// A sequence's tokens, and how many of them are new.
struct TreeLens {
    int len, fresh;
};
__device__ __forceinline__ TreeLens tree_lens(const TreeTask& t, int b, bool& bad) {
    const int n = t.lengths[b];
    const int most = t.max_pages * t.page_size;
    const int w = t.new_lengths ? t.new_lengths[b] : t.new_tokens;
    TreeLens x;
    x.len = n < 0 ? 0 : min(n, most);
    x.fresh = min(max(w, 0), min(t.new_tokens, x.len));
    bad = n < 0 || n > most || w != x.fresh;
    return x;
}

// Blocks of a unit of sequence b.
template <int BLK>
__device__ __forceinline__ int tree_steps(const TreeLens& x) {
    return x.fresh > 0 ? (x.len + BLK - 1) / BLK : 0;
}

// The sum of n over the threads before this one and over all of the CTA of
// 32 WARPS threads; scan: WARPS shared ints, free again after the caller's next
// __syncthreads.
template <int WARPS>
__device__ __forceinline__ void tree_scan(int n, int* scan, int& before, int& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int up = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
    }
    if (lane == 31) scan[warp] = up;
    __syncthreads();
    before = up - n;
    all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
    }
}

// What a group of CTAs has of the list of the batch's blocks: for each sequence,
// for each of its bundles of `width` rows (units side by side), the blocks.
// Blocks g0 .. g1 - 1, the first in sequence b whose first is `base`.
struct TreeDeal {
    int g0, g1, b, base, share;
};

// By a whole CTA; false without blocks.  scan: WARPS + 2 shared ints.
template <int WARPS, int BLK>
__device__ __forceinline__ bool tree_deal(const TreeTask& t, int grp, int* scan, TreeDeal& d) {
    constexpr int kThreads = 32 * WARPS;
    bool bad;
    auto blocks = [&](int i) {
        return i < t.batch ? tree_steps<BLK>(tree_lens(t, i, bad)) * t.bundles : 0;
    };
    int total = 0, before;
    const bool once = t.batch <= kThreads;   // one walk over the lengths is enough
    if (!once) {
        int n = 0;
        for (int i = threadIdx.x; i < t.batch; i += kThreads) n += blocks(i);
        tree_scan<WARPS>(n, scan, before, total);
        __syncthreads();
    }
    int done = 0;
    for (int b0 = 0; b0 < t.batch; b0 += kThreads) {
        const int i = b0 + threadIdx.x;
        const int n = blocks(i);
        int first, all;
        tree_scan<WARPS>(n, scan, first, all);
        if (once) total = all;
        d.share = max(1, (total + t.groups - 1) / t.groups);
        d.g0 = grp * d.share;
        d.g1 = min(total, d.g0 + d.share);
        if (d.g0 >= d.g1) return false;
        first += done;
        if (first <= d.g0 && d.g0 < first + n) {
            scan[WARPS] = i;
            scan[WARPS + 1] = first;
        }
        done += all;
        __syncthreads();
        if (done > d.g0) break;
    }
    // (In range even where the lengths were changed under the call.)
    d.b = max(0, min(scan[WARPS], t.batch - 1));
    d.base = min(scan[WARPS + 1], d.g0);
    return true;
}

// Blocks s0 .. s1 - 1 of a unit of sequence b: all of them, or part `place` of
// the workspace.
struct TreePart {
    int b, row, s0, s1;
    TreeLens n;
    bool whole;
    int place;
};

// A CTA's parts, one after the other; every role walks its own copy.
template <int BLK>
struct TreeWalk {
    int g, g0, g1, b, bundle, s, steps, x;
    TreeLens n;
    bool any;
    __device__ __forceinline__ bool next(const TreeTask& t, TreePart& p) {
        if (!any || g >= g1) return false;
        bool bad;
        while (steps == 0 || bundle == t.bundles) {
            if (b + 1 >= t.batch) return false;
            n = tree_lens(t, ++b, bad);
            steps = tree_steps<BLK>(n);
            bundle = 0;
        }
        p.b = b;
        p.row = bundle * t.width + x;
        p.s0 = s;
        p.s1 = min(steps, s + g1 - g);
        p.n = n;
        p.whole = p.s0 == 0 && p.s1 == steps;
        p.place = 2 * static_cast<int>(blockIdx.x) + (g > g0);
        g += p.s1 - p.s0;
        s = p.s1;
        if (s == steps) {
            s = 0;
            ++bundle;
        }
        return true;
    }
};

// The rows of a unit: first row, rows there and rows whose token is new (rows
// are token by token, `group` heads each).
struct TreeRows {
    int hk, r0, rows, valid;
};
template <int NQ>
__device__ __forceinline__ TreeRows tree_rows(const TreeTask& t, int row, const TreeLens& n) {
    TreeRows u;
    const int tile = row / t.kv_heads;
    u.hk = row - tile * t.kv_heads;
    u.r0 = 128 * NQ * tile;
    u.rows = min(128 * NQ, t.new_tokens * t.group - u.r0);
    u.valid = min(128 * NQ, n.fresh * t.group - u.r0);   // may be negative
    return u;
}

// Blocks s0 .. s1 - 1 that some row of the unit attends: none without rows, and
// none past the last row's token where each attends those before it.
template <int BLK>
__device__ __forceinline__ int tree_blocks(const TreeTask& t, const TreePart& p,
                                           const TreeRows& u) {
    if (u.valid <= 0) return 0;
    int last = p.s1;
    if (!t.mask) {
        const int token = (u.r0 + u.valid - 1) / t.group;
        last = min(last, (p.n.len - p.n.fresh + token + BLK) / BLK);
    }
    return max(0, last - p.s0);
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];"
                 :: "r"(smem_addr(bar)) : "memory");
}

// Elements d .. d + 7 of one row of the output, from unnormalised sums.
template <class E>
__device__ __forceinline__ void tree_store8(uint16_t* row, int d, const float (&acc)[8],
                                            float inv) {
    *reinterpret_cast<uint4*>(row + d) =
        make_uint4(E::pack(acc[0] * inv, acc[1] * inv), E::pack(acc[2] * inv, acc[3] * inv),
                   E::pack(acc[4] * inv, acc[5] * inv), E::pack(acc[6] * inv, acc[7] * inv));
}

__device__ __forceinline__ uint16_t* tree_out(const TreeTask& t, int b, int i, int h) {
    return t.out + b * t.o_stride[0] + i * t.o_stride[1] + h * t.o_stride[2];
}

// A row's lse, and whether its sum is finite, from the maximum in base 2.
__device__ __forceinline__ void tree_lse(const TreeTask& t, int b, int i, int h, float top,
                                         float sum) {
    if (t.lse)
        t.lse[(static_cast<int64_t>(b) * t.new_tokens + i) * t.heads + h] =
            sum == 0.0f ? -INFINITY : (top + log2f(sum) - kTrWeightBits) * kLn2;
    if (!isfinite(sum)) raise_error(t.err, kBitNan);
}

template <int DP, int NQ, class E>
__global__ void __launch_bounds__(kTrThreads, 1) tree_kernel(const TreeTask t) {
    using L = TreePlan<DP, NQ>;
    constexpr int NS = L::kStages, BLK = L::kBlk, NT = L::kTiles;
    // (No room is left to align it here: the swizzled tiles want 1024 bytes.)
    extern __shared__ __align__(1024) unsigned char smem[];
    if (smem_addr(smem) & 1023u) {
        if (threadIdx.x == 0) raise_error(t.err, kBitTimeout);
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* k_full = bars;                  // [NS] copies landed
    uint64_t* k_empty = k_full + NS;          // [NS] products that read it completed
    uint64_t* v_full = k_empty + NS;
    uint64_t* v_empty = v_full + NS;
    uint64_t* s_full = v_empty + NS;          // [2] scores of a block
    uint64_t* o_full = s_full + 2;            // [2] its P V completed
    uint64_t* p_full = o_full + 2;            // [2] its weights, from four warps
    uint64_t* q_full = p_full + 2;
    uint64_t* q_empty = q_full + 1;           // the part's last scores completed
    uint64_t* o_done = q_empty + 1;           // the part's last P V completed
    uint64_t* drained = o_done + 1;
    uint64_t* joined = drained + 1;           // eight softmax warps
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kWords);
    volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags);
    const WaitLimit limit{flags, t.wait_limit_cycles};
    allow_next_kernel();

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (warp == kTrCopyWarp) {
        for (int i = lane; i < L::kNumBars; i += 32) {
            uint64_t* bar = bars + i;
            mbar_init(bar, bar < k_empty ? 128u + 4u
                           : (bar >= v_full && bar < v_empty) || bar == q_full ? 128u
                           : bar >= p_full && bar < q_full ? 4u
                           : bar == joined ? 8u : 1u);
        }
        if (lane == 0) flags[0] = 0u;
        fence_mbar_init();
    } else if (warp == kTrMmaWarp) {
        tmem_alloc(const_cast<uint32_t*>(flags) + 1, L::kTmemCols);
    }
    TreeWalk<BLK> walk{};
    {
        const int grp = static_cast<int>(blockIdx.x) / t.width;
        walk.x = static_cast<int>(blockIdx.x) - grp * t.width;
        bool bad;
        if (t.split) {
            TreeDeal d;
            walk.any = tree_deal<kTrThreads / 32, BLK>(
                t, grp, reinterpret_cast<int*>(smem + L::kScan), d);
            if (walk.any) {
                walk.g = walk.g0 = d.g0;
                walk.g1 = d.g1;
                walk.b = d.b;
                walk.n = tree_lens(t, d.b, bad);
                walk.steps = tree_steps<BLK>(walk.n);
                if (walk.steps > 0) {
                    walk.bundle = min((d.g0 - d.base) / walk.steps, t.bundles);
                    walk.s = (d.g0 - d.base) % walk.steps;
                }
            }
        } else {
            // Each group one bundle of one sequence, blocks or not.
            walk.b = grp / t.bundles;
            walk.bundle = grp - walk.b * t.bundles;
            walk.n = tree_lens(t, walk.b, bad);
            walk.steps = max(1, tree_steps<BLK>(walk.n));
            walk.g1 = walk.steps;
            walk.any = true;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = flags[1];
    const int group = t.group;

    if (warp < 8) {
        // -------------------------------------------------------- softmax
        take_registers<L::kRegsSoftmax>();
        const int wg = warp >> 2;              // warpgroup
        const int tile = NT == 2 ? wg : 0;
        const int tr = 32 * (warp & 3) + lane; // row of the tile
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + BLK * tile;
        const uint32_t out0 = tmem + lanes + L::kOut;
        const uint32_t to = out0 + DP * tile;
        const float c = t.scale * kLog2e;
        float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
        int visit = 0;      // blocks of this warpgroup so far, over all parts
        int parts = 0;      // parts with blocks
        int block0 = 0;     // blocks of the parts before
        int joins = 0;
        bool ok = true;
        TreePart p;
        while (ok && walk.next(t, p)) {
            const TreeRows u = tree_rows<NQ>(t, p.row, p.n);
            const int n = tree_blocks<BLK>(t, p, u);
            // This warpgroup's blocks: all of them, or every other one.
            const int first = NQ == 1 && NT == 2 ? wg : 0, step = NQ == 1 && NT == 2 ? 2 : 1;
            const int mine = NT == 1 && wg > 0 ? 0 : n > first ? (n - first + step - 1) / step : 0;
            const int r = (NQ == 2 ? 128 * wg : 0) + tr;      // row of the unit
            const int warp_r = (NQ == 2 ? 128 * wg : 0) + 32 * (warp & 3);
            const int token = (u.r0 + r) / group;             // new token
            const bool valid = r < u.valid;
            const bool warp_valid = warp_r < u.valid;
            const int context = p.n.len - p.n.fresh;
            // Rows keep the tokens below this, and of them those the mask keeps.
            const int row_limit = !valid ? 0 : t.mask ? p.n.len : context + token + 1;
            float m = -INFINITY, l = 0.0f;
            for (int k = 0; k < mine; ++k, ++visit) {
                const int block = first + step * k;
                const int key = (p.s0 + block) * BLK;
                uint32_t kept[BLK / 32];
#pragma unroll
                for (int w = 0; w < BLK / 32; ++w) kept[w] = bits_below(row_limit, key + 32 * w);
                if (t.mask && warp_valid && key + BLK > context) {
                    // The mask's rows of this warp's tokens, 32 bytes at a time.
                    const uint8_t* rows = t.mask + p.b * t.mask_stride[0];
                    const int i0 = (u.r0 + warp_r) / group;
                    const int i1 = min((u.r0 + warp_r + 31) / group, p.n.fresh - 1);
#pragma unroll 2
                    for (int i = i0; i <= i1; ++i) {
#pragma unroll
                        for (int w = 0; w < BLK / 32; ++w) {
                            const int j = key + 32 * w + lane - context;
                            bool keep = j < 0;
                            if (j >= 0 && j < p.n.fresh)
                                keep = rows[i * t.mask_stride[1] + j] != 0;
                            const uint32_t bits = __ballot_sync(0xffffffffu, keep);
                            if (i == token) kept[w] &= bits;
                        }
                    }
                }
                ok = warp_wait(&s_full[tile], visit, limit);
                if (!ok) break;
                tc_fence_after_sync();
                if (warp_valid) {
                    bool edge = false;
#pragma unroll
                    for (int w = 0; w < BLK / 32; ++w) {
                        kept[w] &= words[4 * ((block0 + block) % kTrWords) + w];
                        edge = edge || kept[w] != ~0u;
                    }
                    edge = __any_sync(0xffffffffu, edge);
                    uint32_t s[BLK];
#pragma unroll
                    for (int x = 0; x < BLK / 32; ++x) tmem_ld32_async(ts + 32 * x, s + 32 * x);
                    tmem_wait_ld<BLK>(s);
                    if (edge) {
#pragma unroll
                        for (int x = 0; x < BLK; ++x)
                            if (!((kept[x >> 5] >> (x & 31)) & 1u))
                                s[x] = __float_as_uint(-INFINITY);
                    }
                    float mx[4] = {m, m, m, m};
#pragma unroll
                    for (int x = 0; x < BLK; x += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            mx[y] = max3(mx[y], __uint_as_float(s[x + 2 * y]),
                                         __uint_as_float(s[x + 2 * y + 1]));
                    const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                    if (k == 0) {
                        m = top;
                    } else if (__any_sync(0xffffffffu, (top - m) * c > kTrLagBits)) {
                        const float f = m == -INFINITY ? 0.0f : ex2((m - top) * c);
                        m = top;
                        l *= f;
                        ok = warp_wait(&o_full[tile], visit - 1, limit);
                        if (!ok) break;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int x = 0; x < DP / 32; ++x) {
                            uint32_t o[32];
                            tmem_ld32_async(to + 32 * x, o);
                            tmem_wait_ld<32>(o);
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st32(to + 32 * x, o);
                        }
                    }
                    const float mc = (m == -INFINITY ? 0.0f : m * c) - kTrWeightBits;
                    const float2 c2 = make_float2(c, c), mc2 = make_float2(-mc, -mc);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int x = 0; x < BLK / 2; ++x) {
                        const float2 y = fma2(make_float2(__uint_as_float(s[2 * x]),
                                                          __uint_as_float(s[2 * x + 1])),
                                              c2, mc2);
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum[x & 1] = add2(sum[x & 1], e);
                        s[x] = E::pack(e.x, e.y);
                    }
#pragma unroll
                    for (int x = 0; x < BLK / 64; ++x) tmem_st32(ts + 32 * x, s + 32 * x);
                    tmem_wait_st();
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                }
                // (Of a warp without rows the weights are what was there.)
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[tile]);
            }
            if (!ok) break;
            block0 += n;
            if (n > 0) {
                ok = warp_wait(o_done, parts++, limit);
                if (!ok) break;
                tc_fence_after_sync();
            }
            // The row's maximum (base 2) and sum, and the factors of the outputs
            // in tensor memory: with one tile, both warpgroups' parts.
            float top = m == -INFINITY ? 0.0f : m * c, sum = l;
            float f[2] = {1.0f, 1.0f};
            bool has[2] = {mine > 0, false};
            int d0 = 0, d1 = DP;
            if (NQ == 1) {
                stats[128 * wg + tr] = make_float2(top, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                ok = warp_wait(joined, joins++, limit);
                if (!ok) break;
                const float2 a = stats[tr], z = stats[128 + tr];
                top = a.y == 0.0f ? z.x : z.y == 0.0f ? a.x : fmaxf(a.x, z.x);
                f[0] = a.y == 0.0f ? 0.0f : ex2(a.x - top);
                f[1] = z.y == 0.0f ? 0.0f : ex2(z.x - top);
                sum = fmaf(a.y, f[0], z.y * f[1]);
                has[0] = n > 0;
                has[1] = NT == 2 && n > 1;
                d0 = wg * (DP / 2);
                d1 = d0 + DP / 2;
            }
            const uint32_t from0 = NQ == 1 ? out0 : to;
            const int h = u.hk * group + (u.r0 + r) - token * group;
            const bool here = r < u.rows;
            const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
            uint16_t* row = here ? tree_out(t, p.b, token, h) : nullptr;
            float* part = nullptr;
            if (!p.whole) {
                const int64_t at = static_cast<int64_t>(p.place) * t.part_rows;
                part = t.part_out + at * t.d_head + r * 8;
                if (here && (NQ == 2 || wg == 0)) t.part_stats[at + r] = make_float2(top, sum);
            } else if (here && (NQ == 2 || wg == 0)) {
                tree_lse(t, p.b, token, h, top, sum);
            }
            if (warp_r < u.rows) {
#pragma unroll 1
                for (int d = d0; d < d1 && d < t.d_head; d += 32) {
                    uint32_t o[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = 0u;
                    if (has[0]) {
                        tmem_ld32_async(from0 + d, o);
                        tmem_wait_ld<32>(o);
                    }
                    // (Exactly 0 of what has no kept token: 0 times a NaN is not.)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        o[x] = f[0] == 0.0f || (NQ == 2 && sum == 0.0f)
                                   ? 0u : __float_as_uint(__uint_as_float(o[x]) * f[0]);
                    if (NQ == 1 && has[1]) {
                        uint32_t z[32];
                        tmem_ld32_async(out0 + DP + d, z);
                        tmem_wait_ld<32>(z);
                        if (f[1] != 0.0f) {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = __float_as_uint(fmaf(__uint_as_float(z[x]), f[1],
                                                            __uint_as_float(o[x])));
                        }
                    }
                    if (!here) continue;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        if (d + 8 * y >= t.d_head) break;
                        float v[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) v[x] = __uint_as_float(o[8 * y + x]);
                        if (p.whole) {
                            tree_store8<E>(row, d + 8 * y, v, inv);
                        } else {
                            float4* w = reinterpret_cast<float4*>(
                                part + static_cast<int64_t>(d / 8 + y) * t.part_rows * 8);
                            w[0] = make_float4(v[0], v[1], v[2], v[3]);
                            w[1] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
            }
            // The next part's products write over what was read here.
            if (NQ == 1) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                ok = warp_wait(joined, joins++, limit);
                tc_fence_after_sync();
            }
        }
    } else {
        give_registers<L::kRegsOther>();
        if (warp == kTrMmaWarp) {
            // ------------------------------------------------- MMA issuer
            const bool leader = elect_lane();
            const uint32_t q = tile_desc(smem_addr(smem + L::kQ));
            const uint32_t kd = tile_desc(smem_addr(smem + L::kK));
            const uint32_t vd = weights_desc<BLK>(smem_addr(smem + L::kV));
            constexpr uint32_t tile_step = NQ == 2 ? L::kTile / 16 : 0;
            constexpr uint32_t stage_step = L::kBlock / 16;
            const int steps = (t.d_head + 15) / 16;
            const uint32_t idesc = idesc_half(128, 16 * steps, true, E::kFp16);
            constexpr int kPerBlock = NQ;      // visits of a block
            int block0 = 0, parts = 0, visits[2] = {0, 0};
            bool ok = true;
            TreePart p;
            while (ok && walk.next(t, p)) {
                const TreeRows u = tree_rows<NQ>(t, p.row, p.n);
                const int n = tree_blocks<BLK>(t, p, u);
                if (n == 0) continue;
                const int all = n * kPerBlock;
                auto scores = [&](int v) {
                    const int i = NT == 2 ? v & 1 : 0;
                    const int kb = block0 + v / kPerBlock, st = kb % NS;
                    if (!warp_wait(&k_full[st], kb / NS, limit)) return false;
                    if (v == 0 && !warp_wait(q_full, parts, limit)) return false;
                    fence_proxy_async_smem();
                    tc_fence_after_sync();
                    mma_tiles<BLK, DP, E::kFp16>(tmem + BLK * i, q + i * tile_step,
                                                 kd + st * stage_step, steps, leader);
                    mma_commit(&s_full[i], leader);
                    if ((v + 1) % kPerBlock == 0) mma_commit(&k_empty[st], leader);
                    if (v + 1 == all) mma_commit(q_empty, leader);
                    return true;
                };
                for (int v = 0; v < NT && v < all && ok; ++v) ok = scores(v);
                for (int v = 0; v < all && ok; ++v) {
                    const int i = NT == 2 ? v & 1 : 0;
                    const int kb = block0 + v / kPerBlock, st = kb % NS;
                    ok = warp_wait(&v_full[st], kb / NS, limit) &&
                         warp_wait(&p_full[i], visits[i], limit);
                    if (!ok) break;
                    fence_proxy_async_smem();
                    tc_fence_after_sync();
                    mma_weights<BLK>(tmem + L::kOut + DP * i, tmem + BLK * i, vd + st * stage_step,
                                     idesc, v >= NT, leader);
                    mma_commit(&o_full[i], leader);
                    ++visits[i];
                    if ((v + 1) % kPerBlock == 0) mma_commit(&v_empty[st], leader);
                    if (v + 1 == all) mma_commit(o_done, leader);
                    if (v + NT < all) ok = scores(v + NT);
                }
                block0 += n;
                ++parts;
            }
            // No product may be in flight when the tensor memory is freed.
            mma_commit(drained, leader);
            mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
            __syncwarp();
        } else if (warp >= kTrCopyWarp) {
            // ----------------------------------------------------- copies
            constexpr int kUnits = DP / 8;         // 16-byte units of a row
            constexpr int kRows = BLK / 4;         // of a block, of this warp
            constexpr int kAtOnce = 32 / kUnits;   // rows an instruction copies
            const int cw = warp - kTrCopyWarp;
            const int unit = lane % kUnits;
            const bool in_head = 8 * unit < t.d_head;
            const uint32_t at_unit = in_head ? 8 * unit : 0;
            // Rows r0 + kAtOnce x + lane / kUnits of a tile of ROWS rows, from
            // the addresses that lanes 0, 1, .. hold of them.
            auto copy_rows = [&](unsigned char* tile, int tile_rows, int r0, int count,
                                 const uint16_t* address, uint32_t there) {
#pragma unroll 4
                for (int x = 0; x < count / kAtOnce; ++x) {
                    const int y = kAtOnce * x + lane / kUnits, r = r0 + y;
                    const uint64_t a = __shfl_sync(
                        0xffffffffu, reinterpret_cast<unsigned long long>(address), y);
                    const uint32_t bytes = in_head && (there >> y & 1u) ? 16u : 0u;
                    cp_async16_zfill(tile + (unit >> 3) * tile_rows * 128 + r * 128 +
                                         (((unit & 7) ^ (r & 7)) << 4),
                                     reinterpret_cast<const uint16_t*>(a) + at_unit, bytes);
                }
            };
            const int skip = BLK / t.page_size, rest = BLK - skip * t.page_size;
            int block0 = 0, parts = 0;
            bool ok = true;
            TreePart p;
            while (ok && walk.next(t, p)) {
                const TreeRows u = tree_rows<NQ>(t, p.row, p.n);
                const int n = tree_blocks<BLK>(t, p, u);
                if (n == 0) continue;
                // This lane's token of a block (lanes past the rows as others),
                // its entry of the table, its slot; looked up three blocks
                // ahead, a table's entry takes a microsecond to come when it is
                // not in a cache.
                int tok = p.s0 * BLK + cw * kRows + lane % kRows;
                int entry = tok / t.page_size, slot = tok - entry * t.page_size;
                struct Place {
                    int page, slot;   // slot -1: no token
                };
                auto locate = [&]() {
                    Place at{0, -1};
                    if (tok < p.n.len) {
                        at.slot = slot;
                        at.page = t.page_table[p.b * t.table_stride + entry];
                    }
                    tok += BLK;
                    entry += skip;
                    slot += rest;
                    if (slot >= t.page_size) {
                        slot -= t.page_size;
                        ++entry;
                    }
                    return at;
                };
                Place ahead[3];
#pragma unroll
                for (int x = 0; x < 3; ++x) ahead[x] = locate();
                auto load_q = [&]() {
                    if (parts > 0 && !warp_wait(q_empty, parts - 1, limit)) return false;
#pragma unroll 1
                    for (int i = 0; i < NQ; ++i) {
                        const int r = 128 * i + 32 * cw + lane;
                        const int token = (u.r0 + r) / group;
                        const bool valid = r < u.valid;
                        const uint16_t* a = t.q;
                        if (valid)
                            a = t.q + p.b * t.q_stride[0] + token * t.q_stride[1] +
                                (u.hk * group + (u.r0 + r) - token * group) * t.q_stride[2];
                        copy_rows(smem + L::kQ + i * L::kTile, 128, 32 * cw, 32, a,
                                  __ballot_sync(0xffffffffu, valid));
                    }
                    cp_async_arrive(q_full);
                    return true;
                };
                const uint16_t* kbase = t.k_pages + u.hk * t.k_stride[2];
                const uint16_t* vbase = t.v_pages + u.hk * t.v_stride[2];
                for (int j = 0; j < n && ok; ++j) {
                    const Place at = ahead[0];
                    ahead[0] = ahead[1];
                    ahead[1] = ahead[2];
                    ahead[2] = locate();
                    const bool valid = at.slot >= 0 && at.page >= 0 && at.page < t.num_pages;
                    if (at.slot >= 0 && !valid) raise_error(t.err, kBitBadPage);
                    const uint16_t *k = t.q, *v = t.q;
                    if (valid) {
                        k = kbase + at.page * t.k_stride[0] + at.slot * t.k_stride[1];
                        v = vbase + at.page * t.v_stride[0] + at.slot * t.v_stride[1];
                    }
                    const uint32_t there = __ballot_sync(0xffffffffu, valid);
                    const int kb = block0 + j, st = kb % NS;
                    if (kb >= NS) ok = warp_wait(&k_empty[st], kb / NS - 1, limit);
                    if (!ok) break;
                    copy_rows(smem + L::kK + st * L::kBlock, BLK, kRows * cw, kRows, k, there);
                    cp_async_arrive(&k_full[st]);
                    if (lane == 0) {
                        // The tokens that are there, one bit each.
                        uint32_t* w = words + 4 * (kb % kTrWords);
                        if (kRows == 32) w[cw] = there;
                        else reinterpret_cast<uint16_t*>(w)[cw] = static_cast<uint16_t>(there);
                        mbar_arrive(&k_full[st]);
                    }
                    if (kb >= NS) ok = warp_wait(&v_empty[st], kb / NS - 1, limit);
                    if (!ok) break;
                    copy_rows(smem + L::kV + st * L::kBlock, BLK, kRows * cw, kRows, v, there);
                    cp_async_arrive(&v_full[st]);
                    if (j == 0) ok = load_q();
                }
                block0 += n;
                ++parts;
            }
            cp_async_wait_all();
        }
    }

    // Sequences without blocks in a dealt batch: zeros, by the CTAs in turn;
    // what is wrong with a length is reported here too.
    for (int b = t.split ? static_cast<int>(blockIdx.x)
                         : static_cast<int>(blockIdx.x) / (t.width * t.bundles);
         b < t.batch; b += t.split ? static_cast<int>(gridDim.x) : t.batch) {
        bool bad;
        const TreeLens n = tree_lens(t, b, bad);
        if (bad && threadIdx.x == 0) raise_error(t.err, kBitBadPage);
        if (t.split && tree_steps<BLK>(n) == 0) {
            const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const int units = t.d_head / 8;
            for (int64_t e = threadIdx.x;
                 e < static_cast<int64_t>(t.new_tokens) * t.heads * units; e += kTrThreads) {
                const int64_t row = e / units;
                const int i = static_cast<int>(row / t.heads);
                const int h = static_cast<int>(row - static_cast<int64_t>(i) * t.heads);
                const int d = 8 * static_cast<int>(e - row * units);
                tree_store8<E>(tree_out(t, b, i, h), d, zero, 0.0f);
                if (d == 0) tree_lse(t, b, i, h, 0.0f, 0.0f);
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kTrMmaWarp) tmem_dealloc(tmem, L::kTmemCols);
    if (threadIdx.x == 0 && flags[0]) raise_error(t.err, kBitTimeout);
}

constexpr int kTrJoinThreads = 128;

// Joins a unit's parts: a CTA takes 32 rows, a lane each, and 32 columns.  A
// small batch has CTAs for every unit, a larger one for every place between two
// groups, where alone a unit can be cut, which join the unit that is cut there
// first (CUTS).
template <int BLK, class E, bool CUTS>
__global__ void __launch_bounds__(kTrJoinThreads) tree_join_kernel(const TreeTask t) {
    constexpr int kWarps = kTrJoinThreads / 32;
    __shared__ int scan[kWarps + 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int x = blockIdx.x % t.width, chunk = blockIdx.x / t.width;
    int b, bundle = 0, begin = 0, steps = 0, share = 1;
    bool bad, cut = true;
    if constexpr (!CUTS) {
        b = blockIdx.y / t.bundles;
        bundle = blockIdx.y - b * t.bundles;
        int before = 0, total = 0;
        for (int i = threadIdx.x; i < t.batch; i += kTrJoinThreads) {
            const int n = tree_steps<BLK>(tree_lens(t, i, bad)) * t.bundles;
            total += n;
            if (i < b) before += n;
        }
        int skip, all;
        tree_scan<kWarps>(total, scan, skip, all);
        __syncthreads();
        share = max(1, (all + t.groups - 1) / t.groups);
        tree_scan<kWarps>(before, scan, skip, all);
        steps = tree_steps<BLK>(tree_lens(t, b, bad));
        begin = all + bundle * steps;
    } else {
        TreeDeal d;
        const int later = blockIdx.y + 1;
        cut = tree_deal<kWarps, BLK>(t, later, scan, d);
        if (cut) {
            b = d.b;
            share = d.share;
            steps = tree_steps<BLK>(tree_lens(t, b, bad));
            bundle = steps > 0 ? min((d.g0 - d.base) / steps, t.bundles - 1) : 0;
            begin = d.base + bundle * steps;
            cut = begin < d.g0 && begin / share == later - 1;
        }
    }
    const int c0 = begin / share;
    const int c1 = cut && steps > 0 ? min((begin + steps - 1) / share, t.groups - 1) : c0;
    wait_for_previous_kernel();
    // Not cut (here first), without blocks, or finished by the only group that
    // had it.
    if (c0 >= c1) return;
    const int tiles = t.part_rows / 32;
    const int row = bundle * t.width + x;
    const int tile = row / t.kv_heads, hk = row - tile * t.kv_heads;
    const int r = 32 * (chunk % tiles) + lane;                 // of the unit
    const int col = 4 * (chunk / tiles) + warp;                // of 8 elements
    const int r_all = tile * t.unit_rows + r;
    if (8 * col >= t.d_head || r_all >= t.new_tokens * t.group || r >= t.unit_rows) return;
    // Part i: group c0 + i's first, but group c0's last where it had others
    // before.
    const int late = begin > c0 * share ? 1 : 0;
    auto place = [&](int i) {
        return static_cast<int64_t>(2 * ((c0 + i) * t.width + x) + (i == 0 ? late : 0)) *
               t.part_rows;
    };
    const int n = c1 - c0 + 1;
    float top = -INFINITY, sum = 0.0f;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < n; i0 += 4) {
        float2 st[4];
        float4 v[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            st[k] = make_float2(0.0f, 0.0f);
            v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + k < n) {
                const int64_t at = place(i0 + k);
                st[k] = t.part_stats[at + r];
                const float4* w = reinterpret_cast<const float4*>(
                    t.part_out + at * t.d_head + (static_cast<int64_t>(col) * t.part_rows + r) * 8);
                v[k][0] = w[0];
                v[k][1] = w[1];
            }
        }
        float m = top;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (st[k].y != 0.0f) m = fmaxf(m, st[k].x);
        const float f = top == -INFINITY ? 0.0f : ex2(top - m);
        sum *= f;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (st[k].y == 0.0f) continue;   // no kept tokens there
            const float g = ex2(st[k].x - m);
            sum = fmaf(st[k].y, g, sum);
            const float y[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                                v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(y[e], g, acc[e]);
        }
        top = m;
    }
    const int token = r_all / t.group, h = hk * t.group + r_all - token * t.group;
    tree_store8<E>(tree_out(t, b, token, h), 8 * col, acc,
                   sum == 0.0f ? 0.0f : __frcp_rn(sum));
    if (col == 0) tree_lse(t, b, token, h, top, sum);
}

template <int DP, int NQ, class E>
cudaError_t launch(const TreeTask& t, int slot, cudaStream_t stream) {
    using L = TreePlan<DP, NQ>;
    const auto kernel = tree_kernel<DP, NQ, E>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), slot, L::kBytes,
                                          false);
    if (e != cudaSuccess) return e;
    const int grid = (t.split ? t.groups : t.batch * t.bundles) * t.width;
    kernel<<<grid, kTrThreads, L::kBytes, stream>>>(t);
    e = cudaGetLastError();
    if (e != cudaSuccess || !t.split || t.groups == 1) return e;
    const int64_t units = static_cast<int64_t>(t.batch) * t.bundles;
    const bool cuts = units >= t.groups;
    const int chunks = t.part_rows / 32 * ((t.d_head + 31) / 32);
    return launch_shaped(
        cuts ? tree_join_kernel<L::kBlk, E, true> : tree_join_kernel<L::kBlk, E, false>,
        {dim3(t.width * chunks, cuts ? t.groups - 1 : static_cast<unsigned>(units)),
         kTrJoinThreads, 0, stream, true, 1},
        t);
}

template <class E>
cudaError_t launch_type(const TreeTask& t, int slot, cudaStream_t stream) {
    if (t.d_head > 128) return launch<256, 1, E>(t, slot, stream);
    const bool pair = t.unit_rows == 256;
    if (t.d_head > 64)
        return pair ? launch<128, 2, E>(t, slot + 1, stream)
                    : launch<128, 1, E>(t, slot + 2, stream);
    return pair ? launch<64, 2, E>(t, slot + 3, stream) : launch<64, 1, E>(t, slot + 4, stream);
}

}  // namespace

cudaError_t launch_tree(const TreeTask& task, cudaStream_t stream) {
    return task.fp16 ? launch_type<TrFP16>(task, 80, stream)
                     : launch_type<TrBF16>(task, 85, stream);
}

}  // namespace cs
