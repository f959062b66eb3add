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
//   warp 9          works out the CTA's parts, a few ahead;
//   warps 12, 13    look pages up and keep the rings of K and V full by tensor
//                   copies, a lane a box: the tokens of one page, 8 or more;
//   warps 14, 15    queries, by a tensor copy of whole tokens where the query
//                   heads of a key head divide 128, or 16 bytes at a time;
//   warps 12-15     all of it 16 bytes at a time, where pages are not of a
//                   multiple of 8 tokens or strides are none of a tensor map's
//                   (131072 tokens in pages of one: 105 us, of 64 91.5).
//
// Measured, bf16, heads of 128, 32 on 8 key heads, GPU time of a call in a graph:
//   1 x 32 tokens over 131072   91.5 us, 5.9 TB/s (87% of a plain copy), 0.75
//                               PFLOP/s: DRAM, a block of 64 KB in 2750 cycles;
//   32 x 16 over 256 .. 4096    40.0 us, 4.4 TB/s: as above, and 8 us until
//                               the first pages are there (lengths, table and
//                               copies one after the other), 3 us of join;
//   8 x 64 over 8192            65.2 us, 4.2 TB/s and 1.05 PFLOP/s: a pair's block
//                               takes 3120 cycles, of which the tensor pipe works
//                               2048: a tile's chain (products, softmax, products)
//                               is longer than the other tile's products, and its
//                               256 columns leave no room for a second score tile;
//   2 x 512 of 8192 (a chunk)   106.5 us, 1.25 PFLOP/s (66% of a library product):
//                               the same; start and join take 15 us.
// (Both chains are also fused_attention's.)
//
// The weights are rounded to the cache's type, the one the tensor cores take
// beside its values; their sum is taken in fp32 before that.  Their maximum may
// lag by 2^6.  In fp16, which has no exponents below 2^-24, they carry a factor
// 2^8: the largest, 2^8 to 2^14, leaves 2^-32 of it.  In bf16, whose values reach
// as far as fp32, they carry 2^-6 / n, n the sequence's tokens, up to a power of
// two: the weights of any of them have a sum of at most 1, and no sum of weights
// and finite values overflows (with 2^8, values from about 2^114 on could; a value
// keeps bf16's bits down to n 2^-134).
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "cs_fattn.cuh"
#include "cs_pages.h"
#include "cs_tensormap.h"

namespace cs {
namespace {

using namespace csd;

constexpr int kTrThreads = 512;
constexpr int kTrMmaWarp = 8;
constexpr int kTrPartWarp = 9;
constexpr int kTrCopyWarp = 12;
constexpr int kTrWarpBatch = 256;      // sequences whose lengths one warp adds up
constexpr float kTrLagBits = 6.0f;     // how far the maximum may lag
// Above this, fma(s, c, -m c) of the maximum itself, which is what rounding m c
// took off, is no longer a small number (from 2^31 on 2^x overflows, or leaves no
// weight): the maximum is taken off the scores first.  (256 x 512 tokens in trees of
// 4: 82.5 us without that code, 85.0 with it; others within 1%.)
constexpr float kTrLarge = 0x1p22f;
constexpr int kTrWords = 8;            // blocks whose kept tokens are noted
constexpr int kTrParts = 4;            // parts that are known ahead
constexpr int kTrPartWarps = 13;       // that read them

// weight_bits: log2 of the common factor of the weights of a sequence's tokens.
struct TrBF16 {
    static constexpr bool kFp16 = false;
    static __device__ __forceinline__ float weight_bits(int tokens) {
        return -kTrLagBits - static_cast<float>(32 - __clz(tokens - 1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        return pack_bf16(lo, hi);
    }
};
struct TrFP16 {
    static constexpr bool kFp16 = true;
    static __device__ __forceinline__ float weight_bits(int) { return 8.0f; }
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
    static constexpr int kNumBars = 4 * kStages + 9 + 2 * kTrParts;
    static constexpr int kWords = kBars + (8 * kNumBars + 15) / 16 * 16;  // [kTrWords][4]
    static constexpr int kParts = kWords + kTrWords * 16;
    static constexpr int kScan = kParts + kTrParts * 48;   // [20] ints
    static constexpr int kFlags = kScan + 80;              // abort, tmem
    static constexpr int kStats = kFlags + 16;             // [2][128] float2 (one tile)
    static constexpr int kBytes = kStats + (NQ == 1 ? 2 * 128 * 8 : 0);
    static_assert(kBytes <= 232448, "shared memory of a CTA");
    static_assert(kStages + 2 <= kTrWords, "a block's words outlive its keys' stage");
};

__device__ __forceinline__ TreeLens tree_lens(const TreeTask& t, int b, bool& bad) {
    const int n = t.lengths[b];
    const int most = t.max_pages * t.page_size;
    const int w = t.new_lengths ? t.new_lengths[b] : t.new_tokens;
    const TreeLens x = tree_lens_of(n, w, most, t.new_tokens);
    bad = n < 0 || n > most || w != x.fresh;
    return x;
}

__device__ __forceinline__ int tree_places(int steps) {
    return steps > 0 ? steps + kTreePartCost : 0;
}

// Blocks of a unit of sequence b.
template <int BLK>
__device__ __forceinline__ int tree_steps(const TreeLens& x) {
    return x.fresh > 0 ? (x.len + BLK - 1) / BLK : 0;
}

// The sum of n over the threads before this one and over all of the CTA of
// 32 WARPS threads, or of the calling warp (WARPS 1); scan: WARPS shared ints,
// free again after the caller's next barrier.
template <int WARPS>
__device__ __forceinline__ void tree_scan(int n, int* scan, int& before, int& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int up = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
    }
    before = up - n;
    if (WARPS == 1) {
        all = __shfl_sync(0xffffffffu, up, 31);
        return;
    }
    if (lane == 31) scan[warp] = up;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
    }
}
template <int WARPS>
__device__ __forceinline__ void tree_sync() {
    if (WARPS == 1) __syncwarp();
    else __syncthreads();
}

// What a group of CTAs has of the batch's list: for each sequence, for each of
// its bundles of `width` units side by side, kTreePartCost places for a part's
// start and end and then its blocks.  Places g0 .. g1 - 1, the first in sequence
// b whose first is `base`.
struct TreeDeal {
    int g0, g1, b, base, share;
    TreeLens n;
};

// By a whole CTA of 32 WARPS threads, or one warp; false without places.  scan:
// WARPS + 4 shared ints.
template <int WARPS, int BLK>
__device__ __forceinline__ bool tree_deal(const TreeTask& t, int grp, int* scan, TreeDeal& d) {
    constexpr int kThreads = 32 * WARPS;
    const int thread = WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
    bool bad;
    TreeLens mine{};
    auto places = [&](int i) {
        if (i < t.batch) mine = tree_lens(t, i, bad);
        return i < t.batch ? tree_places(tree_steps<BLK>(mine)) * t.bundles : 0;
    };
    int total = 0, before;
    const bool once = t.batch <= kThreads;   // one walk over the lengths is enough
    if (!once) {
        int n = 0;
#pragma unroll 4
        for (int i = thread; i < t.batch; i += kThreads) n += places(i);
        tree_scan<WARPS>(n, scan, before, total);
        tree_sync<WARPS>();
    }
    int done = 0;
    for (int b0 = 0; b0 < t.batch; b0 += kThreads) {
        const int i = b0 + thread;
        const int n = places(i);
        int first, all;
        tree_scan<WARPS>(n, scan, first, all);
        if (once) total = all;
        d.share = max(1, t.by_groups(total + t.groups - 1));
        d.g0 = grp * d.share;
        d.g1 = min(total, d.g0 + d.share);
        if (d.g0 >= d.g1) return false;
        first += done;
        if (first <= d.g0 && d.g0 < first + n) {
            scan[WARPS] = i;
            scan[WARPS + 1] = first;
            scan[WARPS + 2] = mine.len;
            scan[WARPS + 3] = mine.fresh;
        }
        done += all;
        tree_sync<WARPS>();
        if (done > d.g0) break;
    }
    // (In range even where the lengths were changed under the call: what comes of
    // them is then wrong, but no page table, row or part is left.)
    const TreeStart x = tree_start_of(scan + WARPS, d.g0, t.batch, t.max_pages * t.page_size,
                                      t.new_tokens);
    d.b = x.b;
    d.base = x.base;
    d.n = x.n;
    return true;
}

// Blocks of a unit that a CTA takes, all of them or a part of them, as one warp
// works them out for the others.  Rows are token by token, `group` heads each.
struct alignas(16) TreePart {
    int n;         // blocks, which may be none; -1: no part is left
    int key0;      // the first one's first token
    int b, hk;
    int r0, rows;  // first row of the unit, and rows there
    int valid;     // of those: rows of new tokens, may be negative
    int len;       // tokens of the sequence,
    int context;   // those before all new ones
    int place;     // of the workspace; -1: finished here
    int pad[2];
};

template <int BLK, int NQ>
__device__ __forceinline__ TreePart tree_part(const TreeTask& t, int b, const TreeLens& n,
                                              int unit, int s0, int s1, int steps) {
    TreePart p{};
    const int tile = t.by_kv_heads(unit);
    p.b = b;
    p.hk = unit - tile * t.kv_heads;
    p.r0 = 128 * NQ * tile;
    p.rows = min(128 * NQ, t.new_tokens * t.group - p.r0);
    p.valid = min(128 * NQ, n.fresh * t.group - p.r0);
    p.key0 = s0 * BLK;
    p.len = n.len;
    p.context = n.len - n.fresh;
    // A part at a share's end begins its unit, one at the start does not.
    p.place = s0 == 0 && s1 == steps ? -1 : 2 * static_cast<int>(blockIdx.x) + (s0 == 0);
    // None without rows, and none past the last row's token where each row
    // attends those before it.
    int last = p.valid > 0 ? s1 : s0;
    if (!t.mask && p.valid > 0)
        last = min(last, (p.context + t.by_group(p.r0 + p.valid - 1) + BLK) / BLK);
    p.n = max(0, last - s0);
    return p;
}

// A row's kept tokens of a block: token x is new token j0 + x, of the row's
// `fresh`, where that is not negative, and a token before the new ones, which
// all rows keep, where it is.  Clears the bits of what the row, `fresh` bytes,
// does not keep.  A thread a row: words of 4 bytes, eight under way at once,
// single bytes at the row's ends; words that no row of the warp, which have up to
// `most` bytes, reaches into are passed over.  (Whole warps a row, 32 bytes at a
// time, took ten microseconds for 64 rows of 64 in a CTA of its own.)
template <int BLK>
__device__ __forceinline__ void tree_mask_row(const uint8_t* row, int j0, int fresh, int most,
                                              uint32_t (&kept)[BLK / 32]) {
    const int lo = max(0, -j0), hi = min(BLK, fresh - j0);   // x of the row's bytes
    const int64_t at = reinterpret_cast<int64_t>(row) + j0;  // of x = 0
    const int head = static_cast<int>(at & 3);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(at - head);
    uint32_t bits[BLK / 32 + 1];   // of x = -head ..
#pragma unroll
    for (int w = 0; w <= BLK / 32; ++w) bits[w] = 0u;
    const int first = (lo + head + 3) / 4 * 4 - head, last = (hi + head) / 4 * 4 - head;
    bool edge[6];
    int edge_x[6];
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        edge_x[e] = lo + e;
        edge_x[3 + e] = max(first, last) + e;
        edge[e] = edge_x[e] < min(first, hi) && row[j0 + edge_x[e]] != 0;
        edge[3 + e] = edge_x[3 + e] < hi && row[j0 + edge_x[3 + e]] != 0;
    }
#pragma unroll 1
    for (int g = 0; g <= BLK / 32; ++g) {
        if (-j0 >= 32 * g + 32 || most - j0 <= 32 * g - 3) continue;
        uint32_t v[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int x = 32 * g + 4 * k - head;
            v[k] = x >= lo && x + 4 <= hi ? __ldg(words + 8 * g + k) : 0u;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // Bytes that are not 0, to their lowest bits, and these side by side.
            const uint32_t m = ((((v[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | v[k]) >> 7) & 0x01010101u;
            sum |= (m * 0x01020408u >> 24 & 15u) << (4 * k);
        }
#pragma unroll
        for (int y = 0; y <= BLK / 32; ++y) bits[y] = y == g ? sum : bits[y];
    }
#pragma unroll
    for (int w = 0; w < BLK / 32; ++w) {
        uint32_t keep = __funnelshift_r(bits[w], bits[w + 1], head) | bits_below(-j0, 32 * w);
#pragma unroll
        for (int e = 0; e < 6; ++e)
            if (edge[e] && edge_x[e] >> 5 == w) keep |= 1u << (edge_x[e] & 31);
        kept[w] &= keep;
    }
}

// Of a block whose boxes with bit 0 lie on pages outside the cache: reports
// that, and gives lane w the tokens 32 w to 32 w + 31 that are there.
__device__ __forceinline__ uint32_t tree_lost(const TreeTask& t, uint32_t good) {
    const int lane = threadIdx.x & 31;
    uint32_t bits = 0;
#pragma unroll 1
    for (int x = 0; x < 32; ++x)
        bits |= (good >> (((32 * lane + x) >> t.box_bits) & 31) & 1u) << x;
    if (lane == 0) raise_error(t.err, kBitBadPage);
    return bits;
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];"
                 :: "r"(smem_addr(bar)) : "memory");
}

// warp_wait for two barriers at once.  (Every lane polls both: lanes that poll
// different ones leave the warp in two halves, each of which would run what
// follows, and the products want a whole warp.)
__device__ __forceinline__ bool warp_wait2(uint64_t* a, int phase_a, uint64_t* b, int phase_b,
                                           const WaitLimit& w) {
    const uint32_t bar_a = smem_addr(a), bar_b = smem_addr(b);
    const uint32_t parity_a = phase_a & 1, parity_b = phase_b & 1;
    auto both = [&] {
        const bool x = mbar_try_wait<false>(bar_a, parity_a);
        const bool y = mbar_try_wait<false>(bar_b, parity_b);
        return __all_sync(0xffffffffu, x && y);
    };
    bool ok = both();
    if (!ok) {
        const long long c0 = clock64();
        for (uint32_t i = 0; i < (1u << 31); ++i) {
            ok = both();
            const bool over = *w.abort_flag || clock64() - c0 > static_cast<long long>(w.cycles);
            if (ok || __any_sync(0xffffffffu, over)) break;
        }
        if (!ok) *w.abort_flag = 1u;
    }
    __syncwarp();
    return ok;
}

__device__ __forceinline__ uint16_t* tree_out(const TreeTask& t, int b, int i, int h) {
    return t.out + b * t.o_stride[0] + i * t.o_stride[1] + h * t.o_stride[2];
}

// A row's lse, and whether its sum is finite: weights are 2^(score - top).
__device__ __forceinline__ void tree_lse(const TreeTask& t, int b, int i, int h, float top,
                                         float sum) {
    if (t.lse)
        t.lse[(static_cast<int64_t>(b) * t.new_tokens + i) * t.heads + h] =
            sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    if (!isfinite(sum)) raise_error(t.err, kBitNan);
}

template <int DP, int NQ, class E>
__global__ void __launch_bounds__(kTrThreads, 1)
tree_kernel(const TreeTask t, const __grid_constant__ CUtensorMap map_k,
            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q) {
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
    uint64_t* s_full = v_empty + NS;          // [2] scores of a block, and the P V before
    uint64_t* p_full = s_full + 2;            // [2] its weights, from four warps
    uint64_t* q_full = p_full + 2;
    uint64_t* q_empty = q_full + 1;           // the part's last scores completed
    uint64_t* o_done = q_empty + 1;           // the part's last P V completed
    uint64_t* drained = o_done + 1;
    uint64_t* joined = drained + 1;           // eight softmax warps
    uint64_t* part_full = joined + 1;         // [kTrParts]
    uint64_t* part_empty = part_full + kTrParts;
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kWords);
    TreePart* ahead_of = reinterpret_cast<TreePart*>(smem + L::kParts);
    int* scan = reinterpret_cast<int*>(smem + L::kScan);
    volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags);
    const WaitLimit limit{flags, t.wait_limit_cycles};

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const bool tensor_copies = t.box_bits >= 0;
    if (warp == kTrCopyWarp) {
        for (int i = lane; i < L::kNumBars; i += 32) {
            uint64_t* bar = bars + i;
            mbar_init(bar, bar < k_empty ? (tensor_copies ? 1 : 128 + 4)
                           : bar >= v_full && bar < v_empty ? (tensor_copies ? 1 : 128)
                           : bar == q_full ? (t.tensor_q ? 1 : tensor_copies ? 64 : 128)
                           : bar >= p_full && bar < q_full ? 4
                           : bar == joined ? 8
                           : bar >= part_empty ? kTrPartWarps : 1);
        }
        if (lane == 0) flags[0] = 0u;
        fence_mbar_init();
    } else if (warp == kTrMmaWarp) {
        tmem_alloc(const_cast<uint32_t*>(flags) + 1, L::kTmemCols);
    } else if (warp == kTrCopyWarp + 1 && lane == 0 && tensor_copies) {
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
        if (t.tensor_q) prefetch_tmap(&map_q);
    }
    // Launched while the kernel before ends; nothing of memory is touched above.
    // The join may start only after this wait, since it reads the lengths, which
    // a kernel before this one (paged_extend's) may have written, before its own.
    wait_for_previous_kernel();
    allow_next_kernel();
    const int grp = t.by_width(static_cast<int>(blockIdx.x));
    TreeDeal deal{};
    bool any = false;
    // A large batch's lengths are added up by the whole CTA.
    const bool large = t.split && t.batch > kTrWarpBatch;
    if (large) any = tree_deal<kTrThreads / 32, BLK>(t, grp, scan, deal);
    else if (t.split && warp == kTrPartWarp) any = tree_deal<1, BLK>(t, grp, scan, deal);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = flags[1];
    const int group = t.group;
    // Part i, to be given back after its last use by one arrival of the warp.
    auto part = [&](int i, bool& ok) {
        ok = warp_wait(&part_full[i % kTrParts], i / kTrParts, limit);
        return &ahead_of[i % kTrParts];
    };
    auto done_with = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&part_empty[i % kTrParts]);
    };

    if (warp < 8) {
        // -------------------------------------------------------- softmax
        take_registers<L::kRegsSoftmax>();
        const int wg = warp >> 2;              // warpgroup
        const int tile = NT == 2 ? wg : 0;
        const int tr = 32 * (warp & 3) + lane; // row of the tile
        const int warp_r = (NQ == 2 ? 128 * wg : 0) + 32 * (warp & 3);   // of the unit
        const int r = warp_r + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + BLK * tile;
        const uint32_t out0 = tmem + lanes + L::kOut;
        const uint32_t to = out0 + DP * tile;
        const float c = t.scale * kLog2e;
        // This warpgroup's blocks: all of them, or every other one.
        constexpr int kStep = NQ == 1 && NT == 2 ? 2 : 1;
        const int first = kStep == 2 ? wg : 0;
        int visit = 0;      // blocks of this warpgroup so far, over all parts
        int with_blocks = 0;   // parts so far that have some
        int block0 = 0;     // blocks of the parts before
        int joins = 0;
        for (int ip = 0;; ++ip) {
            bool ok;
            const TreePart* p = part(ip, ok);
            if (!ok) break;
            const int n = p->n;
            if (n < 0) break;
            const int mine = NT == 1 && wg > 0 ? 0 : (n - first + kStep - 1) / kStep;
            const float bits = E::weight_bits(p->len);
            float m = -INFINITY, l = 0.0f;
            bool large = false;   // any maximum of the warp
            auto is_large = [&](float x) { return x != -INFINITY && fabsf(x * c) > kTrLarge; };
            if (mine > 0) {
                const int context = p->context, token = t.by_group(p->r0 + r);
                const bool warp_valid = warp_r < p->valid;
                // The row keeps the tokens below this, and of them those the
                // mask keeps; every row of the warp those below `all_below`.
                // (Rows past the new tokens count for nothing in the end.)
                const int row_limit = t.mask || r >= p->valid ? p->len : context + token + 1;
                const int all_below =
                    __reduce_min_sync(0xffffffffu, t.mask ? min(row_limit, context) : row_limit);
                int key = p->key0 + first * BLK;
                for (int k = 0; k < mine; ++k, ++visit, key += kStep * BLK) {
                    uint32_t kept[BLK / 32];
                    bool edge = key + BLK > all_below;
                    if (edge) {
#pragma unroll
                        for (int w = 0; w < BLK / 32; ++w)
                            kept[w] = bits_below(row_limit, key + 32 * w);
                        if (t.mask && warp_valid && key + BLK > context)
                            tree_mask_row<BLK>(
                                t.mask + p->b * t.mask_stride[0] + token * t.mask_stride[1],
                                key - context, r < p->valid ? p->len - context : 0,
                                p->len - context, kept);
                    }
                    ok = warp_wait(&s_full[tile], visit, limit);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (warp_valid) {
                        // (Tokens that are not in the cache, too.)
                        const uint4 there = *reinterpret_cast<const uint4*>(
                            words + 4 * ((block0 + first + kStep * k) % kTrWords));
                        const uint32_t in[4] = {there.x, there.y, there.z, there.w};
                        uint32_t every = ~0u;
#pragma unroll
                        for (int w = 0; w < BLK / 32; ++w) every &= in[w];
                        if (every != ~0u || edge) {
#pragma unroll
                            for (int w = 0; w < BLK / 32; ++w)
                                kept[w] = edge ? kept[w] & in[w] : in[w];
                            edge = true;
                        }
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
                            large = __any_sync(0xffffffffu, is_large(m));
                        } else if (__any_sync(0xffffffffu, (top - m) * c > kTrLagBits)) {
                            const float f = m == -INFINITY ? 0.0f : ex2((m - top) * c);
                            m = top;
                            large = __any_sync(0xffffffffu, is_large(m));
                            l *= f;
                            // (The P V before has completed: the scores came
                            // after it from the same thread.)
#pragma unroll 1
                            for (int x = 0; x < DP; x += 16) {
                                float o[16];
                                tmem_ld16(to + x, o);
                                uint32_t w[16];
#pragma unroll
                                for (int y = 0; y < 16; ++y) w[y] = __float_as_uint(o[y] * f);
                                tmem_st16(to + x, w);
                            }
                        }
                        float mc = (m == -INFINITY ? 0.0f : m * c) - bits;
                        if (__builtin_expect(large, 0)) {
                            // (The warp's other rows as without this.)
                            const bool here = is_large(m);
                            const float off = here ? -m : 0.0f;
                            const float2 m2 = make_float2(off, off);
                            mc = here ? -bits : mc;
#pragma unroll
                            for (int x = 0; x < BLK; x += 2) {
                                const float2 y = add2(make_float2(__uint_as_float(s[x]),
                                                                  __uint_as_float(s[x + 1])),
                                                      m2);
                                s[x] = __float_as_uint(y.x);
                                s[x + 1] = __float_as_uint(y.y);
                            }
                        }
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
            }
            block0 += n;
            if (r >= p->valid) l = 0.0f;
            // What the row's weights are relative to (base 2; mc above) and their
            // sum, and the factors of the outputs in tensor memory: with one tile,
            // both warpgroups' parts.
            // (Finite: a part's maximum past fp32 in base 2 is its end.)
            float top = (m == -INFINITY ? 0.0f : m * c) - bits, sum = l;
            top = fminf(fmaxf(top, -FLT_MAX), FLT_MAX);
            float f0 = l == 0.0f ? 0.0f : 1.0f, f1 = 0.0f;
            if (NQ == 1) {
                float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
                stats[128 * wg + tr] = make_float2(top, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                ok = warp_wait(joined, joins++, limit);
                if (!ok) break;
                const float2 a = stats[tr], z = stats[128 + tr];
                top = a.y == 0.0f ? z.x : z.y == 0.0f ? a.x : fmaxf(a.x, z.x);
                f0 = a.y == 0.0f ? 0.0f : ex2(a.x - top);
                f1 = z.y == 0.0f ? 0.0f : ex2(z.x - top);
                sum = fmaf(a.y, f0, z.y * f1);
            }
            // Where the row goes, worked out while the last products run.
            const int rows = p->rows, place = p->place;
            const bool here = r < rows;
            const int token = t.by_group(p->r0 + r);
            const int h = p->hk * group + (p->r0 + r) - token * group;
            // Whose columns: with one tile each warpgroup half of them.
            const int d0 = NQ == 1 ? wg * (DP / 2) : 0;
            const int d1 = min(t.d_head, NQ == 1 ? d0 + DP / 2 : DP);
            const uint32_t from = NQ == 1 ? out0 : to;
            uint16_t* row = nullptr;
            float4* part_row = nullptr;
            if (place < 0) {
                if (here) row = tree_out(t, p->b, token, h);
                if (here && (NQ == 2 || wg == 0)) tree_lse(t, p->b, token, h, top, sum);
                const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
                f0 *= inv;
                f1 *= inv;
            } else {
                const int64_t at = static_cast<int64_t>(place) * t.part_rows;
                part_row = reinterpret_cast<float4*>(t.part_out + at * t.d_head) + r;
                if (here && (NQ == 2 || wg == 0)) t.part_stats[at + r] = make_float2(top, sum);
            }
            done_with(ip);
            if (n > 0) {
                ok = warp_wait(o_done, with_blocks++, limit);
                if (!ok) break;
                tc_fence_after_sync();
            }
            if (warp_r < rows) {
                const bool second = NQ == 1 && NT == 2 && n > 1;
#pragma unroll 1
                for (int d = d0; d < d1; d += 32) {
                    uint32_t o[32], z[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = z[x] = 0u;
                    if (n > 0) {
                        tmem_ld16_async(from + d, o);
                        tmem_ld16_async(from + d + 16, o + 16);
                    }
                    if (second) {
                        tmem_ld16_async(out0 + DP + d, z);
                        tmem_ld16_async(out0 + DP + d + 16, z + 16);
                    }
                    tmem_wait_ld<32>(o);
                    tmem_wait_ld<32>(z);
                    float v[32];
                    // (Exactly 0 of what has no kept token: 0 times a NaN is not.)
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        v[x] = f0 == 0.0f ? 0.0f : __uint_as_float(o[x]) * f0;
                        if (NQ == 1 && NT == 2)
                            v[x] = f1 == 0.0f ? v[x] : fmaf(__uint_as_float(z[x]), f1, v[x]);
                    }
                    if (!here) continue;
                    if (place < 0) {
#pragma unroll
                        for (int y = 0; y < 32; y += 8)
                            if (d + y < t.d_head)
                                *reinterpret_cast<uint4*>(row + d + y) = make_uint4(
                                    E::pack(v[y], v[y + 1]), E::pack(v[y + 2], v[y + 3]),
                                    E::pack(v[y + 4], v[y + 5]), E::pack(v[y + 6], v[y + 7]));
                    } else {
                        float4* w = part_row + (d / 4) * t.part_rows;
#pragma unroll
                        for (int y = 0; y < 32; y += 4, w += t.part_rows)
                            if (d + y < t.d_head)
                                *w = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                    }
                }
            }
            // The next part's products write over what was read here.
            if (NQ == 1) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(joined);
                ok = warp_wait(joined, joins++, limit);
                if (!ok) break;
                tc_fence_after_sync();
            }
        }
    } else {
        give_registers<L::kRegsOther>();
        if (warp == kTrMmaWarp) {
            // ------------------------------------------------- MMA issuer
            // (One warp for both accumulators: with one for each, whose products
            // mix in the tensor pipe, two prompts' chunks of 512 over 8192
            // tokens took 132 us, and 121 so.  Nor could two warps take one
            // tile's blocks in turn: a ring's barriers are told apart by the
            // parity of their phase alone, so who waits for one has to wait for
            // all.)
            const bool leader = elect_lane();
            const uint32_t q = tile_desc(smem_addr(smem + L::kQ));
            const uint32_t kd = tile_desc(smem_addr(smem + L::kK));
            const uint32_t vd = weights_desc<BLK>(smem_addr(smem + L::kV));
            constexpr uint32_t tile_step = NQ == 2 ? L::kTile / 16 : 0;
            constexpr uint32_t stage_step = L::kBlock / 16;
            const int steps = (t.d_head + 15) / 16;
            const uint32_t idesc = idesc_half(128, 16 * steps, true, E::kFp16);
            int block0 = 0, with_blocks = 0;
            int before[2] = {0, 0};   // visits of the parts before
            for (int ip = 0;; ++ip) {
                bool ok;
                const TreePart* p = part(ip, ok);
                if (!ok) break;
                const int n = p->n, past = p->len - p->key0;
                done_with(ip);
                if (n < 0) break;
                if (n == 0) continue;
                // Visits: block v with accumulator v mod 2, or of a pair block
                // v / 2 with each tile.  i: the accumulator of v.
                const int all = n * NQ;
                auto scores = [&](int v, int i) {
                    const int kb = block0 + v / NQ, st = kb % NS;
                    if (NQ == 1 || i == 0) {
                        if (!warp_wait2(&k_full[st], kb / NS, q_full, with_blocks, limit))
                            return false;
                        if (!tensor_copies || v == 0) fence_proxy_async_smem();
                        tc_fence_after_sync();
                    }
                    mma_tiles<BLK, DP, E::kFp16>(tmem + BLK * i, q + i * tile_step,
                                                 kd + st * stage_step, steps, leader);
                    mma_commit(&s_full[i], leader);
                    if (NQ == 1 || i == 1) mma_commit(&k_empty[st], leader);
                    if (v + 1 == all) mma_commit(q_empty, leader);
                    return true;
                };
                auto weights = [&](int v, int i) {
                    const int kb = block0 + v / NQ, st = kb % NS;
                    if (!warp_wait2(&v_full[st], kb / NS, &p_full[i], before[i] + v / NT, limit))
                        return false;
                    if (!tensor_copies) {
                        fence_proxy_async_smem();
                    } else if (NQ == 1 || i == 0) {
                        // Values past the length, which a tensor copy brings in
                        // with the last ones before: 0 times them has to be 0.
                        const int there = past - v / NQ * BLK;
                        const int rows = -there & ((1 << t.box_bits) - 1);
                        if (there < BLK && rows != 0) {
                            unsigned char* tile = smem + L::kV + st * L::kBlock + there * 128;
#pragma unroll 1
                            for (int e = lane; e < rows * (DP / 8); e += 32) {
                                const int r = e / (DP / 8), unit = e % (DP / 8);
                                *reinterpret_cast<uint4*>(tile + (unit >> 3) * BLK * 128 +
                                                          r * 128 + (unit & 7) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    tc_fence_after_sync();
                    mma_weights<BLK>(tmem + L::kOut + DP * i, tmem + BLK * i, vd + st * stage_step,
                                     idesc, v >= NT, leader);
                    if (NQ == 1 || i == 1) mma_commit(&v_empty[st], leader);
                    if (v + 1 == all) mma_commit(o_done, leader);
                    return true;
                };
                ok = scores(0, 0);
                if (NT == 2 && all > 1 && ok) ok = scores(1, 1);
                for (int v = 0; v < all && ok; v += NT) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        if (!ok || v + i >= all) break;
                        ok = weights(v + i, i);
                        if (ok && v + i + NT < all) ok = scores(v + i + NT, i);
                    }
                }
                if (!ok) break;
                block0 += n;
                before[0] += (all + NT - 1) / NT;
                before[1] += all / 2;
                ++with_blocks;
            }
            // No product may be in flight when the tensor memory is freed.
            mma_commit(drained, leader);
            mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
            __syncwarp();
        } else if (warp == kTrPartWarp) {
            // ------------------------------------------------------ parts
            int ip = 0;
            bool ok = true, bad;
            auto give = [&](const TreePart& p) {
                if (ip >= kTrParts)
                    ok = warp_wait(&part_empty[ip % kTrParts], ip / kTrParts - 1, limit);
                if (!ok) return;
                if (lane == 0) {
                    ahead_of[ip % kTrParts] = p;
                    mbar_arrive(&part_full[ip % kTrParts]);
                }
                ++ip;
                __syncwarp();
            };
            if (t.split) {
                int g = deal.g0, b = deal.b - 1, bundle = t.bundles, at = 0, steps = 0;
                TreeLens n{};
                if (any) {
                    n = deal.n;
                    ++b;
                    steps = tree_steps<BLK>(n);
                    const int places = max(1, tree_places(steps));
                    bundle = min((g - deal.base) / places, t.bundles);
                    at = (g - deal.base) % places;
                }
                while (any && ok && g < deal.g1) {
                    while (b < t.batch && (steps == 0 || bundle == t.bundles)) {
                        if (++b == t.batch) break;
                        n = tree_lens(t, b, bad);
                        steps = tree_steps<BLK>(n);
                        bundle = 0;
                    }
                    if (b >= t.batch) break;
                    const int places = tree_places(steps);
                    const int to = min(places, at + deal.g1 - g);
                    const int s0 = max(0, at - kTreePartCost), s1 = to - kTreePartCost;
                    if (s1 > s0)
                        give(tree_part<BLK, NQ>(
                            t, b, n, bundle * t.width + static_cast<int>(blockIdx.x) - grp * t.width,
                            s0, s1, steps));
                    g += to - at;
                    at = to;
                    if (at == places) {
                        at = 0;
                        ++bundle;
                    }
                }
            } else {
                // Each group one bundle of one sequence, blocks or not.
                const int b = grp / t.bundles;
                const TreeLens n = tree_lens(t, b, bad);
                const int steps = tree_steps<BLK>(n);
                give(tree_part<BLK, NQ>(t, b, n,
                                        (grp - b * t.bundles) * t.width +
                                            static_cast<int>(blockIdx.x) - grp * t.width,
                                        0, steps, steps));
            }
            TreePart none{};
            none.n = -1;
            if (ok) give(none);
        } else if (warp >= kTrCopyWarp) {
            // ----------------------------------------------------- copies
            constexpr int kUnits = DP / 8;         // 16-byte units of a row
            constexpr int kRows = BLK / 4;         // of a block, of this warp
            constexpr int kAtOnce = 32 / kUnits;   // rows an instruction copies
            const int cw = warp - kTrCopyWarp;
            // Rows r0 + kAtOnce x + lane / kUnits of a tile of ROWS rows, from
            // the addresses that lanes 0, 1, .. hold of them.
            auto copy_rows = [&](unsigned char* tile, int tile_rows, int r0, int count,
                                 const uint16_t* address, uint32_t there) {
                const int unit = lane % kUnits;
                const bool in_head = 8 * unit < t.d_head;
                const uint32_t at_unit = in_head ? 8 * unit : 0;
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
            // A lane's token of every block, its entry of the table and its
            // slot; looked up three blocks ahead: a table's entry takes a
            // microsecond to come when it is not in a cache.
            struct Place {
                int page, slot;   // slot -1: no token
            };
            const int32_t* table = nullptr;
            int tok = 0, len = 0, entry = 0, slot = 0;
            Place ahead[3];
            auto locate = [&]() {
                Place at{0, -1};
                if (tok < len) {
                    at.slot = slot;
                    at.page = table[entry];
                }
                tok += BLK;
                entry += t.skip;
                slot += t.rest;
                if (slot >= t.page_size) {
                    slot -= t.page_size;
                    ++entry;
                }
                return at;
            };
            auto begin = [&](const TreePart* p, int first) {
                table = t.page_table + p->b * t.table_stride;
                len = p->len;
                tok = p->key0 + first;
                entry = t.by_page(tok);
                slot = tok - entry * t.page_size;
#pragma unroll
                for (int x = 0; x < 3; ++x) ahead[x] = locate();
            };
            auto next_place = [&]() {
                const Place at = ahead[0];
                ahead[0] = ahead[1];
                ahead[1] = ahead[2];
                ahead[2] = locate();
                return at;
            };
            // A part's queries, by `warps` warps of which this is number w.
            int with_blocks = 0;
            auto load_q = [&](const TreePart* p, int w, int warps) {
                if (with_blocks > 0 && !warp_wait(q_empty, with_blocks - 1, limit)) return false;
                ++with_blocks;
#pragma unroll 1
                for (int r0 = 32 * w; r0 < 128 * NQ; r0 += 32 * warps) {
                    const int r = r0 + lane;
                    const int token = t.by_group(p->r0 + r);
                    const bool valid = r < p->valid;
                    const uint16_t* a = t.q;
                    if (valid)
                        a = t.q + p->b * t.q_stride[0] + token * t.q_stride[1] +
                            (p->hk * group + (p->r0 + r) - token * group) * t.q_stride[2];
                    copy_rows(smem + L::kQ + (r0 >> 7) * L::kTile, 128, r0 & 127, 32, a,
                              __ballot_sync(0xffffffffu, valid));
                }
                cp_async_arrive(q_full);
                return true;
            };
            // The same by tensor copies, a box of 128 rows each; into L2 before
            // the last part's products have left the room for them.
            auto fetch_q = [&](const TreePart* p) {
                const int head = p->hk * group, token = t.by_group(p->r0);
                auto each = [&](auto copy) {
#pragma unroll
                    for (int y = 0; y < NQ; ++y)
#pragma unroll
                        for (int x = 0; x < DP / 64; ++x)
                            copy(L::kQ + y * L::kTile + x * 128 * 128, 64 * x,
                                 token + y * t.by_group(128));
                };
                if (with_blocks > 0) {
                    if (lane == 0)
                        each([&](int, int x, int z) { tma_prefetch_4d(&map_q, x, head, z, p->b); });
                    __syncwarp();
                    if (!warp_wait(q_empty, with_blocks - 1, limit)) return false;
                }
                ++with_blocks;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, NQ * L::kTile);
                    each([&](int to, int x, int z) {
                        tma_load_4d(smem + to, &map_q, x, head, z, p->b, q_full);
                    });
                }
                __syncwarp();
                return true;
            };
            int block0 = 0;
            if (tensor_copies && cw >= 2) {
                // Two warps for the queries, or one thread where a tile's rows
                // are a box of whole tokens,
                for (int ip = 0;; ++ip) {
                    bool ok;
                    const TreePart* p = part(ip, ok);
                    if (!ok || p->n < 0) break;
                    if (p->n > 0) {
                        if (!t.tensor_q) ok = load_q(p, cw - 2, 2);
                        else if (cw == 2) ok = fetch_q(p);
                    }
                    if (!ok) break;
                    done_with(ip);
                }
                if (t.tensor_q && cw == 2 && *limit.abort_flag) {
                    for (int phase = 0; phase < 2; ++phase)
                        mbar_wait<false>(q_full, phase, t.wait_limit_cycles / 8);
                    __syncwarp();
                }
            } else if (tensor_copies) {
                // one for the keys and one for the values: a lane a box.
                const bool keys = cw == 0;
                const CUtensorMap* map = keys ? &map_k : &map_v;
                uint64_t* full = keys ? k_full : v_full;
                uint64_t* empty = keys ? k_empty : v_empty;
                unsigned char* ring = smem + (keys ? L::kK : L::kV);
                const int boxes = BLK >> t.box_bits;
                for (int ip = 0;; ++ip) {
                    bool ok;
                    const TreePart* p = part(ip, ok);
                    if (!ok || p->n < 0) break;
                    const int n = p->n, hk = p->hk;
                    if (n > 0) begin(p, (lane & (boxes - 1)) << t.box_bits);
                    done_with(ip);
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        const Place at = next_place();
                        const bool valid = at.page >= 0 && at.page < t.num_pages;
                        const int kb = block0 + j, st = kb % NS;
                        if (kb >= NS) ok = warp_wait(&empty[st], kb / NS - 1, limit);
                        if (!ok) break;
                        if (keys) {
                            // Boxes whose page is in the cache, and their tokens.
                            const bool lost = at.slot >= 0 && !valid;
                            const uint32_t good = __ballot_sync(0xffffffffu, !lost);
                            uint32_t bits = ~0u;
                            if (good != ~0u) bits = tree_lost(t, good);   // rare
                            if (lane < BLK / 32) words[4 * (kb % kTrWords) + lane] = bits;
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&full[st], L::kBlock);
                        __syncwarp();
                        if (lane < boxes) {
                            // (Outside the cache: zeros.)
                            const int page = at.slot >= 0 && valid ? at.page : t.num_pages;
                            unsigned char* dst = ring + st * L::kBlock + (lane << t.box_bits) * 128;
#pragma unroll
                            for (int x = 0; x < DP / 64; ++x)
                                tma_load_4d(dst + x * BLK * 128, map, 64 * x, hk,
                                            max(at.slot, 0), page, &full[st]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    block0 += n;
                }
                // None may land in shared memory after the CTA has ended.
                if (*limit.abort_flag) {
                    for (int st = 0; st < NS; ++st)
                        for (int phase = 0; phase < 2; ++phase)
                            mbar_wait<false>(&full[st], phase, t.wait_limit_cycles / 8);
                }
                __syncwarp();
            } else {
                for (int ip = 0;; ++ip) {
                    bool ok;
                    const TreePart* p = part(ip, ok);
                    if (!ok || p->n < 0) break;
                    const int n = p->n;
                    if (n > 0) begin(p, cw * kRows + lane % kRows);
                    const uint16_t* kbase = t.k_pages + p->hk * t.k_stride[2];
                    const uint16_t* vbase = t.v_pages + p->hk * t.v_stride[2];
#pragma unroll 1
                    for (int j = 0; j < n && ok; ++j) {
                        const Place at = next_place();
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
                        if (j == 0) ok = load_q(p, cw, 4);
                    }
                    if (!ok) break;
                    done_with(ip);
                    block0 += n;
                }
            }
            cp_async_wait_all();
        }
    }

    // Sequences without blocks in a dealt batch: zeros, by the CTAs in turn;
    // what is wrong with a length is reported here too.
    for (int b = t.split ? static_cast<int>(blockIdx.x) : grp / t.bundles; b < t.batch;
         b += t.split ? static_cast<int>(gridDim.x) : t.batch) {
        bool bad;
        const TreeLens n = tree_lens(t, b, bad);
        if (bad && threadIdx.x == 0) raise_error(t.err, kBitBadPage);
        if (t.split && tree_steps<BLK>(n) == 0) {
            const int units = t.d_head / 8;
#pragma unroll 1
            for (int64_t e = threadIdx.x;
                 e < static_cast<int64_t>(t.new_tokens) * t.heads * units; e += kTrThreads) {
                const int64_t row = e / units;
                const int i = static_cast<int>(row / t.heads);
                const int h = static_cast<int>(row - static_cast<int64_t>(i) * t.heads);
                const int d = 8 * static_cast<int>(e - row * units);
                *reinterpret_cast<uint4*>(tree_out(t, b, i, h) + d) = make_uint4(0u, 0u, 0u, 0u);
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
constexpr int kTrJoinFew = 2;    // CTAs an SM with C 2, up to which it is 1
constexpr int kTrJoinFull = 8;   // CTAs an SM with C 4, from which on it is 4

// Joins a unit's parts: a CTA takes 32 rows, a lane each, and 16 C columns, 4 C a
// thread.  A small batch has CTAs for every unit, a larger one for every place
// between two groups, where alone a unit can be cut, which join the unit that is
// cut there first (CUTS).  Bound by latency: eight loads of 16 bytes are under
// way in a thread, of eight parts where there are few CTAs (C 1: 131072 tokens in
// 19 parts, 91.5 us with the kernel before, with C 2 95, with 4 99), of four
// columns where there are enough (C 4: two prompts' chunks of 512 over 8192
// tokens, 2048 CTAs of 2 or 3 parts, 107.5, with C 2 110, with 1 120).  C 2 in
// between: 8 x 64 over 8192, 65.0, with 1 71, with 4 65.4.
template <int BLK, class E, bool CUTS, int C>
__global__ void __launch_bounds__(kTrJoinThreads) tree_join_kernel(const TreeTask t) {
    constexpr int kWarps = kTrJoinThreads / 32;
    __shared__ int scan[kWarps + 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = t.by_width(blockIdx.x), x = blockIdx.x - chunk * t.width;
    int b, bundle = 0, begin = 0, steps = 0, share = 1;
    bool bad, cut = true;
    if constexpr (!CUTS) {
        b = blockIdx.y / t.bundles;
        bundle = blockIdx.y - b * t.bundles;
        int before = 0, total = 0;
        for (int i = threadIdx.x; i < t.batch; i += kTrJoinThreads) {
            const int n = tree_places(tree_steps<BLK>(tree_lens(t, i, bad))) * t.bundles;
            total += n;
            if (i < b) before += n;
        }
        int skip, all;
        tree_scan<kWarps>(total, scan, skip, all);
        __syncthreads();
        share = max(1, t.by_groups(all + t.groups - 1));
        tree_scan<kWarps>(before, scan, skip, all);
        steps = tree_steps<BLK>(tree_lens(t, b, bad));
        begin = all + bundle * tree_places(steps) + kTreePartCost;
    } else {
        TreeDeal d;
        const int later = blockIdx.y + 1;
        cut = tree_deal<kWarps, BLK>(t, later, scan, d);
        if (cut) {
            b = d.b;
            share = d.share;
            steps = tree_steps<BLK>(tree_lens(t, b, bad));
            const int places = max(1, tree_places(steps));
            bundle = min((d.g0 - d.base) / places, t.bundles - 1);
            begin = d.base + bundle * places + kTreePartCost;
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
    const int col = C * (kWarps * (chunk / tiles) + warp);     // of 4 elements
    const int r_all = tile * t.unit_rows + r;
    if (4 * col >= t.d_head || r_all >= t.new_tokens * t.group || r >= t.unit_rows) return;
    // Part i: the first begins the unit (see TreePart).
    auto place = [&](int i) {
        return static_cast<int64_t>(2 * ((c0 + i) * t.width + x) + (i == 0)) * t.part_rows;
    };
    constexpr int kAtOnce = 8 / C;
    const int n = c1 - c0 + 1;
    float top = -INFINITY, sum = 0.0f;
    float acc[C][4] = {};
    for (int i0 = 0; i0 < n; i0 += kAtOnce) {
        float2 st[kAtOnce];
        float4 v[kAtOnce][C];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            st[k] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int y = 0; y < C; ++y) v[k][y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + k < n) {
                const int64_t at = place(i0 + k);
                st[k] = t.part_stats[at + r];
                const float4* w = reinterpret_cast<const float4*>(t.part_out + at * t.d_head) +
                                  col * t.part_rows + r;
#pragma unroll
                for (int y = 0; y < C; ++y)
                    if (4 * (col + y) < t.d_head) v[k][y] = w[y * t.part_rows];
            }
        }
        float m = top;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (st[k].y != 0.0f) m = fmaxf(m, st[k].x);
        const float f = top == -INFINITY ? 0.0f : ex2(top - m);
        sum *= f;
#pragma unroll
        for (int y = 0; y < C; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[y][e] *= f;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (st[k].y == 0.0f) continue;   // no kept tokens there
            const float g = ex2(st[k].x - m);
            sum = fmaf(st[k].y, g, sum);
#pragma unroll
            for (int y = 0; y < C; ++y) {
                acc[y][0] = fmaf(v[k][y].x, g, acc[y][0]);
                acc[y][1] = fmaf(v[k][y].y, g, acc[y][1]);
                acc[y][2] = fmaf(v[k][y].z, g, acc[y][2]);
                acc[y][3] = fmaf(v[k][y].w, g, acc[y][3]);
            }
        }
        top = m;
    }
    const int token = r_all / t.group, h = hk * t.group + r_all - token * t.group;
    uint16_t* to = tree_out(t, b, token, h) + 4 * col;
    const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
    if constexpr (C == 1) {
        *reinterpret_cast<uint2*>(to) = make_uint2(E::pack(acc[0][0] * inv, acc[0][1] * inv),
                                                    E::pack(acc[0][2] * inv, acc[0][3] * inv));
    } else {
#pragma unroll
        for (int y = 0; y < C; y += 2)
            if (4 * (col + y) < t.d_head)
                *reinterpret_cast<uint4*>(to + 4 * y) = make_uint4(
                    E::pack(acc[y][0] * inv, acc[y][1] * inv),
                    E::pack(acc[y][2] * inv, acc[y][3] * inv),
                    E::pack(acc[y + 1][0] * inv, acc[y + 1][1] * inv),
                    E::pack(acc[y + 1][2] * inv, acc[y + 1][3] * inv));
    }
    if (col == 0) tree_lse(t, b, token, h, top, sum);
}

template <int DP, int NQ, class E>
cudaError_t launch(TreeTask t, int slot, cudaStream_t stream) {
    using L = TreePlan<DP, NQ>;
    const auto kernel = tree_kernel<DP, NQ, E>;
    cudaError_t e = ensure_smem_attribute(reinterpret_cast<const void*>(kernel), slot, L::kBytes,
                                          false);
    if (e != cudaSuccess) return e;
    // Tensor copies take boxes of one page: the rows of the largest power of two
    // that divides the page and the block, 8 (a swizzled atom) at least.
    CUtensorMap map_k{}, map_v{}, map_q{};
    t.box_bits = 0;
    while ((t.page_size >> t.box_bits & 1) == 0 && (1 << t.box_bits) < L::kBlk) ++t.box_bits;
    if (t.box_bits < 3 || t.num_pages == 0 ||
        !encode_pages_map(&map_k, t.k_pages, t, t.k_stride, 1 << t.box_bits) ||
        !encode_pages_map(&map_v, t.v_pages, t, t.v_stride, 1 << t.box_bits))
        t.box_bits = -1;
    t.tensor_q = t.box_bits >= 0 && encode_queries_map(&map_q, t);
    t.skip = L::kBlk / t.page_size;
    t.rest = L::kBlk - t.skip * t.page_size;
    t.by_page = FastDiv(t.page_size);
    t.by_group = FastDiv(t.group);
    t.by_kv_heads = FastDiv(t.kv_heads);
    t.by_groups = FastDiv(t.groups);
    t.by_width = FastDiv(t.width);
    const int grid = (t.split ? t.groups : t.batch * t.bundles) * t.width;
    e = launch_shaped(kernel, {dim3(grid), kTrThreads, L::kBytes, stream, true, 1}, t, map_k,
                      map_v, map_q);
    if (e != cudaSuccess || !t.split || t.groups == 1) return e;
    const int64_t units = static_cast<int64_t>(t.batch) * t.bundles;
    const bool cuts = units >= t.groups;
    const unsigned joins = static_cast<unsigned>(cuts ? t.groups - 1 : units);
    const int sms = t.groups * t.width;
    auto ctas = [&](int c) {   // of a join
        return t.width * (t.part_rows / 32) * ((t.d_head + 16 * c - 1) / (16 * c));
    };
    auto join = [&](auto kernel, int c) {
        return launch_shaped(kernel, {dim3(ctas(c), joins), kTrJoinThreads, 0, stream, true, 1},
                             t);
    };
    if (static_cast<int64_t>(joins) * ctas(2) <= kTrJoinFew * sms)
        return join(cuts ? tree_join_kernel<L::kBlk, E, true, 1>
                         : tree_join_kernel<L::kBlk, E, false, 1>, 1);
    if (static_cast<int64_t>(joins) * ctas(4) >= kTrJoinFull * sms)
        return join(cuts ? tree_join_kernel<L::kBlk, E, true, 4>
                         : tree_join_kernel<L::kBlk, E, false, 4>, 4);
    return join(cuts ? tree_join_kernel<L::kBlk, E, true, 2>
                     : tree_join_kernel<L::kBlk, E, false, 2>, 2);
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
