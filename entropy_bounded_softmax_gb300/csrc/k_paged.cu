// Attention of one new token per sequence over a paged key-value cache.  For
// sequence b, query head h and its key head hk, over tokens j < lengths[b]
// (token j in slot j % page_size of page table[b][j / page_size]):
//   s_j = scale q . k_j,  out = sum e^(s_j - m) v_j / sum e^(s_j - m).
//
// Every key and value is read once for up to 16 query heads that share its
// head, and again for every 16 more: bound by the cache's bytes.  A sequence's
// tokens are steps of 64.
// The steps of the batch, one sequence after the other, are dealt to groups
// of CTAs in equal shares, so that a batch of any lengths keeps every SM
// streaming to the end.  A group has a CTA for every row, a key head's tile
// of up to 16 query heads: its CTAs walk the same pages at the same time,
// where the rows of all heads are neighbours (one sequence of 131072 tokens:
// 83 us so, 87 with each CTA on a stretch of its own).  A CTA takes its
// share's sequences one after the other.  Its four warps walk a part's tiles
// of 16 tokens, each with a ring of its own that asynchronous copies keep
// full (no barrier between warps until the part's end), a running maximum and
// sum, and two products on m16n8k16 tensor-core instructions with the query
// heads along M: scores = Q K^T and out += P V.  The instruction's rate does
// not matter here (a group of 16 heads or less leaves tcgen05's 128 rows
// empty, and the bytes take longer).  The warps' sums are joined in shared
// memory; a sequence that lies in one share is finished there, the others'
// parts (maximum, sum, unnormalised output) go to the workspace and a second
// small kernel, launched to overlap the first's end, joins them, with a CTA a
// head for every sequence or place where one can be cut.  Where no
// sequence can be longer than a few steps every CTA takes one whole row of one
// sequence, and there is no second kernel.
//
// Measured with 8 key heads of 128 in bf16: 83 us for 32 query heads of 131072
// tokens (6.5 TB/s of the cache, DRAM 83% busy), 39 us for 32 sequences of up
// to 4096 tokens (5.1 TB/s; the start of the copies, 5 us, and the join, 3,
// do not overlap with them), 4.3 us for a call of few tokens.
//
// The weights enter the second product as two halves of the cache's type,
// the nearest value and the nearest to the rest, so that their rounding
// (2^-16 in bf16) stays below the result's.  Their maximum may lag by 2^6.  In
// fp16, which has no exponents below 2^-24, they carry a factor 2^8: the largest
// weight, 2^8 to 2^14, leaves 2^-32 of it.  In bf16, whose values reach as far
// as fp32, they carry 2^-6 / n, n the tokens of a table's row, up to a power of
// two: the weights of any of them have a sum of at most 1, and no sum of weights
// and finite values overflows (with 2^8, values from about 2^114 on could).  (By
// each sequence's own tokens, the batch of 32 takes 39.3 us, and 38.7 so.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "cs_device.cuh"

namespace cs {
namespace {

using namespace csd;

constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgTile = 16;            // tokens
constexpr int kPgStep = kPgTile * kPgWarps;
constexpr int kPgStages = 3;
constexpr float kLagBits = 6.0f;       // how far the maximum may lag

__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The cache's element types: the tensor-core product and the two halves of a
// pair of weights.
struct PgBF16 {
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4],
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return make_float2(InBF16::lo(u), InBF16::hi(u));
    }
};

struct PgFP16 {
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4],
                                               uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 x = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
};

template <int DP>
struct PgSmem {
    static constexpr int kRow = DP * 2;                       // bytes of a token's row
    static constexpr int kHalf = kPgTile * kRow;              // a tile's keys, or values
    static constexpr int kWarp = kPgStages * 2 * kHalf;
    static constexpr int kRing = kPgWarps * kWarp;
    // At a part's end a warp's output, 16 rows of DP floats, takes exactly the
    // space of its ring's last stage, while the next part's first tiles land
    // in the others.
    static constexpr int kOut = (kPgStages - 1) * 2 * kHalf;
    static constexpr int kStats = kRing;                      // [warps][16] float2
    // [warps][2][16]: where a tile's tokens have their keys and values.
    static constexpr int kRows = kStats + kPgWarps * 16 * 8;
    static constexpr int kScan = kRows + kPgWarps * 2 * 16 * 16;     // [kPgWarps + 4]
    static constexpr int kBytes = kScan + (kPgWarps + 4) * 4;
    static_assert(16 * DP * 4 <= 2 * kHalf, "an output fits a stage");
};

// A sequence's length, and whether it is one the table can hold.
__device__ __forceinline__ int length_of(const PagedTask& t, int b, bool& bad) {
    const int n = t.lengths[b];
    const int most = t.max_pages * t.page_size;
    bad = n < 0 || n > most;
    return n < 0 ? 0 : min(n, most);
}

// Writes elements d .. d + 7 of one head's output, and with d = 0 its lse,
// from what the weights are relative to (2^(score - top)), their joined sum and
// the unnormalised output.
template <class T>
__device__ __forceinline__ void paged_finish(const PagedTask& t, int b, int h, int d,
                                             const float (&acc)[8], float top, float sum) {
    if (d < t.d_head) {
        const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);
        uint4 w;
        w.x = T::pack(acc[0] * inv, acc[1] * inv);
        w.y = T::pack(acc[2] * inv, acc[3] * inv);
        w.z = T::pack(acc[4] * inv, acc[5] * inv);
        w.w = T::pack(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(t.out + b * t.o_stride[0] + h * t.o_stride[1] + d) = w;
    }
    if (d == 0) {
        if (t.lse)
            t.lse[static_cast<int64_t>(b) * t.heads + h] =
                sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        if (!isfinite(sum)) raise_error(t.err, kBitNan);
    }
}

__device__ __forceinline__ int steps_of(int len) { return (len + kPgStep - 1) / kPgStep; }

// The steps of the sequences before `upto`, by the whole CTA; scan: kPgWarps
// shared ints.
__device__ __forceinline__ int steps_before(const PagedTask& t, int upto, int* scan) {
    int n = 0;
    bool bad;
    for (int b = threadIdx.x; b < upto; b += kPgThreads) n += steps_of(length_of(t, b, bad));
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) scan[threadIdx.x >> 5] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) n += scan[w];
    __syncthreads();
    return n;
}

// Steps of a group's share.
__device__ __forceinline__ int share_of(const PagedTask& t, int total) {
    const int n = (total + t.groups - 1) / t.groups;
    return n > 0 ? n : 1;
}

// The sum of n over the threads before this one and over all of the CTA; scan:
// kPgWarps shared ints, free again after the caller's next __syncthreads.
__device__ __forceinline__ void block_scan(int n, int* scan, int& before, int& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int up = n;   // inclusive sum of the warp
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
    for (int w = 0; w < kPgWarps; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
    }
}

// A group's steps g0 .. g1 - 1 of the batch's, the sequence that holds g0 and
// its first step, by a whole CTA; false without steps.  scan: kPgWarps + 2
// shared ints.
__device__ __forceinline__ bool deal(const PagedTask& t, int grp, int* scan, int& g0, int& g1,
                                     int& b, int& base) {
    const bool once = t.batch <= kPgThreads;   // one walk over the lengths is enough
    int total = once ? 0 : steps_before(t, t.batch, scan);
    int done = 0;
    for (int b0 = 0; b0 < t.batch; b0 += kPgThreads) {
        const int i = b0 + threadIdx.x;
        bool bad;
        const int n = i < t.batch ? steps_of(length_of(t, i, bad)) : 0;
        int first, all;
        block_scan(n, scan, first, all);
        if (once) total = all;
        const int share = share_of(t, total);
        g0 = grp * share;
        g1 = min(total, g0 + share);
        if (g0 >= g1) return false;
        first += done;
        if (first <= g0 && g0 < first + n) {
            scan[kPgWarps] = i;
            scan[kPgWarps + 1] = first;
        }
        done += all;
        __syncthreads();
        if (done > g0) break;
    }
    // (In range even where the lengths were changed under the call: what it
    // returns is then wrong, but no walk leaves the batch.)
    b = max(0, min(scan[kPgWarps], t.batch - 1));
    base = min(scan[kPgWarps + 1], g0);
    return true;
}

// Tokens t0 .. t1 - 1 of sequence b: all of them, or part `place` of the
// workspace.
struct Part {
    int b, t0, t1;
    bool whole;
    int place;
};

// CTAs an SM: what the rings' shared memory allows.
template <int DP, class T>
__global__ void __launch_bounds__(kPgThreads, DP == 64 ? 4 : DP == 128 ? 2 : 1)
paged_kernel(const PagedTask t) {
    using L = PgSmem<DP>;
    extern __shared__ __align__(128) unsigned char smem[];
    allow_next_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const int rows = t.kv_heads * t.head_tiles;   // of a sequence
    const int grp = cta / rows, row = cta - grp * rows;
    const int hk = row / t.head_tiles, ht = row - hk * t.head_tiles;
    const int group = t.heads / t.kv_heads;
    const int h0 = hk * group + 16 * ht;          // first query head
    const int nh = min(16, group - 16 * ht);      // query heads here
    bool bad;

    // The walk over this CTA's parts: step g of g0 .. g1 - 1, in sequence b
    // whose first step is base.
    int g = 0, g0 = 0, g1 = 1, b = grp, base = 0;
    bool any = true;
    if (t.split) any = deal(t, grp, reinterpret_cast<int*>(smem + L::kScan), g0, g1, b, base);
    int len = any ? length_of(t, b, bad) : 0, steps = steps_of(len);
    g = g0;
    auto next = [&](Part& p) {
        if (!any || g >= g1) return false;
        int s0 = 0, s1 = steps;
        if (t.split) {
            while (g >= base + steps) {   // (sequences without tokens too)
                if (b + 1 >= t.batch) return false;
                base += steps;
                len = length_of(t, ++b, bad);
                steps = steps_of(len);
            }
            s0 = g - base;
            s1 = min(steps, s0 + g1 - g);
        }
        p.b = b;
        p.t0 = s0 * kPgStep;
        p.t1 = min(len, s1 * kPgStep);
        p.whole = s0 == 0 && s1 == steps;
        p.place = 2 * cta + (g > g0);
        g += t.split ? s1 - s0 : 1;
        return true;
    };

    unsigned char* ring = smem + warp * L::kWarp;
    ulonglong2* rows_of = reinterpret_cast<ulonglong2*>(smem + L::kRows) + warp * 2 * 16;
    // A part's tiles that are this warp's.
    auto tiles_of = [&](const Part& p) {
        const int tiles = (p.t1 - p.t0 + kPgTile - 1) / kPgTile;
        return tiles > warp ? (tiles - warp + kPgWarps - 1) / kPgWarps : 0;
    };
    // A tile's way, in this warp (lanes 16 to 31 as the 16 before): its tokens'
    // pages are looked up (locate), a table's entry takes a microsecond to come
    // when it is not in a cache; the addresses of their rows are left in shared
    // memory (aim) an iteration later; its copies start (issue) in the next,
    // and two iterations later it is used.  Every lane working out the
    // addresses that it copies from took 980 cycles of a tile's 2000.
    struct Place {
        int page, slot;   // slot -1: no token
    };
    // The next token to look up, its entry of the table and its slot.
    int tok = 0, entry = 0, slot = 0;
    const int skip = kPgStep / t.page_size, rest = kPgStep - skip * t.page_size;
    auto locate = [&](const Part& p) {
        Place at{0, -1};
        if (tok < p.t1) {
            at.slot = slot;
            at.page = t.page_table[p.b * t.table_stride + entry];
        }
        tok += kPgStep;
        entry += skip;
        slot += rest;
        if (slot >= t.page_size) {
            slot -= t.page_size;
            ++entry;
        }
        return at;
    };
    constexpr int kUnits = DP / 8;     // 16-byte units of a row
    const uint16_t* kbase = t.k_pages + hk * t.k_stride[2];
    const uint16_t* vbase = t.v_pages + hk * t.v_stride[2];
    // Leaves the rows' addresses in table `buf`; the tokens that are there, one
    // bit each.  (A __syncwarp before the copies.)
    auto aim = [&](const Place& where, int buf) {
        const bool valid = where.slot >= 0 && where.page >= 0 && where.page < t.num_pages;
        if (where.slot >= 0 && !valid) raise_error(t.err, kBitBadPage);
        const uint16_t *k = t.q, *v = t.q;
        if (valid) {
            k = kbase + where.page * t.k_stride[0] + where.slot * t.k_stride[1];
            v = vbase + where.page * t.v_stride[0] + where.slot * t.v_stride[1];
        }
        if (lane < 16)
            rows_of[16 * buf + lane] = make_ulonglong2(reinterpret_cast<uintptr_t>(k),
                                                       reinterpret_cast<uintptr_t>(v));
        return __ballot_sync(0xffffffffu, valid) & 0xffffu;
    };
    // Starts a tile's copies into stage st: 32 / kUnits rows at a time; zeros
    // past d_head and for tokens that are not there.
    const int unit = lane % kUnits;
    const bool in_head = 8 * unit < t.d_head;
    const uint32_t at_unit = in_head ? 16 * unit : 0;
    auto issue = [&](uint32_t there, int buf, int st) {
        unsigned char* dk = ring + st * 2 * L::kHalf;
        unsigned char* dv = dk + L::kHalf;
#pragma unroll
        for (int n = 0; n < kPgTile * kUnits / 32; ++n) {
            const int r = n * (32 / kUnits) + lane / kUnits;
            const ulonglong2 row = rows_of[16 * buf + r];
            const uint32_t bytes = in_head && (there >> r & 1u) ? 16u : 0u;
            const int at = r * L::kRow + ((unit ^ (r & 7)) << 4);
            cp_async16_zfill(dk + at, reinterpret_cast<const void*>(row.x + at_unit), bytes);
            cp_async16_zfill(dv + at, reinterpret_cast<const void*>(row.y + at_unit), bytes);
        }
    };

    // A part's first tiles.  From then on, before tile i: its tokens that are
    // there in here0, the next tile's in here1, and those of tile i + 2, aimed
    // in table i % 2, in here2; tile i + 3 is `soon`.
    uint32_t here0 = 0, here1 = 0, here2 = 0;
    Place soon{0, -1};
    auto begin = [&](const Part& p) {
        static_assert(kPgStages == 3, "two tiles under way");
        const int mine = tiles_of(p);
        tok = p.t0 + warp * kPgTile + (lane & 15);
        entry = tok / t.page_size;
        slot = tok - entry * t.page_size;
        const Place first = locate(p), second = locate(p), third = locate(p);
        soon = locate(p);
        here0 = aim(first, 0);
        here1 = aim(second, 1);
        __syncwarp();
        if (mine > 0) issue(here0, 0, 0);
        cp_async_commit();
        if (mine > 1) issue(here1, 1, 1);
        cp_async_commit();
        __syncwarp();
        here2 = aim(third, 0);
    };
    // Unit n (8 floats) of row r of warp w's output, at the end of a part:
    // units permuted within a row by its number, so that the rows' stores
    // fall in different banks.
    auto out_of = [&](int w, int r, int n) {
        return reinterpret_cast<float4*>(smem + w * L::kWarp + L::kOut + r * DP * 4 +
                                         ((n ^ (r & 7)) << 5));
    };
    float2* stats = reinterpret_cast<float2*>(smem + L::kStats);

    Part now, then;
    bool more = next(now);
    if (more) begin(now);
    while (more) {
        const int mine = tiles_of(now);
        // Query fragments: rows lane / 4 and lane / 4 + 8, columns 2 (lane % 4)
        // and 8 more of each 16.
        const int gr = lane >> 2, c2 = 2 * (lane & 3);
        uint32_t q[DP / 16][4];
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = gr + 8 * (i & 1), col = 16 * ks + c2 + 8 * (i >> 1);
                q[ks][i] = 0u;
                if (row < nh && col < t.d_head)
                    q[ks][i] = *reinterpret_cast<const uint32_t*>(
                        t.q + now.b * t.q_stride[0] + (h0 + row) * t.q_stride[1] + col);
            }

        const float c = t.scale * kLog2e;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        float o[DP / 8][4];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;

        const int mat = lane >> 3, r8 = lane & 7;
        for (int i = 0; i < mine; ++i) {
            const int st = i % kPgStages;
            cp_async_wait_group<kPgStages - 2>();
            __syncwarp();
            // Stage (i - 1) % kPgStages was read before the __syncwarp.
            if (i + kPgStages - 1 < mine) issue(here2, i & 1, (i + kPgStages - 1) % kPgStages);
            cp_async_commit();
            const Place later = locate(now);

            const uint32_t sk = smem_addr(ring + st * 2 * L::kHalf), sv = sk + L::kHalf;
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            {
                const int row = (mat >> 1) * 8 + r8;
    #pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    uint32_t k[4];
                    ldmatrix4(k, sk + row * L::kRow + (((2 * ks + (mat & 1)) ^ r8) << 4));
                    T::mma(s[0], q[ks], k[0], k[1]);
                    T::mma(s[1], q[ks], k[2], k[3]);
                }
            }
            const uint32_t here = here0;
    #pragma unroll
            for (int n = 0; n < 2; ++n)
    #pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = 8 * n + c2 + (k & 1);
                    s[n][k] = (here >> tok) & 1u ? s[n][k] * c : -INFINITY;
                }
            float top[2];
    #pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]),
                               fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                top[r] = fmaxf(top[r], m[r]);
            }
            // m = -inf and a finite top: an infinite difference, above the lag.
            if (__any_sync(0xffffffffu, top[0] - m[0] > kLagBits || top[1] - m[1] > kLagBits)) {
    #pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = m[r] == -INFINITY ? 0.0f : ex2(m[r] - top[r]);
                    m[r] = top[r];
                    l[r] *= f;
    #pragma unroll
                    for (int n = 0; n < DP / 8; ++n) {
                        o[n][2 * r] *= f;
                        o[n][2 * r + 1] *= f;
                    }
                }
            }
            float p[2][4];
    #pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float base = m[r] == -INFINITY ? 0.0f : m[r] - t.weight_bits;
    #pragma unroll
                for (int n = 0; n < 2; ++n)
    #pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        p[n][2 * r + k] = ex2(s[n][2 * r + k] - base);
                        l[r] += p[n][2 * r + k];
                    }
            }
            uint32_t hi[4], lo[4];
    #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = p[k >> 1][2 * (k & 1)], z = p[k >> 1][2 * (k & 1) + 1];
                hi[k] = T::pack(a, z);
                const float2 w = T::unpack(hi[k]);
                lo[k] = T::pack(a - w.x, z - w.y);
            }
            {
                const int row = (mat & 1) * 8 + r8;
    #pragma unroll
                for (int n2 = 0; n2 < DP / 16; ++n2) {
                    uint32_t v[4];
                    ldmatrix4_trans(v, sv + row * L::kRow + (((2 * n2 + (mat >> 1)) ^ r8) << 4));
                    T::mma(o[2 * n2], hi, v[0], v[1]);
                    T::mma(o[2 * n2], lo, v[0], v[1]);
                    T::mma(o[2 * n2 + 1], hi, v[2], v[3]);
                    T::mma(o[2 * n2 + 1], lo, v[2], v[3]);
                }
            }
            // (Table (i + 1) % 2 was read before this iteration's __syncwarp.)
            here0 = here1;
            here1 = here2;
            here2 = aim(soon, (i + 1) & 1);
            soon = later;
        }

        // The next part's first tiles come while this one's warps are joined.
        __syncwarp();
        more = next(then);
        if (more) begin(then);

        // Join the warps: rows gr and gr + 8 of each, the row's sum over its
        // four lanes first.
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            const int row = gr + 8 * r;
            if ((lane & 3) == 0) stats[warp * 16 + row] = make_float2(m[r] - t.weight_bits, l[r]);
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
                reinterpret_cast<float2*>(out_of(warp, row, n))[lane & 3] =
                    make_float2(o[n][2 * r], o[n][2 * r + 1]);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < nh * (DP / 8); e += kPgThreads) {
            const int row = e / (DP / 8), d = 8 * (e % (DP / 8));
            float top = -INFINITY;
    #pragma unroll
            for (int w = 0; w < kPgWarps; ++w) top = fmaxf(top, stats[w * 16 + row].x);
            float sum = 0.0f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    #pragma unroll
            for (int w = 0; w < kPgWarps; ++w) {
                const float2 st = stats[w * 16 + row];
                const float f = st.x == -INFINITY ? 0.0f : ex2(st.x - top);
                sum = fmaf(st.y, f, sum);
                const float4* a = out_of(w, row, d >> 3);
                const float4 a0 = a[0], a1 = a[1];
                const float v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    #pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = fmaf(v[k], f, acc[k]);
            }
            if (now.whole) {
                paged_finish<T>(t, now.b, h0 + row, d, acc, top, sum);
            } else {
                const int64_t at = static_cast<int64_t>(now.place) * 16 + row;
                if (d == 0) t.part_stats[at] = make_float2(top, sum);
                if (d < t.d_head) {
                    float4* w = reinterpret_cast<float4*>(t.part_out + at * t.d_head + d);
                    w[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    w[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                }
            }
        }
        __syncthreads();   // the next part's later tiles take the outputs' space
        now = then;
    }
    cp_async_wait_all();

    // Sequences without tokens have no steps: their rows are zeros, written
    // by the CTAs in turn; so is what is wrong with a length reported.
    for (int i = t.split ? cta : grp; i < t.batch; i += gridDim.x) {
        const int n = length_of(t, i, bad);
        if (bad && threadIdx.x == 0) raise_error(t.err, kBitBadPage);
        if (n == 0 && t.split) {
            const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int e = threadIdx.x; e < t.heads * (DP / 8); e += kPgThreads)
                paged_finish<T>(t, i, e / (DP / 8), 8 * (e % (DP / 8)), zero, 0.0f, 0.0f);
        }
    }
}

// Joins a sequence's parts, one CTA a head: every warp takes the largest
// maximum and the sum over all parts, then the CTA's threads, DP / 8 of them to
// a part, add the parts' outputs.  Launched while the parts are still computed
// (it waits for them here), so that its start costs nothing.  Only the places
// between two groups can cut a sequence: a batch of fewer sequences than groups
// has a CTA for every sequence, a larger one a CTA for every such place, which
// joins the sequence that is cut there first, so that what the launch takes
// grows with the batch and not with its square (32768 sequences of up to 32
// tokens, 8 heads of 64 on one key head: 1015 us, with a CTA for every sequence
// 7368; 4096 sequences: 124 and 172).  CUTS: the latter (an instance of its own:
// in one kernel with a branch 7 sequences of up to 1531 tokens took 1% longer).
template <int DP, class T, bool CUTS>
__global__ void __launch_bounds__(kPgThreads)
paged_join_kernel(const PagedTask t) {
    constexpr int kUnits = DP / 8, kRows = kPgThreads / kUnits;
    __shared__ float part[kRows][DP + 4];
    __shared__ int scan[kPgWarps + 2];
    const int h = blockIdx.x;
    int b = blockIdx.y, begin = 0, share = 1;
    bool bad, cut = true;
    if constexpr (!CUTS) {
        share = share_of(t, steps_before(t, t.batch, scan));
        begin = steps_before(t, b, scan);
    } else {
        // The place before group `later`: its first step, and whose it is.
        const int later = blockIdx.y + 1;
        int g0 = 0, g1;
        cut = deal(t, later, scan, g0, g1, b, begin);
        if (cut) {
            share = g0 / later;
            cut = begin < g0 && begin / share == later - 1;
        }
    }
    const int steps = cut ? steps_of(length_of(t, b, bad)) : 0;
    const int c0 = begin / share, c1 = min((begin + steps - 1) / share, t.groups - 1);
    wait_for_previous_kernel();
    // Not cut (here first), without steps, or finished by the only group that
    // had it.
    if (steps == 0 || c0 >= c1) return;
    const int group = t.heads / t.kv_heads;
    const int hk = h / group, hh = h - hk * group;
    const int rows = t.kv_heads * t.head_tiles, row = hk * t.head_tiles + hh / 16;
    const int n = c1 - c0 + 1;
    // Part i: group c0 + i's first, but group c0's last where it had others
    // before.
    const int late = begin > c0 * share ? 1 : 0;
    auto place = [&](int i) {
        return static_cast<int64_t>(2 * ((c0 + i) * rows + row) + (i == 0 ? late : 0)) * 16 +
               hh % 16;
    };
    // The first outputs of this thread come while the maximum is taken.
    const int line = threadIdx.x / kUnits, d = 8 * (threadIdx.x % kUnits);
    auto output = [&](int i) {
        return reinterpret_cast<const float4*>(t.part_out + place(i) * t.d_head + d);
    };
    const bool any = d < t.d_head && line < n;
    float4 first0 = make_float4(0.f, 0.f, 0.f, 0.f), first1 = first0;
    float x0 = -INFINITY;
    if (any) {
        first0 = output(line)[0];
        first1 = output(line)[1];
        x0 = t.part_stats[place(line)].x;
    }
    const int lane = threadIdx.x & 31;
    float top = -INFINITY, sum = 0.0f;
    for (int i0 = lane; i0 < n; i0 += 4 * 32) {
        float2 st[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 32 * u;
            st[u] = i < n ? t.part_stats[place(i)] : make_float2(-INFINITY, 0.0f);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float m = fmaxf(top, st[u].x);
            // (Both maxima -inf: nothing to rescale.)
            const float f = top == -INFINITY ? 0.0f : ex2(top - m);
            const float g = st[u].x == -INFINITY ? 0.0f : ex2(st[u].x - m);
            sum = fmaf(sum, f, st[u].y * g);
            top = m;
        }
    }
    const float mine = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    sum = mine == -INFINITY ? sum : sum * ex2(mine - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](float x, const float4& a0, const float4& a1) {
        const float f = x == -INFINITY ? 0.0f : ex2(x - top);
        const float v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(v[k], f, acc[k]);
    };
    if (any) {
        add(x0, first0, first1);
        // (Four at a time, all loads first; the last ones too.)
        for (int i0 = line + kRows; i0 < n; i0 += 4 * kRows) {
            float x[4];
            float4 a0[4], a1[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * kRows;
                x[u] = -INFINITY;
                a0[u] = a1[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    x[u] = t.part_stats[place(i)].x;
                    a0[u] = output(i)[0];
                    a1[u] = output(i)[1];
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) add(x[u], a0[u], a1[u]);
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) part[line][d + k] = acc[k];
    __syncthreads();
    if (threadIdx.x >= kUnits) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        acc[k] = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[k] += part[r][d + k];
    }
    paged_finish<T>(t, b, h, d, acc, top, sum);
}

template <int DP, class T>
cudaError_t launch(PagedTask t, int slot, cudaStream_t stream) {
    t.weight_bits = 8.0f;
    if (!t.fp16) {
        t.weight_bits = -kLagBits;
        const int64_t most = static_cast<int64_t>(t.max_pages) * t.page_size;
        for (int64_t n = 1; n < most; n <<= 1) t.weight_bits -= 1.0f;
    }
    const void* kern = reinterpret_cast<const void*>(paged_kernel<DP, T>);
    cudaError_t e = ensure_smem_attribute(kern, slot, PgSmem<DP>::kBytes, false);
    if (e != cudaSuccess) return e;
    const int grid = (t.split ? t.groups : t.batch) * t.kv_heads * t.head_tiles;
    paged_kernel<DP, T><<<grid, kPgThreads, PgSmem<DP>::kBytes, stream>>>(t);
    e = cudaGetLastError();
    if (e != cudaSuccess || !t.split) return e;
    if (t.groups == 1) return cudaSuccess;   // one share: nothing is cut
    const bool cuts = t.batch >= t.groups;
    return launch_shaped(cuts ? paged_join_kernel<DP, T, true> : paged_join_kernel<DP, T, false>,
                         {dim3(t.heads, cuts ? t.groups - 1 : t.batch), kPgThreads, 0, stream,
                          true, 1},
                         t);
}

template <class T>
cudaError_t launch_type(const PagedTask& t, int slot, cudaStream_t stream) {
    if (t.d_head <= 64) return launch<64, T>(t, slot, stream);
    if (t.d_head <= 128) return launch<128, T>(t, slot + 1, stream);
    return launch<256, T>(t, slot + 2, stream);
}

}  // namespace

cudaError_t launch_paged(const PagedTask& task, cudaStream_t stream) {
    return task.fp16 ? launch_type<PgFP16>(task, 62, stream)
                     : launch_type<PgBF16>(task, 65, stream);
}

}  // namespace cs
