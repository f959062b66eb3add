// Fused attention, forward.  For every query row i of a head:
//   s_j = scale q_i . k_j over the kept keys, m = max s_j,
//   l = sum e^(s_j - m), out_i = sum e^(s_j - m) v_j / l, lse_i = m + ln l,
// in one pass over the keys with the running m and l of a softmax: the
// scores never leave the SM.
//
// A CTA takes 256 query rows of one head as two tiles of 128 and walks the
// keys in blocks of 128.  Tensor memory holds both tiles' scores (128
// columns each) and outputs (DP columns each); a tile's weights overwrite
// its scores as bf16 and are the next product's A operand there.  Roles, one
// mbarrier hand-off each:
//   warps 0-3, 4-7  softmax of tile 0 and 1, one row a thread: the row's 128
//                   scores to registers, the maximum, 2^(s c - m c) and the
//                   sum, the weights back to tensor memory;
//   warp 8          issues the products: for each block and tile P V, then
//                   the next block's Q K^T into the columns P V has read, so
//                   that one tile's products run under the other's softmax;
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

constexpr int kFwdThreads = 384;
// Registers a thread: 168 at launch; the softmax warps, whose row of scores is
// 128 of them, take what the others give up: 256 x 208 + 128 x 72 <= 384 x 168.
constexpr int kFwdRegsSoftmax = 208;
constexpr int kFwdRegsOther = 72;
constexpr int kFwdMmaWarp = 8;
constexpr int kFwdLoadWarp = 9;
constexpr int kFwdMaskWarp = 10;
constexpr uint32_t kFwdTmemCols = 512;
constexpr float kRescaleBits = 8.0f;

template <int DP>
struct FwdSmem {
    static constexpr int kTile = 128 * DP * 2;
    static constexpr int kStages = DP == 64 ? 3 : 2;      // of K and of V
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kBars = kV + kStages * kTile;
    static constexpr int kNumBars = 2 + 5 * kStages + 2 + 2 + 2 + 1;
    static constexpr int kWords = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [kStages][4]
    static constexpr int kFlags = kWords + kStages * 16;  // abort, tmem, lo, hi
    static constexpr int kBytes = kFlags + 16 + 1024;     // and alignment slack
};

// D[128 x DP] (+)= P[128 x R] . B[R x DP], P bf16 in tensor memory, B a tile.
template <int R, int DP>
__device__ __forceinline__ void mma_weights(uint32_t d, uint32_t p, uint32_t b,
                                            bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16(128, DP, true);
#pragma unroll
    for (int ks = 0; ks < R / 16; ++ks)
        mma_bf16_ts(d, p + 8 * ks, smem_desc_mn_sw128(b + ks * 2048, R * 128, 1024), idesc,
                    accumulate || ks > 0);
}

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
fattn_fwd_kernel(const FattnTask t, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
    using L = FwdSmem<DP>;
    constexpr int NS = L::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* q_full = bars;                  // [2] tile's queries landed
    uint64_t* k_full = q_full + 2;            // [NS] ring stage landed
    uint64_t* k_empty = k_full + NS;          // [NS] products that read it completed
    uint64_t* v_full = k_empty + NS;
    uint64_t* v_empty = v_full + NS;
    uint64_t* v_masked = v_empty + NS;        // [NS] removed rows zeroed, bits written
    uint64_t* s_full = v_masked + NS;         // [2] tile's scores of a block
    uint64_t* p_full = s_full + 2;            // [2] tile's weights of a block
    uint64_t* o_full = p_full + 2;            // [2] the block's P V completed
    uint64_t* drained = o_full + 2;
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::kWords);
    volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + L::kFlags);
    const WaitLimit limit{flags, t.wait_limit_cycles};

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int BH = t.batch * t.heads;
    const int q_tiles = (t.query_len + 255) / 256;
    // Under the causal mask later rows keep more keys: longest first.
    const int qt = t.causal ? q_tiles - 1 - static_cast<int>(blockIdx.x / BH)
                            : static_cast<int>(blockIdx.x / BH);
    const int bh = static_cast<int>(blockIdx.x % BH);
    const int b = bh / t.heads, h = bh - b * t.heads;
    const int hk = h / (t.heads / t.kv_heads);
    const int q0 = 256 * qt;
    const int off = t.key_len - t.query_len;   // row i keeps keys j <= i + off

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1u);
            mbar_init(&s_full[i], 1u);
            mbar_init(&p_full[i], 4u);
            mbar_init(&o_full[i], 1u);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&k_full[i], 1u);
            mbar_init(&k_empty[i], 1u);
            mbar_init(&v_full[i], 1u);
            mbar_init(&v_empty[i], 1u);
            mbar_init(&v_masked[i], 1u);
        }
        mbar_init(drained, 1u);
        flags[0] = 0u;
        fence_mbar_init();
    }
    if (warp == kFwdMmaWarp)
        tmem_alloc(const_cast<uint32_t*>(flags) + 1, kFwdTmemCols);
    const uint8_t* mask = t.mask ? t.mask + b * t.mask_stride : nullptr;
    int key_lo = 0, key_hi = t.key_len;
    if (mask)
        block_nonzero_range(mask, t.key_len,
                            reinterpret_cast<int*>(smem + L::kFlags) + 2, key_lo, key_hi);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = flags[1];

    // Blocks j0, j0 + 1, ..: n[i] of them for tile i, none for a tile without
    // rows or without kept keys.
    const int j0 = key_lo >> 7;
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int last = min(q0 + 128 * (i + 1), t.query_len) - 1;
        const int hi = t.causal ? min(key_hi, last + off + 1) : key_hi;
        n[i] = last >= q0 + 128 * i && hi > key_lo ? ((hi + 127) >> 7) - j0 : 0;
    }
    const int blocks = max(n[0], n[1]);

    if (warp < 8) {
        // -------------------------------------------------------- softmax
        take_registers<kFwdRegsSoftmax>();
        const int tile = warp >> 2;
        const int row0 = q0 + 128 * tile + 32 * (warp & 3);
        const int i = row0 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * tile;
        const uint32_t to = tmem + lanes + 256 + DP * tile;
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
            uint32_t s[128];
#pragma unroll
            for (int u = 0; u < 4; ++u) tmem_ld32_async(ts + 32 * u, s + 32 * u);
            tmem_wait_ld<128>(s);
            const int key = (j0 + j) << 7;
            uint4 kept = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (mask) kept = *reinterpret_cast<const uint4*>(words + 4 * (j % NS));
            if (warp_limit < key + 128 || (kept.x & kept.y & kept.z & kept.w) != ~0u) {
                const uint32_t bits[4] = {kept.x & bits_below(row_limit, key),
                                          kept.y & bits_below(row_limit, key + 32),
                                          kept.z & bits_below(row_limit, key + 64),
                                          kept.w & bits_below(row_limit, key + 96)};
#pragma unroll
                for (int k = 0; k < 128; ++k)
                    if (!((bits[k >> 5] >> (k & 31)) & 1u)) s[k] = __float_as_uint(-INFINITY);
            }
            float mx[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(s[k]);
#pragma unroll
            for (int k = 4; k < 128; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(s[k]));
            const float top = fmaxf(fmaxf(m, fmaxf(mx[0], mx[1])), fmaxf(mx[2], mx[3]));
            if (j == 0) {
                m = top;
            } else if (__any_sync(0xffffffffu, (top - m) * c > kRescaleBits)) {
                const float f = m == -INFINITY ? 0.0f : ex2((m - top) * c);
                m = top;
                l *= f;
                ok = warp_wait(&o_full[tile], j - 1, limit);
                if (!ok) break;
                tc_fence_after_sync();
#pragma unroll
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
            for (int k = 0; k < 64; ++k) {
                const float2 y = fma2(make_float2(__uint_as_float(s[2 * k]),
                                                  __uint_as_float(s[2 * k + 1])), c2, mc2);
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                sum[k & 1] = add2(sum[k & 1], e);
                s[k] = pack_bf16(e.x, e.y);
            }
            tmem_st32(ts, s);
            tmem_st32(ts + 32, s + 32);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[tile]);
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
        }
        if (ok && nt > 0) ok = warp_wait(&o_full[tile], nt - 1, limit);
        if (ok) {
            tc_fence_after_sync();
            const bool live = i < t.query_len;
            const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
            uint16_t* row = t.out + b * t.o_stride[0] + h * t.o_stride[1] + i * t.o_stride[2];
#pragma unroll
            for (int u = 0; u < DP / 32; ++u) {
                uint32_t o[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
                if (nt > 0) {
                    tmem_ld32_async(to + 32 * u, o);
                    tmem_wait_ld<32>(o);
                }
                if (live) store_row32(row, t.d_head, 32 * u, o, inv);
            }
            if (live && t.lse)
                t.lse[static_cast<int64_t>(bh) * t.query_len + i] =
                    l == 0.0f ? -INFINITY : (m * c + log2f(l)) * kLn2;
            if (live && !isfinite(l)) raise_error(t.err, kBitNan);
        }
    } else if (give_registers<kFwdRegsOther>(); warp == kFwdMmaWarp) {
        // ----------------------------------------------------- MMA issuer
        const uint32_t q = smem_addr(smem + L::kQ);
        const uint32_t k = smem_addr(smem + L::kK);
        const uint32_t v = smem_addr(smem + L::kV);
        auto scores = [&](int i, int j) {
            if (lane == 0) {
                mma_tiles<128, DP>(tmem + 128 * i, q + i * L::kTile, k + (j % NS) * L::kTile);
                mma_commit(&s_full[i]);
            }
        };
        bool ok = true;
        if (blocks > 0) {
            ok = warp_wait(&k_full[0], 0, limit);
            for (int i = 0; i < 2 && ok; ++i) {
                if (n[i] == 0) continue;
                ok = warp_wait(&q_full[i], 0, limit);
                if (ok) scores(i, 0);
            }
            if (ok && lane == 0) mma_commit(&k_empty[0]);
            __syncwarp();
        }
        uint64_t* v_ready = mask ? v_masked : v_full;
        for (int j = 0; j < blocks && ok; ++j) {
            ok = warp_wait(&v_ready[j % NS], j / NS, limit);
            if (ok && j + 1 < blocks) ok = warp_wait(&k_full[(j + 1) % NS], (j + 1) / NS, limit);
            for (int i = 0; i < 2 && ok; ++i) {
                if (j >= n[i]) continue;
                ok = warp_wait(&p_full[i], j, limit);
                if (!ok) break;
                tc_fence_after_sync();
                if (lane == 0) {
                    mma_weights<128, DP>(tmem + 256 + DP * i, tmem + 128 * i,
                                         v + (j % NS) * L::kTile, j > 0);
                    mma_commit(&o_full[i]);
                }
                if (j + 1 < n[i]) scores(i, j + 1);
                __syncwarp();
            }
            if (ok && lane == 0) {
                mma_commit(&v_empty[j % NS]);
                if (j + 1 < blocks) mma_commit(&k_empty[(j + 1) % NS]);
            }
            __syncwarp();
        }
        // No product may be in flight when the tensor memory is freed.
        if (lane == 0) {
            mma_commit(drained);
            mbar_wait<false>(drained, 0u, t.wait_limit_cycles);
        }
        __syncwarp();
    } else if (warp == kFwdLoadWarp) {
        // --------------------------------------------------------- loader
        bool ok = true;
        int issued = 0;
        for (int j = 0; j < blocks; ++j) {
            const int st = j % NS;
            if (j >= NS) ok = warp_wait(&k_empty[st], j / NS - 1, limit);
            if (!ok) break;
            if (lane == 0) {
                if (j == 0 && n[0] > 0) {
                    mbar_arrive_expect_tx(&q_full[0], L::kTile);
                    load_tile<128, DP>(smem + L::kQ, &map_q, q0, h, b, &q_full[0]);
                }
                mbar_arrive_expect_tx(&k_full[st], L::kTile);
                load_tile<128, DP>(smem + L::kK + st * L::kTile, &map_k, (j0 + j) << 7, hk, b,
                                   &k_full[st]);
                if (j == 0 && n[1] > 0) {
                    mbar_arrive_expect_tx(&q_full[1], L::kTile);
                    load_tile<128, DP>(smem + L::kQ + L::kTile, &map_q, q0 + 128, h, b,
                                       &q_full[1]);
                }
            }
            __syncwarp();
            if (j >= NS) ok = warp_wait(&v_empty[st], j / NS - 1, limit);
            if (lane == 0 && ok) {
                mbar_arrive_expect_tx(&v_full[st], L::kTile);
                load_tile<128, DP>(smem + L::kV + st * L::kTile, &map_v, (j0 + j) << 7, hk, b,
                                   &v_full[st]);
            }
            __syncwarp();
            issued = j + 1;
            if (!ok) break;
        }
        // After an abort copies may still be in flight: none may land in
        // shared memory after the CTA exits (bounded waits).
        if (*limit.abort_flag && lane == 0) {
            for (int i = 0; i < 2; ++i)
                if (n[i] > 0) mbar_wait<false>(&q_full[i], 0u, t.wait_limit_cycles);
            for (int j = max(0, issued - NS); j < issued; ++j) {
                mbar_wait<false>(&k_full[j % NS], (j / NS) & 1, t.wait_limit_cycles);
                if (ok || j + 1 < issued)
                    mbar_wait<false>(&v_full[j % NS], (j / NS) & 1, t.wait_limit_cycles);
            }
        }
        __syncwarp();
    } else if (warp == kFwdMaskWarp && mask) {
        // ------------------------------------------------------ key masks
        for (int j = 0; j < blocks; ++j) {
            const int st = j % NS;
            if (!warp_wait(&v_full[st], j / NS, limit)) break;
            mask_tile<128, DP>(mask, t.key_len, (j0 + j) << 7, smem + L::kV + st * L::kTile,
                               words + 4 * st, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_masked[st]);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kFwdMmaWarp) tmem_dealloc(tmem, kFwdTmemCols);
    if (threadIdx.x == 0 && flags[0]) raise_error(t.err, kBitTimeout);
}

template <int DP>
cudaError_t launch_fwd(const FattnTask& t, int slot, cudaStream_t stream) {
    const void* kern = reinterpret_cast<const void*>(fattn_fwd_kernel<DP>);
    cudaError_t e = ensure_smem_attribute(kern, slot, FwdSmem<DP>::kBytes, false);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv;
    if (!encode_heads_map(&mq, t.q, t, t.heads, t.query_len, t.q_stride, 128) ||
        !encode_heads_map(&mk, t.k, t, t.kv_heads, t.key_len, t.k_stride, 128) ||
        !encode_heads_map(&mv, t.v, t, t.kv_heads, t.key_len, t.v_stride, 128))
        return cudaErrorInvalidValue;
    const int64_t grid = static_cast<int64_t>((t.query_len + 255) / 256) * t.batch * t.heads;
    fattn_fwd_kernel<DP><<<static_cast<unsigned>(grid), kFwdThreads, FwdSmem<DP>::kBytes,
                           stream>>>(t, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fattn_forward(const FattnTask& task, cudaStream_t stream) {
    return task.d_head <= 64 ? launch_fwd<64>(task, 56, stream)
                             : launch_fwd<128>(task, 57, stream);
}

}  // namespace cs
