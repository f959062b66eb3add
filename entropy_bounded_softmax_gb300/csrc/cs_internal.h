// Internal interface between the C ABI (cs_api.cu) and the kernel
// translation units.  Not installed; the public API is
// include/entropy_bounded_softmax.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "entropy_bounded_softmax.h"

namespace cs {

// Bits of the device error word.
constexpr unsigned int kBitNan = 1u << CS_ERR_NAN_INPUT;
constexpr unsigned int kBitInf = 1u << CS_ERR_INF_INPUT;
constexpr unsigned int kBitOverflow = 1u << CS_ERR_ENTROPY_OVERFLOW;
constexpr unsigned int kBitTimeout = 1u << CS_ERR_TIMEOUT;
constexpr unsigned int kBitBadPage = 1u << CS_ERR_BAD_PAGE;
constexpr unsigned int kBitOutOfPages = 1u << CS_ERR_OUT_OF_PAGES;

// Default limit of every bounded device wait, in SM cycles: 2^31 cycles,
// about 1 s at GB300's 2.07 GHz maximum clock.
constexpr uint64_t kWaitLimitCycles = 1ull << 31;

// One launch's worth of work: every row of the matrix with the same
// parameters (the arguments of section 2.1's signature plus t_out and the
// error word).
struct RowTask {
    const void* logits;    // fp32, or bf16 bit patterns when in_bf16
    float* out;
    float* t_out;          // may be null
    unsigned int* err;     // device error word
    int64_t batch;
    int32_t num_classes;
    int32_t max_iter;
    float entropy_bound;
    float t_min;
    float hi0;             // min(1, t_max): upper end of the search
    int32_t strict;        // 1: evaluate every bisection midpoint
    int32_t async_stage;   // cluster kernel: stage with asynchronous copies
    uint64_t wait_limit_cycles;
    int32_t* evals_out;    // may be null: temperatures evaluated per row
    int32_t in_bf16;       // 1: logits are bf16 (promoted exactly to fp32)
    float fan_beta0;       // cluster kernel: the fan's first inverse
                           // temperature (the others 4 and 16 times it),
                           // evaluated with T = 1; 0: no fan
};

// Cluster kernel geometry.
constexpr int kMaxCluster = 16;
// Temperatures the cluster kernel evaluates with T = 1 in few-row launches
// (the fan: beta0, 4 beta0, 16 beta0, so that one exponential and two
// squarings give all three), and the threads an SM the fan instantiations
// keep registers for (__launch_bounds__(256, 2)).
constexpr int kFanPoints = 3;
constexpr int kFanThreadsPerSm = 512;
constexpr int kClusterMaxThreads = 512;
constexpr int kSlotVals = 12;         // floats per exchange slot (48 bytes)

// Byte offsets of the cluster kernel's dynamic shared memory for `warps`
// warps and cluster size n: the exchange slots [2][n * warps][kSlotVals]
// floats (one per warp of the cluster, double-buffered), the two exchange
// mbarriers, then (128-byte aligned) the slice.
struct ClusterSmemLayout {
    int cslot, cbar, row;
};

__host__ __device__ inline ClusterSmemLayout cluster_smem_layout(int warps,
                                                                 int n) {
    ClusterSmemLayout L;
    int p = 0;
    L.cslot = p;
    p += 2 * n * warps * kSlotVals * 4;
    p = ((p + 7) / 8) * 8;
    L.cbar = p;
    p += 2 * 8;
    L.row = ((p + 127) / 128) * 128;
    return L;
}

// Dynamic shared memory of the cluster kernel for a slice of `slice_len`
// classes, `threads` threads and cluster size `n`.
inline int64_t cluster_smem_bytes(int64_t slice_len, int threads, int n) {
    const ClusterSmemLayout L = cluster_smem_layout(threads / 32, n);
    const int64_t row = ((slice_len + 8 + 3) / 4) * 16;  // pad + tail room
    return L.row + row;
}

// Classes per CTA the automatic plan aims for: 64 KB slices, so that
// three CTAs share an SM and one's exchange overlaps the others' passes.
constexpr int64_t kTargetSlice = 16384;

// Automatic threads per CTA: about 40 classes per thread for a launch with
// about one CTA per SM (up to a quarter more CTAs than SMs; all of a CTA's
// time goes to one row), about 72 for larger launches (several CTAs share
// an SM), rounded up to whole pairs of warps; 128-256 threads either way
// (64-256 for many one-CTA rows), where the per-round reductions stay
// short.
inline int cluster_threads_for(int64_t slice_len, int64_t ctas,
                               int64_t sm_count, int n) {
    const bool many = ctas * 4 > sm_count * 5;
    const int64_t per = many ? 72 : 40;
    int64_t t = (slice_len + per - 1) / per;
    // An even number of warps: the sweep's 16000-class slices ran 2.5-3%
    // faster on 192 or 256 threads than on 224 (six sweep points), and 160
    // was between.
    t = ((t + 63) / 64) * 64;
    // At least 128 threads, or 64 for many one-CTA rows: 4096 rows of
    // 1500-4000 classes ran 20-28% faster in 64-thread CTAs than in
    // 128-thread ones (fewer warps wait at every exchange of a short row).
    const int64_t lo = (many && n == 1) ? 64 : 128;
    if (t < lo) t = lo;
    if (t > 256) t = 256;
    return static_cast<int>(t);
}

// One backward launch: grad_in = (1/T) p (g - <g, p>) for every row.
struct BwdTask {
    const float* probs;     // [batch, C] the forward's output p
    const float* grad_out;  // [batch, C] upstream gradient g
    const float* t;         // [batch] the forward's temperatures
    float* grad_in;         // [batch, C]
    int64_t batch;
    int32_t num_classes;
};

// Backward geometry.  Row-group CTAs of 256 threads; cluster CTAs of up to
// 512 threads whose dynamic shared memory is a 512-byte header (the
// exchange slots) followed by the slice of p and, when STAGE_G, of g.
constexpr int kBwdGroupThreads = 256;
constexpr int kBwdMaxThreads = 512;
constexpr int kBwdSmemHeader = 512;
// Classes per CTA the automatic backward plan aims for: 64 KB of p and g,
// so that three CTAs share an SM and one's reduction overlaps the others'
// loads and stores.
constexpr int64_t kBwdTargetSlice = 8192;

inline int64_t backward_smem_bytes(int64_t slice_len, bool stage_g) {
    return kBwdSmemHeader + (slice_len / 4 + 1) * 16 * (stage_g ? 2 : 1);
}

cudaError_t launch_backward_rowgroup(const BwdTask& task, int lanes_per_row,
                                     int elems_per_lane, cudaStream_t stream);
cudaError_t launch_backward_cluster(const BwdTask& task, int cluster_size,
                                    int slice_len, int threads, int smem_bytes,
                                    bool stage_g, int64_t grid_ctas,
                                    cudaStream_t stream);

// One attention_softmax launch: rows = B H S rows of S scores.
struct AttnTask {
    const float* scores;   // [B, H, S, S]
    float* out;            // [B, H, S, S]
    const float* mask;     // [B, S] or null
    unsigned int* err;     // device error word
    int64_t rows;          // B H S
    int32_t heads;
    int32_t seq_len;
    int32_t causal;
};

// attention_softmax geometry: row-group CTAs of 256 threads; row-CTA
// kernel of up to 512 threads with a 512-byte header (reduction slots)
// before the row in shared memory.
constexpr int kAttnGroupThreads = 256;
constexpr int kAttnMaxThreads = 512;
constexpr int kAttnSmemHeader = 512;

inline int64_t attention_smem_bytes(int64_t seq_len) {
    return kAttnSmemHeader + ((seq_len + 6) / 4 + 1) * 16;
}

cudaError_t launch_attention_rowgroup(const AttnTask& task, int lanes_per_row,
                                      int elems_per_lane, cudaStream_t stream);
cudaError_t launch_attention_cta(const AttnTask& task, int threads,
                                 int smem_bytes, int64_t grid_ctas,
                                 cudaStream_t stream);

// One biencoder_attention launch: BH = batch x heads pairs of query
// [Q, D], keys and values [K, D].
struct BiencTask {
    const float* q;
    const float* k;
    const float* v;
    float* out;            // [BH, Q, D]
    float* attn_out;       // [BH, Q, K] or null
    float* t_out;          // [BH, Q] or null
    unsigned int* err;     // device error word
    int32_t BH;
    int32_t Q;
    int32_t K;
    int32_t D;
    float scale;
    float entropy_bound;
    float t_min;
    float hi0;             // min(1, t_max)
    int32_t max_iter;
    float* p_out;          // non-null: steps 1-2 only, weights written here
    int64_t p_stride;      // floats between weight rows in p_out
};

// biencoder_attention geometry: G lanes per query row holding eight or
// sixteen context items each (K <= 8 G or 16 G, G <= 32), in CTAs of 256
// threads, or 512 for G >= 16 (a 256-item context: 16-row tiles instead of
// 8 made 4 x 8 x 1024 x 256 x 64 24% faster; at G = 8 the larger CTAs were
// 3% slower); keys transposed in shared memory with rows of kp (K rounded
// up to 4) floats.
constexpr int kBiencMaxThreads = 512;
__host__ __device__ constexpr int bienc_threads(int G) {
    return G >= 16 ? 512 : 256;
}
constexpr int kBiencMaxContext = 256;
constexpr int kBiencMaxDHead = 256;

__host__ __device__ inline int bienc_kp(int K) { return (K + 3) & ~3; }

// Row stride in floats of a tile's scores (then weights): at least kp, and
// for G < 8 congruent to 4 G modulo 32, so that the 16-byte reads of the
// rows a quarter-warp's lanes search fall in different banks.
__host__ __device__ inline int bienc_ss_stride(int K, int G) {
    const int kp = bienc_kp(K);
    if (G >= 8) return kp + 4;
    return kp + (((4 * G - kp) % 32) + 32) % 32;
}

// Shared memory of the one-kernel path: transposed keys, values, a tile
// of queries and a tile of scores (which become the weights).
inline int64_t bienc_smem_bytes(int K, int D, int G) {
    const int64_t R = bienc_threads(G) / G;
    const int64_t kp = bienc_kp(K);
    return 4 * (D * kp + static_cast<int64_t>(K) * D + R * (D + 4) +
                R * bienc_ss_stride(K, G));
}

// Shared memory of the scores-and-search kernel when step 3 runs on the
// tensor cores: the transposed keys, a tile of queries and its scores.
inline int64_t bienc_search_smem_bytes(int K, int D, int G) {
    const int64_t R = bienc_threads(G) / G;
    const int64_t kp = bienc_kp(K);
    return 4 * (D * kp + R * (D + 4) + R * bienc_ss_stride(K, G));
}

// Query tiles one CTA works through with its staged keys and values:
// about 128 query rows, at most the pair's whole query range.
inline int bienc_tiles_per_cta(int Q, int G) {
    const int R = bienc_threads(G) / G;
    const int tiles = (Q + R - 1) / R;
    int per = (128 + R - 1) / R;
    if (per > tiles) per = tiles;
    return per < 1 ? 1 : per;
}

cudaError_t launch_bienc(const BiencTask& task, int lanes_per_row,
                         int keys_per_lane, int smem_bytes,
                         cudaStream_t stream);

// biencoder_attention's step 3 on the tensor cores (k_bienc_pv.cu): out =
// P . V for every bh, P written before by the scores-and-search kernel
// (into attn_out, or into the first K floats of each output row).
struct PvTask {
    const float* p;        // P rows: p + (bh Q + i) p_stride
    int64_t p_stride;      // floats between P rows (K or D)
    const float* v;        // [BH, K, D]
    float* out;            // [BH, Q, D]
    unsigned int* err;     // device error word
    int32_t BH;
    int32_t Q;
    int32_t K;
    int32_t D;
    uint64_t wait_limit_cycles;
};

constexpr int kPvM = 128;               // query rows per tile (the MMA's M)
constexpr uint32_t kPvTmemCols = 128;   // two fp32 accumulators of N <= 64
constexpr int kPvMaxD = 64;             // head sizes the tensor-core step takes

// N of the MMA: d_head rounded up to 16; its K: the context rounded up to 8
// (the context is at most d_head, so one shared-memory stage holds it).
__host__ __device__ inline int pv_np(int D) { return (D + 15) & ~15; }
__host__ __device__ inline int pv_kp(int K) { return (K + 7) & ~7; }

// Byte offsets of the step-3 kernel's shared memory: two stages of the
// TF32 halves of a tile's P (stage s: hi at 2 s a_half, lo a_half later),
// each half 128 rows x pv_chunks(K) chunks of 32 items in the MMA's 128-byte
// swizzled K-major layout (a chunk is 128 rows of 128 bytes, 16 KB); the
// halves of V^T (Np x Kp, no swizzle); the output tile (128 rows of D + 4
// floats); ten mbarriers (full, empty, acc_full, acc_empty, landed, two of
// each), the abort flag and the word that receives the tensor-memory
// address.
__host__ __device__ inline int pv_chunks(int K) { return (K + 31) / 32; }

struct PvSmemLayout {
    int a_half, b_hi, b_lo, stage, bar, flag, tslot, end;
};

__host__ __device__ inline PvSmemLayout pv_smem_layout(int K, int Np, int D) {
    PvSmemLayout L;
    const int Kp = pv_kp(K);
    L.a_half = pv_chunks(K) * kPvM * 128;
    L.b_hi = 4 * L.a_half;
    L.b_lo = L.b_hi + Np * Kp * 4;
    L.stage = L.b_lo + Np * Kp * 4;
    L.bar = L.stage + kPvM * (D + 4) * 4;
    L.flag = L.bar + 10 * 8;
    L.tslot = L.flag + 4;
    L.end = L.tslot + 4;
    return L;
}

// Bytes to allocate: the layout plus slack to align it to 1024 bytes.
inline int64_t pv_smem_bytes(int K, int D) {
    return pv_smem_layout(K, pv_np(D), D).end + 1024;
}

// Persistent CTAs, one per SM at most, each taking a contiguous run of
// tiles.
cudaError_t launch_bienc_pv(const PvTask& task, int sm_count,
                            cudaStream_t stream);

// One fused_attention launch (forward or backward): bf16 tensors [batch,
// heads, length, d_head] with element strides of the first three dimensions.
struct FattnTask {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;           // backward: the forward's, read only
    float* lse;              // [batch, heads, query_len]; forward: may be null
    const uint16_t* go;      // backward: gradient of out
    uint16_t* dq;
    uint16_t* dk;
    uint16_t* dv;
    float* rows;             // backward: workspace, see fattn_workspace_floats
    const uint8_t* mask;     // [batch, key_len], nonzero keeps; may be null
    int64_t mask_stride;
    unsigned int* err;       // device error word
    int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3];
    int64_t go_stride[3], dq_stride[3], dk_stride[3], dv_stride[3];
    int32_t batch, heads, kv_heads, query_len, key_len, d_head;
    int32_t causal;
    float scale;
    float inv_group;         // kv_heads / heads
    int32_t split_bits;      // 2^split_bits CTAs, a cluster, share a tile
    int32_t sm_count;
    uint64_t wait_limit_cycles;
};

constexpr int kFattnMaxDHead = 128;
// Heads, sequences and tiles of 128 rows are the launch's three dimensions.
constexpr int kFattnMaxHeads = 1 << 20;
constexpr int kFattnMaxBatch = 65535;
constexpr int kFattnMaxTiles = 65535;

// The backward's workspace: for every query row minus the log2 of its
// normaliser and minus <grad_out, out>, two arrays of batch * heads rows of query_len rounded
// up to whole tiles of 128.
inline int64_t fattn_rows_padded(int32_t query_len) {
    return (static_cast<int64_t>(query_len) + 127) / 128 * 128;
}
inline int64_t fattn_workspace_floats(int32_t batch, int32_t heads, int32_t query_len) {
    return 2 * static_cast<int64_t>(batch) * heads * fattn_rows_padded(query_len);
}

// log2 of the CTAs that share a tile's blocks: 1 to 8, as many as the device
// holds at once of all tiles, with at least `least` blocks each (backward: four;
// 8 query heads on 2 x 77: 15.1 us with one CTA a tile, 13.8 with two of four
// blocks).
inline int split_bits(int64_t tiles, int64_t blocks, int64_t least, int slots) {
    int bits = 0;
    while (bits < 3 && (tiles << (bits + 1)) <= slots && (blocks >> (bits + 1)) >= least) ++bits;
    return bits;
}

cudaError_t launch_fattn_forward(const FattnTask& task, cudaStream_t stream);
cudaError_t launch_fattn_backward(const FattnTask& task, cudaStream_t stream);

// One paged_attention launch: a new token for each of `batch` sequences.
struct PagedTask {
    const uint16_t* q;         // [batch, heads, d_head], bf16 or (fp16) fp16
    const uint16_t* k_pages;   // [num_pages, page_size, kv_heads, d_head]
    const uint16_t* v_pages;
    const int32_t* page_table; // [batch, max_pages]
    const int32_t* lengths;    // [batch]
    uint16_t* out;             // [batch, heads, d_head]
    float* lse;                // [batch, heads] or null
    float2* part_stats;        // workspace: [groups, rows, 2, 16] (max, sum)
    float* part_out;           // [groups, rows, 2, 16, d_head]
    unsigned int* err;         // device error word
    int64_t q_stride[2], o_stride[2], k_stride[3], v_stride[3];
    int64_t table_stride;
    int32_t batch, heads, kv_heads, d_head;
    int32_t page_size, num_pages, max_pages;
    int32_t head_tiles;        // tiles of 16 query heads to a key head
    int32_t split;             // 1: the sequences' steps are dealt to groups of
    int32_t groups;            // kv_heads * head_tiles CTAs, this many
    int32_t fp16;
    float scale;
    float weight_bits;         // log2 of the weights' common factor
};

constexpr int kPagedMaxDHead = 256;

cudaError_t launch_paged(const PagedTask& task, cudaStream_t stream);

// One paged_extend launch.
struct ExtendTask {
    int32_t* page_table;       // [batch, max_pages], entries from held on written
    const int32_t* lengths;    // [batch]
    const int32_t* new_lengths;
    const int32_t* held;       // [batch] or null: the pages of lengths tokens
    const int32_t* free_pages; // [num_free]
    const int32_t* cursor;     // [1] or null: 0
    long long* slots;          // [batch, max_new]
    int32_t* totals;           // [batch]
    int32_t* held_out;         // [batch]
    int32_t* cursor_out;       // [1]
    unsigned int* err;         // device error word
    int64_t table_stride;
    int32_t batch, max_new, max_pages, page_size, num_free;
    int32_t span, sequences;   // of a CTA: places of a sequence, sequences
    int32_t lane_bits;         // log2 of the threads that share a sequence
    int32_t sm_count;
};

cudaError_t launch_extend(ExtendTask task, cudaStream_t stream);

// One paged_write launch: 16-bit elements of either type.
struct WriteTask {
    const uint16_t* keys;      // [batch, new_tokens, kv_heads, d_head]
    const uint16_t* values;
    const int64_t* slots;      // [batch, new_tokens]
    uint16_t* k_pages;         // [num_pages, page_size, kv_heads, d_head]
    uint16_t* v_pages;
    unsigned int* err;         // device error word
    int64_t key_stride[3], value_stride[3], k_stride[3], v_stride[3];
    int64_t slot_stride;
    int64_t num_slots;         // num_pages * page_size
    int32_t tokens, new_tokens, page_size;
    int32_t units, head_units; // of 16 bytes: a token's keys', a head's
    int32_t cta_tokens, cta_units;
    int32_t sm_count;
};

cudaError_t launch_write(WriteTask task, cudaStream_t stream);

// Division of 0 <= n < 2^31 by a number d > 0 that a launch knows, as a product
// and a shift: with 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d) < 2^32, m n =
// 2^(31+s) n / d + e n / d with 0 <= e < d, and the last term, below n < 2^31,
// is too small to carry n / d, whose fraction is at most (d - 1) / d, past the
// next integer, 2^(31+s) / d >= 2^31 away.
struct FastDiv {
    uint32_t mul = 0;   // 0: d is 1
    int32_t shift = 0;
    FastDiv() = default;
    explicit FastDiv(int32_t d) {
        if (d <= 1) return;
        int s = 0;
        while ((int64_t(1) << s) < d) ++s;
        mul = static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d);
        shift = s - 1;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(int n) const {
        return mul == 0 ? n
                        : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
    }
#endif
};

// One paged_tree_attention launch: new_tokens tokens for each of `batch`
// sequences over the cache of PagedTask.
struct TreeTask {
    const uint16_t* q;         // [batch, new_tokens, heads, d_head]
    const uint16_t* k_pages;
    const uint16_t* v_pages;
    const int32_t* page_table; // [batch, max_pages]
    const int32_t* lengths;    // [batch], the new tokens included
    const int32_t* new_lengths;// [batch] or null: all new_tokens
    const uint8_t* mask;       // [batch, new_tokens, new_tokens] or null: j <= i
    uint16_t* out;             // as q
    float* lse;                // [batch, new_tokens, heads] or null
    float2* part_stats;        // workspace: [groups, width, 2, part_rows] (max, sum)
    float* part_out;           // [groups, width, 2, d_head / 4, part_rows, 4]
    unsigned int* err;         // device error word
    int64_t q_stride[3], o_stride[3], k_stride[3], v_stride[3];
    int64_t table_stride;
    int64_t mask_stride[2];
    int32_t batch, new_tokens, heads, kv_heads, group, d_head;
    int32_t page_size, num_pages, max_pages;
    int32_t unit_rows;         // 128 or 256: rows of a unit
    int32_t part_rows;         // rows of one that are there, whole warps
    int32_t width;             // units that a group of CTAs walks side by side
    int32_t bundles;           // width * bundles units to a sequence
    int32_t split;             // 1: the blocks are dealt to groups, this many
    int32_t groups;
    int32_t fp16;
    int32_t box_bits;          // log2 of the tokens of a tensor copy; -1: copies
                               // of 16 bytes
    int32_t tensor_q;          // 1: tensor copies for the queries, too
    int32_t skip, rest;        // a block's tokens: whole pages, and the rest
    FastDiv by_page, by_group, by_kv_heads, by_groups, by_width;
    float scale;
    uint64_t wait_limit_cycles;
};

// What a part's start and end take, in blocks: counted when blocks are dealt (32
// sequences of 256 to 4096 tokens, trees of 16: 40.2 us with 1, 39.3 with 2, 40.5
// with 3; 8 x 64 over 8192: 66.4, 65.0, 64.8; 2 x 512 of 8192: 109.0, 109.2, 110.5).
constexpr int kTreePartCost = 2;

// Tokens of a block.
__host__ __device__ constexpr int tree_block(int d_head) { return d_head > 128 ? 64 : 128; }

cudaError_t launch_tree(const TreeTask& task, cudaStream_t stream);

cudaError_t launch_rowgroup(const RowTask& task, int lanes_per_row,
                            int elems_per_lane, cudaStream_t stream);
cudaError_t launch_cluster(const RowTask& task, int cluster_size,
                           int slice_len, int threads, int smem_bytes,
                           int64_t grid_ctas, cudaStream_t stream);
cudaError_t launch_probe_ex2(float* sink, int iters, int blocks, int threads,
                             cudaStream_t stream);
cudaError_t launch_wait_timeout(unsigned int* err, uint64_t limit_cycles,
                                cudaStream_t stream);
cudaError_t launch_take_error(unsigned int* err, unsigned int* taken,
                              cudaStream_t stream);

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per device and
// kernel, raised only when a launch needs more than was set before.
// slot: one per kernel instantiation; cluster: it is launched in clusters
// (also allows cluster sizes above 8).
cudaError_t ensure_smem_attribute(const void* func, int slot, int bytes,
                                  bool cluster);

// A launch: in clusters of `cluster` CTAs along x, and, if `overlapped`, such
// that it may start before the kernel before it on the stream has ended: the
// kernel calls csd::wait_for_previous_kernel() before it uses what that one
// writes, and in every CTA.
struct LaunchShape {
    dim3 grid;
    int threads, smem_bytes;
    cudaStream_t stream;
    bool overlapped;
    int cluster;
};

template <class... P, class... A>
cudaError_t launch_shaped(void (*kernel)(P...), const LaunchShape& s, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = s.grid;
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = s.smem_bytes;
    cfg.stream = s.stream;
    cudaLaunchAttribute attr[2] = {};
    int n = 0;
    if (s.overlapped) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (s.cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = s.cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace cs
