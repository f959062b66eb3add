// C ABI of libcsoftmax: argument checks, launch planning, the device error
// word, and dispatch to the kernels.  See include/entropy_bounded_softmax.h
// for the contract of every function.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "cs_internal.h"

// The library's device objects: a bitmask of (1 << code) for the
// asynchronous conditions of "BURT-IMMA CUDA Kernel API Reference",
// section 5.1 (set with atomicOr, so no condition overwrites another), and
// the word cs_get_error exchanges it into before copying it to the host.
__device__ unsigned int g_cs_error_word;
__device__ unsigned int g_cs_error_taken;

namespace cs {
int probe_chains();
}

namespace {

constexpr int kMaxDevices = 64;
constexpr int kProbeThreads = 512;
constexpr int kProbeBlocksPerSm = 4;
// Row-group CTAs of two warps: the block scheduler refills SMs at a fine
// grain, which shortens the launch's tail (rows end at different rounds).
constexpr int kRowgroupThreads = 64;
constexpr int kRowgroupMaxLanes = 32;
constexpr int kRowgroupMaxE4 = 8;      // 32 classes per lane
constexpr int kAutoRowgroupE4 = 4;     // 16 classes per lane
// Widest rows the forward plans on the row-group kernel by default: one
// warp of 32 lanes, 32 classes a lane.  Rows of 513-1024 classes ran
// 1.3-1.4x faster there than in one-CTA clusters with a few rows, and
// 3.1-5.3x faster with 4096-16384 rows (measured at 600, 768, 1000 and
// 1024 classes).  The backward keeps 512 (four float4s of p and of g a
// lane).
constexpr int kAutoRowgroupMaxClassesFwd = 1024;
constexpr int kAutoRowgroupMaxClasses = 512;
constexpr int kMaxIter = 1024;
// Largest t_min accepted: 2^64.  Every temperature a kernel evaluates or
// writes is at most max(1, t_min), so 1/T >= 2^-64 and the floored
// exponent (-2^100) times 1/T stays below -2^36: its term is exactly 0.
constexpr float kMaxTMin = 18446744073709551616.0f;
constexpr int64_t kMaxGridX = 2147483647;
constexpr int64_t kMinWideSlice = 2048;

struct DeviceInfo {
    std::atomic<bool> ready{false};
    int sm_count = 0;
    int smem_optin = 0;
    int smem_per_sm = 0;
    int cc_major = 0;
    int cc_minor = 0;
    int max_cluster = 1;
    unsigned int* err = nullptr;
    unsigned int* err_taken = nullptr;
    std::mutex take_mu;  // one cs_get_error at a time uses err_taken
};

DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

cs_status device_info(DeviceInfo** out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    if (dev < 0 || dev >= kMaxDevices) return CS_ERR_CUDA;
    DeviceInfo& d = g_dev[dev];
    if (!d.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_dev_mu);
        if (!d.ready.load(std::memory_order_relaxed)) {
            int v[5] = {0, 0, 0, 0, 0};
            const cudaDeviceAttr attrs[5] = {
                cudaDevAttrMultiProcessorCount,
                cudaDevAttrMaxSharedMemoryPerBlockOptin,
                cudaDevAttrMaxSharedMemoryPerMultiprocessor,
                cudaDevAttrComputeCapabilityMajor,
                cudaDevAttrComputeCapabilityMinor};
            for (int i = 0; i < 5; ++i) {
                if (cudaDeviceGetAttribute(&v[i], attrs[i], dev) != cudaSuccess) {
                    cudaGetLastError();
                    return CS_ERR_CUDA;
                }
            }
            void* p = nullptr;
            void* q = nullptr;
            if (cudaGetSymbolAddress(&p, g_cs_error_word) != cudaSuccess ||
                cudaGetSymbolAddress(&q, g_cs_error_taken) != cudaSuccess) {
                cudaGetLastError();
                return CS_ERR_CUDA;
            }
            d.sm_count = v[0];
            d.smem_optin = v[1];
            d.smem_per_sm = v[2];
            d.cc_major = v[3];
            d.cc_minor = v[4];
            d.max_cluster = v[3] >= 9 ? cs::kMaxCluster : 1;
            d.err = static_cast<unsigned int*>(p);
            d.err_taken = static_cast<unsigned int*>(q);
            d.ready.store(true, std::memory_order_release);
        }
    }
    *out = &d;
    return CS_OK;
}

bool ranges_overlap(const void* a, int64_t a_bytes, const void* b,
                    int64_t b_bytes) {
    if (!a || !b || a_bytes <= 0 || b_bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a);
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(b_bytes) &&
           b0 < a0 + static_cast<uintptr_t>(a_bytes);
}

int next_pow2(int64_t x) {
    int p = 1;
    while (p < x) p <<= 1;
    return p;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

cs_status plan_rowgroup(int64_t batch, int32_t C, int32_t param,
                        cs_plan* p) {
    const int64_t q = ceil_div(C, 4);
    int G = 0, e4 = 0;
    if (param == 0) {
        for (int g = 1; g <= kRowgroupMaxLanes; g <<= 1) {
            if (ceil_div(q, g) <= kAutoRowgroupE4) {
                G = g;
                break;
            }
        }
        if (G == 0) G = kRowgroupMaxLanes;
    } else {
        if (param < 1 || param > kRowgroupMaxLanes || (param & (param - 1)))
            return CS_ERR_INVALID_ARG;
        G = param;
    }
    e4 = next_pow2(ceil_div(q, G));
    if (e4 > kRowgroupMaxE4) return CS_ERR_OOM;
    *p = cs_plan{};
    p->variant = CS_VARIANT_ROWGROUP;
    p->lanes_per_row = G;
    p->elems_per_lane = 4 * e4;
    p->threads_per_cta = kRowgroupThreads;
    // Registers bound residency: at most 64 per thread (80 for 32 classes
    // per lane) out of 65536 per SM.
    p->ctas_per_sm = 65536 / ((e4 >= 8 ? 80 : 64) * kRowgroupThreads);
    if (p->ctas_per_sm > 32) p->ctas_per_sm = 32;
    int64_t blocks = ceil_div(batch * G, kRowgroupThreads);
    if (blocks > kMaxGridX) blocks = kMaxGridX;
    p->grid_ctas = blocks;
    return CS_OK;
}

// Cluster plan for n CTAs per row: slice, threads and shared memory.
// Returns false if it does not fit smem_optin.
bool cluster_geometry(int64_t batch, int32_t C, int n, int threads_req,
                      int sm_count, int smem_optin, cs_plan* p) {
    const int64_t L = ceil_div(ceil_div(C, n), 4) * 4;
    const int threads = threads_req
        ? threads_req : cs::cluster_threads_for(L, batch * n, sm_count, n);
    const int64_t smem = cs::cluster_smem_bytes(L, threads, n);
    if (smem > smem_optin) return false;
    p->cluster_size = n;
    p->slice_len = static_cast<int32_t>(L);
    p->threads_per_cta = threads;
    p->smem_bytes = static_cast<int32_t>(smem);
    p->staged_tensors = 1;
    return true;
}

cs_status plan_cluster(int64_t batch, int32_t C, const cs_options& o,
                       int sm_count, int smem_optin, int smem_per_sm,
                       int max_cluster, cs_plan* p) {
    if (o.threads != 0 &&
        (o.threads < 64 || o.threads > cs::kClusterMaxThreads || o.threads % 32))
        return CS_ERR_INVALID_ARG;
    if (o.strict != 0 && o.strict != 1) return CS_ERR_INVALID_ARG;
    *p = cs_plan{};
    p->variant = CS_VARIANT_CLUSTER;
    if (o.param == 0) {
        // Smallest cluster whose slices are at most kTargetSlice classes
        // (and fit), widened while the launch has fewer CTAs than SMs.
        int n0 = static_cast<int>(ceil_div(C, cs::kTargetSlice));
        if (n0 > max_cluster) n0 = max_cluster;
        if (n0 < 1) n0 = 1;
        // Widen only while every CTA keeps at least kMinWideSlice classes.
        // Few rows: two CTAs per SM, rounded up when that oversubscribes
        // the SMs by at most a quarter.  Two CTAs of a latency-bound launch
        // share an SM well: one's exchange overlaps the other's pass, and
        // the slices (hence every pass) are half as long.  32 x 50000 runs in
        // clusters of 10 x 128 threads, 320 CTAs: 15.9 us, against 17.5 us
        // in clusters of 5 x 256 (one CTA per SM) and 19.2 in clusters of 4.
        const int64_t rows = batch > 0 ? batch : 1;
        const int64_t slots = 2 * static_cast<int64_t>(sm_count);
        int64_t widen = slots / rows;
        const int64_t up = ceil_div(slots, rows);
        if (up > widen && rows * up * 4 <= slots * 5) widen = up;
        if (widen > C / kMinWideSlice) widen = C / kMinWideSlice;
        if (widen > max_cluster) widen = max_cluster;
        if (widen > n0) n0 = static_cast<int>(widen);
        bool ok = false;
        for (int c = n0; c <= max_cluster && !ok; ++c)
            ok = cluster_geometry(batch, C, c, o.threads, sm_count,
                                  smem_optin, p);
        if (!ok) return CS_ERR_OOM;
    } else {
        if (o.param < 1 || o.param > cs::kMaxCluster) return CS_ERR_INVALID_ARG;
        if (o.param > max_cluster) return CS_ERR_INVALID_ARG;
        if (!cluster_geometry(batch, C, o.param, o.threads, sm_count,
                              smem_optin, p))
            return CS_ERR_OOM;
    }
    const int n = p->cluster_size;
    const int by_smem = static_cast<int>(smem_per_sm / (p->smem_bytes + 1024));
    const int by_threads = 2048 / p->threads_per_cta;
    p->ctas_per_sm = by_smem < by_threads ? by_smem : by_threads;
    int64_t rows = batch;
    const int64_t max_rows = kMaxGridX / n;
    if (rows > max_rows) rows = max_rows;
    p->grid_ctas = rows * n;
    // Launches of at most one wave are bound by the slowest row's chain of
    // rounds: there the fan, a few more exponentials per class in the T = 1
    // pass, saves rounds.  Wider launches are bound by throughput, where the
    // extra exponentials cost more than the rounds they save.  The fan runs
    // in clusters of CTAs of at most 256 threads, built with registers for
    // 512 threads an SM (cs::kFanThreadsPerSm).
    const int64_t fan_ctas_per_sm = cs::kFanThreadsPerSm / p->threads_per_cta;
    const int64_t resident =
        fan_ctas_per_sm < p->ctas_per_sm ? fan_ctas_per_sm : p->ctas_per_sm;
    const bool one_wave = p->grid_ctas <= static_cast<int64_t>(sm_count) * resident;
    p->fan_points = (o.strict == 0 && n > 1 && p->threads_per_cta <= 256 && one_wave)
        ? cs::kFanPoints : 0;
    if (p->fan_points > 0 && o.param == 0 && o.threads == 0 &&
        p->grid_ctas > 2 * static_cast<int64_t>(sm_count)) {
        // With the fan the T = 1 pass is about twice as long, and a CTA
        // that shares its SM with two others holds up its whole cluster's
        // first exchange: when the widening above rounded up past two CTAs
        // an SM, take instead the largest power-of-two cluster that keeps
        // at most two on every SM (32 x 50000: clusters of 8 x 128, 14.5 us,
        // against 15.3 us in the clusters of 10).
        int nf = 1;
        while (nf * 2 <= max_cluster && nf * 2 <= C / kMinWideSlice &&
               rows * nf * 2 <= 2 * static_cast<int64_t>(sm_count))
            nf *= 2;
        cs_plan q = *p;
        if (nf > 1 && nf != n && ceil_div(C, nf) <= cs::kTargetSlice &&
            cluster_geometry(batch, C, nf, 0, sm_count, smem_optin, &q) &&
            q.threads_per_cta <= 256) {
            const int bs = static_cast<int>(smem_per_sm / (q.smem_bytes + 1024));
            const int bt = 2048 / q.threads_per_cta;
            q.ctas_per_sm = bs < bt ? bs : bt;
            q.grid_ctas = rows * nf;
            *p = q;
        }
    }
    return CS_OK;
}

// ------------------------------------------------------------------ backward
// Row-group backward: G lanes per row, the smallest power of two that leaves
// at most four float4s of p (and of g) per lane; float4s counted for the
// worst alignment of a row start (pad 3), since rows of a num_classes that
// is not a multiple of 4 start at every alignment.
cs_status plan_backward_rowgroup(int64_t batch, int32_t C, int32_t param,
                                 cs_plan* p) {
    const int64_t q = (static_cast<int64_t>(C) + 6) / 4;
    int G = 0;
    if (param == 0) {
        for (int g = 1; g <= kRowgroupMaxLanes; g <<= 1) {
            if (ceil_div(q, g) <= kAutoRowgroupE4) {
                G = g;
                break;
            }
        }
        if (G == 0) G = kRowgroupMaxLanes;
    } else {
        if (param < 1 || param > kRowgroupMaxLanes || (param & (param - 1)))
            return CS_ERR_INVALID_ARG;
        G = param;
    }
    const int e4 = next_pow2(ceil_div(q, G));
    if (e4 > kRowgroupMaxE4) return CS_ERR_OOM;
    const int64_t blocks = ceil_div(batch * G, cs::kBwdGroupThreads);
    if (blocks > kMaxGridX) return CS_ERR_DIM_MISMATCH;
    *p = cs_plan{};
    p->variant = CS_VARIANT_ROWGROUP;
    p->lanes_per_row = G;
    p->elems_per_lane = 4 * e4;
    p->threads_per_cta = cs::kBwdGroupThreads;
    // Registers bound residency: 2 x 4 e4 for the row plus about 28
    // (ptxas: 32, 38, 60 and 90 for e4 = 1, 2, 4, 8).
    int regs = ((8 * e4 + 28 + 7) / 8) * 8;
    if (regs < 32) regs = 32;
    p->ctas_per_sm = 65536 / (regs * cs::kBwdGroupThreads);
    if (p->ctas_per_sm > 2048 / cs::kBwdGroupThreads)
        p->ctas_per_sm = 2048 / cs::kBwdGroupThreads;
    p->grid_ctas = blocks;
    return CS_OK;
}

// Cluster backward geometry for n CTAs per row: p and g staged when both
// fit, else p alone (stage_both = false); false if neither fits.  per: the
// float4s of each staged tensor per thread the automatic thread count aims
// for.
bool backward_geometry(int32_t C, int n, int threads_req, int smem_optin,
                       bool stage_both, int per, cs_plan* p) {
    const int64_t L = ceil_div(ceil_div(C, n), 4) * 4;
    const int64_t smem = cs::backward_smem_bytes(L, stage_both);
    if (smem > smem_optin) return false;
    int threads = threads_req;
    if (threads == 0) {
        int64_t t = ceil_div(ceil_div(L, 4), per);
        t = ceil_div(t, 32) * 32;
        if (t < 64) t = 64;
        if (t > cs::kBwdMaxThreads) t = cs::kBwdMaxThreads;
        threads = static_cast<int>(t);
    }
    p->cluster_size = n;
    p->slice_len = static_cast<int32_t>(L);
    p->threads_per_cta = threads;
    p->smem_bytes = static_cast<int32_t>(smem);
    p->staged_tensors = stage_both ? 2 : 1;
    return true;
}

cs_status plan_backward_cluster(int64_t batch, int32_t C, const cs_options& o,
                                int sm_count, int smem_optin, int smem_per_sm,
                                int max_cluster, cs_plan* p) {
    if (o.threads != 0 &&
        (o.threads < 64 || o.threads > cs::kBwdMaxThreads || o.threads % 32))
        return CS_ERR_INVALID_ARG;
    *p = cs_plan{};
    p->variant = CS_VARIANT_CLUSTER;
    bool ok = false;
    if (o.param == 0) {
        // Smallest cluster whose slices are at most kBwdTargetSlice classes,
        // widened to about two CTAs per SM for few rows while slices keep
        // kMinWideSlice classes (32 x 50000: clusters of 10, 5000-class
        // slices).
        int n0 = static_cast<int>(ceil_div(C, cs::kBwdTargetSlice));
        if (n0 > max_cluster) n0 = max_cluster;
        if (n0 < 1) n0 = 1;
        const int64_t rows = batch > 0 ? batch : 1;
        int64_t widen = ceil_div(2 * static_cast<int64_t>(sm_count), rows);
        if (widen > C / kMinWideSlice) widen = C / kMinWideSlice;
        if (widen > max_cluster) widen = max_cluster;
        // Launches of few CTAs are latency-bound: fewer float4s per thread
        // (32 x 50000 in clusters of 10: 6.9 us on 160 threads, 6.6 on
        // 256); larger ones aim for eight, enough in flight per SM.
        const int per = widen > n0 ? 5 : 8;
        if (widen > n0) n0 = static_cast<int>(widen);
        for (int c = n0; c <= max_cluster && !ok; ++c)
            ok = backward_geometry(C, c, o.threads, smem_optin, true, per, p);
        if (!ok)
            ok = backward_geometry(C, max_cluster, o.threads, smem_optin,
                                   false, per, p);
    } else {
        if (o.param < 1 || o.param > cs::kMaxCluster) return CS_ERR_INVALID_ARG;
        if (o.param > max_cluster) return CS_ERR_INVALID_ARG;
        ok = backward_geometry(C, o.param, o.threads, smem_optin, true, 8, p) ||
             backward_geometry(C, o.param, o.threads, smem_optin, false, 8, p);
    }
    if (!ok) return CS_ERR_OOM;
    const int n = p->cluster_size;
    const int by_smem = static_cast<int>(smem_per_sm / (p->smem_bytes + 1024));
    const int by_threads = 2048 / p->threads_per_cta;
    p->ctas_per_sm = by_smem < by_threads ? by_smem : by_threads;
    int64_t rows = batch;
    const int64_t max_rows = kMaxGridX / n;
    if (rows > max_rows) rows = max_rows;
    p->grid_ctas = rows * n;
    return CS_OK;
}

// ------------------------------------------------------------------ attention
cs_status plan_attention(int32_t batch, int32_t heads, int32_t S,
                         int32_t aligned, const cs_options& o, int sm_count,
                         int smem_optin, int smem_per_sm, cs_plan* p) {
    (void)sm_count;
    if (o.strict != 0 || o.evals_out) return CS_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(batch) * heads * S;
    // Float4s a row spans: exact for aligned rows, else at the worst
    // alignment of a row start.
    int64_t q = aligned ? ceil_div(S, 4) : (static_cast<int64_t>(S) + 6) / 4;
    if (q < 1) q = 1;
    int variant = o.variant;
    if (variant == CS_VARIANT_AUTO) {
        if (o.param != 0 || o.threads != 0) return CS_ERR_INVALID_ARG;
        variant = q <= kRowgroupMaxLanes * kRowgroupMaxE4 ? CS_VARIANT_ROWGROUP
                                                          : CS_VARIANT_CLUSTER;
    }
    *p = cs_plan{};
    if (variant == CS_VARIANT_ROWGROUP) {
        if (o.threads != 0) return CS_ERR_INVALID_ARG;
        int G = 0;
        if (o.param == 0) {
            for (int g = 1; g <= kRowgroupMaxLanes; g <<= 1) {
                if (ceil_div(q, g) <= kAutoRowgroupE4) {
                    G = g;
                    break;
                }
            }
            if (G == 0) G = kRowgroupMaxLanes;
        } else {
            if (o.param < 1 || o.param > kRowgroupMaxLanes || (o.param & (o.param - 1)))
                return CS_ERR_INVALID_ARG;
            G = o.param;
        }
        const int e4 = next_pow2(ceil_div(q, G));
        if (e4 > kRowgroupMaxE4) return CS_ERR_OOM;
        const int64_t blocks = ceil_div(rows * G, cs::kAttnGroupThreads);
        if (blocks > kMaxGridX) return CS_ERR_DIM_MISMATCH;
        p->variant = CS_VARIANT_ROWGROUP;
        p->lanes_per_row = G;
        p->elems_per_lane = 4 * e4;
        p->threads_per_cta = cs::kAttnGroupThreads;
        int regs = ((4 * e4 + 30 + 7) / 8) * 8;
        p->ctas_per_sm = 65536 / (regs * cs::kAttnGroupThreads);
        if (p->ctas_per_sm > 2048 / cs::kAttnGroupThreads)
            p->ctas_per_sm = 2048 / cs::kAttnGroupThreads;
        p->grid_ctas = blocks;
        return CS_OK;
    }
    if (variant != CS_VARIANT_CLUSTER) return CS_ERR_INVALID_ARG;
    if (o.param != 0 && o.param != 1) return CS_ERR_INVALID_ARG;
    if (o.threads != 0 &&
        (o.threads < 64 || o.threads > cs::kAttnMaxThreads || o.threads % 32))
        return CS_ERR_INVALID_ARG;
    const int64_t smem = cs::attention_smem_bytes(S);
    if (smem > smem_optin) return CS_ERR_OOM;
    int threads = o.threads;
    if (threads == 0) {
        // About eight float4s per thread.
        int64_t t = ceil_div(ceil_div(q, 8), 32) * 32;
        if (t < 64) t = 64;
        if (t > cs::kAttnMaxThreads) t = cs::kAttnMaxThreads;
        threads = static_cast<int>(t);
    }
    p->variant = CS_VARIANT_CLUSTER;
    p->cluster_size = 1;
    p->slice_len = S;
    p->threads_per_cta = threads;
    p->smem_bytes = static_cast<int32_t>(smem);
    p->staged_tensors = 1;
    const int by_smem = static_cast<int>(smem_per_sm / (smem + 1024));
    const int by_threads = 2048 / threads;
    p->ctas_per_sm = by_smem < by_threads ? by_smem : by_threads;
    p->grid_ctas = rows < kMaxGridX ? rows : kMaxGridX;
    return CS_OK;
}

}  // namespace

namespace {

// Argument check of the forward for logits of in_bytes (4: fp32, 2: bf16)
// per element.
cs_status check_forward_args(const void* logits, const float* out,
                             int64_t batch, int32_t num_classes,
                             float entropy_bound, float t_min, float t_max,
                             int32_t max_iter, const float* t_out,
                             int in_bytes) {
    if (batch < 0 || num_classes < 1) return CS_ERR_DIM_MISMATCH;
    if (num_classes > CS_MAX_NUM_CLASSES) return CS_ERR_OOM;
    if (batch > INT64_MAX / 4 / num_classes) return CS_ERR_DIM_MISMATCH;
    if (isnan(entropy_bound)) return CS_ERR_INVALID_ARG;
    if (!(t_min >= FLT_MIN) || !(t_min <= kMaxTMin)) return CS_ERR_INVALID_ARG;
    if (isnan(t_max) || t_max < t_min) return CS_ERR_INVALID_ARG;
    if (max_iter < 0 || max_iter > kMaxIter) return CS_ERR_INVALID_ARG;
    if (batch == 0) return CS_OK;
    if (!logits || !out) return CS_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % in_bytes) return CS_ERR_INVALID_ARG;
    const int64_t in_size = batch * num_classes * in_bytes;
    const int64_t bytes = batch * num_classes * 4;
    if (ranges_overlap(logits, in_size, out, bytes)) return CS_ERR_INVALID_ARG;
    if (t_out && (ranges_overlap(t_out, batch * 4, logits, in_size) ||
                  ranges_overlap(t_out, batch * 4, out, bytes)))
        return CS_ERR_INVALID_ARG;
    return CS_OK;
}

// The forward for fp32 (in_bf16 = false) or bf16 logits.
cs_status forward(const void* logits, bool in_bf16, float* out, int64_t batch,
                  int32_t num_classes, float entropy_bound, float t_min,
                  float t_max, int32_t max_iter, float* t_out,
                  const cs_options* options, void* stream) {
    const int in_bytes = in_bf16 ? 2 : 4;
    cs_status st = check_forward_args(logits, out, batch, num_classes,
                                      entropy_bound, t_min, t_max, max_iter,
                                      t_out, in_bytes);
    if (st != CS_OK) return st;
    if (batch == 0) return CS_OK;
    if (options && options->evals_out) {
        const int64_t bytes = batch * num_classes * 4;
        const void* e = options->evals_out;
        if (ranges_overlap(e, batch * 4, logits, batch * num_classes * in_bytes) ||
            ranges_overlap(e, batch * 4, out, bytes) ||
            (t_out && ranges_overlap(e, batch * 4, t_out, batch * 4)))
            return CS_ERR_INVALID_ARG;
    }
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs_plan p;
    st = cs_plan_host(batch, num_classes, options, d->sm_count, d->smem_optin,
                      d->smem_per_sm, d->max_cluster, &p);
    if (st != CS_OK) return st;

    cs::RowTask task;
    task.logits = logits;
    task.out = out;
    task.t_out = t_out;
    task.err = d->err;
    task.batch = batch;
    task.num_classes = num_classes;
    task.max_iter = max_iter;
    task.entropy_bound = entropy_bound;
    task.t_min = t_min;
    task.hi0 = t_max < 1.0f ? t_max : 1.0f;
    task.strict = options ? options->strict : 0;
    // Asynchronous staging pays when several CTAs share an SM (the same
    // threshold as the per-thread work rule of the thread count).
    task.async_stage = p.grid_ctas * 4 > static_cast<int64_t>(d->sm_count) * 5;
    task.wait_limit_cycles = cs::kWaitLimitCycles;
    task.evals_out = options ? options->evals_out : nullptr;
    task.in_bf16 = in_bf16 ? 1 : 0;
    // The fan's inverse temperatures sqrt(1 / (hi0 t_min)) times 1/4, 1 and
    // 4: the middle of the search's range in log beta and a factor 4 on
    // either side; only when that range spans a factor 64 or more.
    task.fan_beta0 = 0.0f;
    if (p.variant == CS_VARIANT_CLUSTER && p.fan_points > 0 &&
        entropy_bound > 0.0f && 64.0 * t_min <= task.hi0)
        task.fan_beta0 = static_cast<float>(
            0.25 / sqrt(static_cast<double>(task.hi0) * t_min));

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.variant == CS_VARIANT_ROWGROUP) {
        e = cs::launch_rowgroup(task, p.lanes_per_row, p.elems_per_lane, s);
    } else {
        e = cs::launch_cluster(task, p.cluster_size, p.slice_len,
                               p.threads_per_cta, p.smem_bytes, p.grid_ctas, s);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

// ------------------------------------------------------------ fused attention
// Whether rows of d elements at these strides (n <= 3 dimensions, more than
// one element each or not looked at) can share an element: unless each stride,
// in ascending order, steps past all that the smaller ones span.  (Orders that
// interleave without sharing any are refused with them.)
bool overlaps_itself(const int64_t* dim, const int64_t* stride, int n, int32_t d) {
    int64_t span = d;
    int taken = 0;
    for (int round = 0; round < n; ++round) {
        int next = -1;   // the smallest stride not taken
        for (int i = 0; i < n; ++i)
            if (dim[i] > 1 && !(taken >> i & 1) && (next < 0 || stride[i] < stride[next]))
                next = i;
        if (next < 0) break;
        taken |= 1 << next;
        if (stride[next] < span) return true;
        span += (dim[next] - 1) * stride[next];
    }
    return false;
}

// Sizes and strides of one [batch, heads, length, d_head] bf16 tensor: the
// bytes from its first to past its last element, or -1 when a stride is
// refused (negative, not a multiple of 8 elements, or 0 over more than one
// element; strides of dimensions of one element are not looked at; of a
// written tensor also strides that may share elements).
int64_t heads_extent(const cs_attention_shape& s, int32_t heads, int32_t length,
                     const int64_t* stride, bool written = false) {
    const int64_t dim[3] = {s.batch, heads, length};
    int64_t last = s.d_head;
    for (int i = 0; i < 3; ++i) {
        if (dim[i] == 0) return 0;
    }
    for (int i = 0; i < 3; ++i) {
        if (dim[i] == 1) continue;
        // The tensor copies take strides below 2^40 bytes.
        if (stride[i] <= 0 || stride[i] % 8 != 0 || stride[i] >= (int64_t(1) << 39))
            return -1;
        if (stride[i] > (int64_t(1) << 60) / dim[i]) return -1;
        last += (dim[i] - 1) * stride[i];
        if (last > (int64_t(1) << 60)) return -1;
    }
    if (written && overlaps_itself(dim, stride, 3, s.d_head)) return -1;
    return 2 * last;
}

// The kernels multiply scores by scale log2(e), which has to be finite too.
bool good_scale(float scale) { return scale > 0.0f && scale <= 0x1p127f; }

cs_status check_attention_shape(const cs_attention_shape* s) {
    if (!s) return CS_ERR_INVALID_ARG;
    if (s->batch < 0 || s->heads < 1 || s->kv_heads < 1 || s->query_len < 0 ||
        s->key_len < 0 || s->d_head < 1 || s->heads % s->kv_heads != 0)
        return CS_ERR_DIM_MISMATCH;
    if (s->d_head > cs::kFattnMaxDHead) return CS_ERR_OOM;
    if (s->d_head % 8 != 0) return CS_ERR_INVALID_ARG;
    if (s->causal != 0 && s->causal != 1) return CS_ERR_INVALID_ARG;
    if (!good_scale(s->scale)) return CS_ERR_INVALID_ARG;
    if (s->heads > cs::kFattnMaxHeads || s->batch > cs::kFattnMaxBatch ||
        ceil_div(s->query_len, 128) > cs::kFattnMaxTiles ||
        ceil_div(s->key_len, 128) > cs::kFattnMaxTiles)
        return CS_ERR_DIM_MISMATCH;
    return CS_OK;
}

// One tensor of a call: where it is, how far it reaches, whether the call
// writes it.
struct Span {
    const void* data;
    int64_t bytes;
    int align;
    bool written;
};

// Every span present, aligned, and no written one overlapping another.
cs_status check_spans(const Span* x, int n) {
    for (int i = 0; i < n; ++i) {
        if (x[i].bytes < 0) return CS_ERR_INVALID_ARG;
        if (x[i].bytes == 0) continue;
        if (!x[i].data || reinterpret_cast<uintptr_t>(x[i].data) % x[i].align)
            return CS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if ((x[i].written || x[j].written) &&
                ranges_overlap(x[i].data, x[i].bytes, x[j].data, x[j].bytes))
                return CS_ERR_INVALID_ARG;
    }
    return CS_OK;
}

// The most bytes, or entries, between the rows of a mask or a page table, so
// that their extent stays within 64 bits.
constexpr int64_t kMaxRowStride = int64_t(1) << 40;

int64_t mask_extent(const cs_attention_shape& s, const uint8_t* mask) {
    if (!mask || s.batch == 0 || s.key_len == 0) return 0;
    if (s.batch > 1 && (s.mask_stride < s.key_len || s.mask_stride > kMaxRowStride)) return -1;
    return s.key_len + (s.batch > 1 ? (s.batch - 1) * s.mask_stride : 0);
}

cs::FattnTask attention_task(const cs_attention_shape& s, const uint8_t* mask,
                             const DeviceInfo& d) {
    cs::FattnTask t{};
    t.mask = mask;
    t.mask_stride = s.mask_stride;
    t.err = d.err;
    t.sm_count = d.sm_count;
    for (int i = 0; i < 3; ++i) {
        t.q_stride[i] = s.q_stride[i];
        t.k_stride[i] = s.k_stride[i];
        t.v_stride[i] = s.v_stride[i];
        t.o_stride[i] = s.o_stride[i];
        t.go_stride[i] = s.go_stride[i];
        t.dq_stride[i] = s.dq_stride[i];
        t.dk_stride[i] = s.dk_stride[i];
        t.dv_stride[i] = s.dv_stride[i];
    }
    t.batch = s.batch;
    t.heads = s.heads;
    t.kv_heads = s.kv_heads;
    t.query_len = s.query_len;
    t.key_len = s.key_len;
    t.d_head = s.d_head;
    t.causal = s.causal;
    t.scale = s.scale;
    t.inv_group = static_cast<float>(static_cast<double>(s.kv_heads) / s.heads);
    t.wait_limit_cycles = cs::kWaitLimitCycles;
    return t;
}

// ------------------------------------------------------------ paged attention
constexpr int32_t kPagedMaxTokens = 1 << 30;
constexpr int64_t kPagedStep = 64;      // tokens
// The workspace, whose size is worked out without a device, is for the groups
// of this many SMs, a GB300's; a device with fewer deals to fewer groups.
constexpr int kPagedMaxSms = 152;

cs_status check_paged_shape(const cs_paged_shape* s) {
    if (!s) return CS_ERR_INVALID_ARG;
    if (s->batch < 0 || s->heads < 1 || s->kv_heads < 1 || s->d_head < 1 ||
        s->heads % s->kv_heads != 0 || s->page_size < 1 || s->num_pages < 0 ||
        s->max_pages < 0)
        return CS_ERR_DIM_MISMATCH;
    if (s->d_head > cs::kPagedMaxDHead) return CS_ERR_OOM;
    if (s->d_head % 8 != 0) return CS_ERR_INVALID_ARG;
    if (s->fp16 != 0 && s->fp16 != 1) return CS_ERR_INVALID_ARG;
    if (!good_scale(s->scale)) return CS_ERR_INVALID_ARG;
    if (static_cast<int64_t>(s->max_pages) * s->page_size > kPagedMaxTokens ||
        s->batch > cs::kFattnMaxBatch || s->heads > cs::kFattnMaxHeads)
        return CS_ERR_DIM_MISMATCH;
    return CS_OK;
}

int32_t paged_head_tiles(const cs_paged_shape& s) {
    return static_cast<int32_t>(ceil_div(s.heads / s.kv_heads, 16));
}

// The most steps a sequence can have, and the rows of one.
int64_t paged_steps(const cs_paged_shape& s) {
    return ceil_div(static_cast<int64_t>(s.max_pages) * s.page_size, kPagedStep);
}
int64_t paged_rows(const cs_paged_shape& s) {
    return static_cast<int64_t>(s.kv_heads) * paged_head_tiles(s);
}

// Groups of CTAs that the steps are dealt to: as many as `sms` SMs hold at once
// (4, 2 or 1 CTAs each by the shared memory of their rings), because a CTA's
// start and end cost it microseconds of streaming.  One sequence of 131072
// tokens, 8 key heads, on 152 SMs cut for 304 CTAs: 82 us, for 608: 88, for
// 1216: 96.  Whole groups only: rows that do not divide the SMs' CTAs leave the
// rest of them idle, up to half with just over half as many rows (d_head 256
// and 80 key heads: 80 of 152).
// 0: every row of a sequence is one CTA's, and there is nothing to join: where
// no sequence can be longer than 4 steps, or than 8 with at least 128 such
// CTAs, which keep the device busy by themselves.  Lengths up to 512 tokens,
// from a quarter of it on: 128 CTAs 10.5 us whole and 11.5 cut (d_head 128),
// 256 CTAs 12.3 and 15.8; 64 CTAs 10.4 and 9.7, 16 CTAs 10.1 and 7.2.  Up to
// 1024 cut is faster with 128 CTAs, 13.6 and 17.3, and as fast with 256.
int64_t paged_groups(const cs_paged_shape& s, int sms) {
    const int64_t steps = paged_steps(s);
    if (steps <= 4 || (steps <= 8 && s.batch * paged_rows(s) >= 128)) return 0;
    const int64_t ctas = sms * (s.d_head <= 64 ? 4 : s.d_head <= 128 ? 2 : 1);
    int64_t n = ctas / paged_rows(s);
    if (n < 1) n = 1;
    const int64_t total = paged_steps(s) * s.batch;
    return n < total ? n : total;
}

// The bytes of a strided tensor with a contiguous last dimension of d, from
// its first to past its last element; -1 for a refused stride.
int64_t strided_extent(const int64_t* dim, const int64_t* stride, int n, int32_t d) {
    int64_t last = d;
    for (int i = 0; i < n; ++i)
        if (dim[i] == 0) return 0;
    for (int i = 0; i < n; ++i) {
        if (dim[i] == 1) continue;
        if (stride[i] < 0 || stride[i] % 8 != 0 || stride[i] > (int64_t(1) << 40))
            return -1;
        if (stride[i] > (int64_t(1) << 60) / dim[i]) return -1;
        last += (dim[i] - 1) * stride[i];
        if (last > (int64_t(1) << 60)) return -1;
    }
    return 2 * last;
}

// ------------------------------------------- several new tokens over a cache
int64_t tree_steps(const cs_tree_shape& s) {
    return ceil_div(static_cast<int64_t>(s.max_pages) * s.page_size, cs::tree_block(s.d_head));
}

cs_status check_tree_shape(const cs_tree_shape* s) {
    if (!s) return CS_ERR_INVALID_ARG;
    if (s->batch < 0 || s->new_tokens < 0 || s->heads < 1 || s->kv_heads < 1 || s->d_head < 1 ||
        s->heads % s->kv_heads != 0 || s->page_size < 1 || s->num_pages < 0 ||
        s->max_pages < 0)
        return CS_ERR_DIM_MISMATCH;
    if (s->d_head > cs::kPagedMaxDHead) return CS_ERR_OOM;
    if (s->d_head % 8 != 0) return CS_ERR_INVALID_ARG;
    if (s->fp16 != 0 && s->fp16 != 1) return CS_ERR_INVALID_ARG;
    if (!good_scale(s->scale)) return CS_ERR_INVALID_ARG;
    if (static_cast<int64_t>(s->max_pages) * s->page_size > kPagedMaxTokens ||
        s->batch > cs::kFattnMaxBatch || s->heads > cs::kFattnMaxHeads ||
        static_cast<int64_t>(s->new_tokens) * (s->heads / s->kv_heads) > (1 << 30))
        return CS_ERR_DIM_MISMATCH;
    return CS_OK;
}

// How the blocks of a batch are dealt on `sms` SMs, each with room for one CTA.
struct TreePlan {
    int32_t unit_rows, part_rows, width, groups;
    int64_t units;   // of a sequence
};

TreePlan tree_plan(const cs_tree_shape& s, int sms) {
    TreePlan p;
    const int64_t rows = static_cast<int64_t>(s.new_tokens) * (s.heads / s.kv_heads);
    p.unit_rows = rows > 128 && s.d_head <= 128 ? 256 : 128;
    p.part_rows = static_cast<int32_t>(rows >= p.unit_rows ? p.unit_rows : ceil_div(rows, 32) * 32);
    p.units = s.kv_heads * ceil_div(rows, p.unit_rows);
    // CTAs side by side on the same pages: as many as leave few SMs out.
    int32_t w = static_cast<int32_t>(p.units < sms ? p.units : sms);
    while (w > 1 && (p.units % w != 0 || (sms / w) * w * 20 < sms * 19)) --w;
    p.width = w < 1 ? 1 : w;
    // 0: a CTA for every unit, and nothing to join: with no more units than SMs,
    // where no sequence can be longer than 4 blocks, or than 8 with units for at
    // least three quarters of the SMs.  Blocks of 128, cut and whole, on the GPU
    // (a call from the host takes 5 us less whole): 1 x 512 tokens, 8 units, 10.6
    // and 10.6 us; 16 x 1024, 128 units, 16.4 and 15.2, 4 x 1024 12.7 and 14.5;
    // 7 x 1531, 84 units, 15.5 and 19.4; 256 x 512, 2048 units, 85 and 115.
    // (The workspace's size goes by this too, and knows no device: so the SMs
    // are a GB300's.)
    const int64_t steps = tree_steps(s), total = steps * s.batch * (p.units / p.width);
    const int64_t all = s.batch * p.units;
    const bool whole = all <= kPagedMaxSms &&
                       (steps <= 4 || (steps <= 8 && 4 * all >= 3 * kPagedMaxSms));
    p.groups = whole ? 0 : static_cast<int32_t>(sms / p.width < total ? sms / p.width : total);
    return p;
}

int64_t tree_workspace(const cs_tree_shape& s, const TreePlan& p) {
    if (p.groups == 0) return 0;
    // Two parts a CTA: the (maximum, sum) pairs, the outputs.  (However the
    // device's SMs are grouped: at most one CTA an SM, and one a block.)
    const int64_t blocks = tree_steps(s) * s.batch;
    const int64_t ctas =
        blocks >= kPagedMaxSms || blocks * p.units >= kPagedMaxSms ? kPagedMaxSms : blocks * p.units;
    const int64_t rows = ctas * 2 * p.part_rows;
    return rows * 8 + rows * s.d_head * 4;
}

// cs_check_paged_tree_attention_args, which leaves the plan for a GB300's SMs.
cs_status check_tree(const uint16_t* query, const uint16_t* key_pages,
                     const uint16_t* value_pages, const int32_t* page_table,
                     const int32_t* lengths, const int32_t* new_lengths, const uint8_t* mask,
                     const uint16_t* out, const float* lse, const cs_tree_shape* shape,
                     const void* workspace, int64_t workspace_bytes, TreePlan& p) {
    const cs_status st = check_tree_shape(shape);
    if (st != CS_OK) return st;
    const cs_tree_shape& s = *shape;
    if (s.batch == 0 || s.new_tokens == 0) return CS_OK;
    // Blocks, with what a part's start and end count, and CTAs are counted in 32
    // bits.
    p = tree_plan(s, kPagedMaxSms);
    if (p.units * s.batch > (1 << 30) ||
        tree_steps(s) + cs::kTreePartCost > (1 << 30) / (s.batch * (p.units / p.width)))
        return CS_ERR_DIM_MISMATCH;
    const int64_t need = tree_workspace(s, p);
    if (workspace_bytes < need) return CS_ERR_INVALID_ARG;
    if (s.batch > 1 && (s.table_stride < s.max_pages || s.table_stride > kMaxRowStride))
        return CS_ERR_INVALID_ARG;
    int64_t mask_bytes = 0;
    if (mask) {
        if ((s.new_tokens > 1 &&
             (s.mask_stride[1] < s.new_tokens || s.mask_stride[1] > kMaxRowStride >> 10)) ||
            (s.batch > 1 && (s.mask_stride[0] < 0 || s.mask_stride[0] > kMaxRowStride)))
            return CS_ERR_INVALID_ARG;
        mask_bytes = s.new_tokens +
                     (s.new_tokens > 1 ? (s.new_tokens - 1) * s.mask_stride[1] : 0) +
                     (s.batch > 1 ? (s.batch - 1) * s.mask_stride[0] : 0);
    }
    const int64_t rows[3] = {s.batch, s.new_tokens, s.heads};
    const int64_t pages[3] = {s.num_pages, s.page_size, s.kv_heads};
    const int64_t table = s.max_pages == 0 ? 0
        : 4 * ((s.batch > 1 ? (s.batch - 1) * s.table_stride : 0) + s.max_pages);
    const int64_t b = s.batch;
    const Span spans[10] = {
        {query, strided_extent(rows, s.q_stride, 3, s.d_head), 16, false},
        {key_pages, strided_extent(pages, s.k_stride, 3, s.d_head), 16, false},
        {value_pages, strided_extent(pages, s.v_stride, 3, s.d_head), 16, false},
        {page_table, table, 4, false},
        {lengths, 4 * b, 4, false},
        {new_lengths, new_lengths ? 4 * b : 0, 4, false},
        {mask, mask_bytes, 1, false},
        {out, strided_extent(rows, s.o_stride, 3, s.d_head), 16, true},
        {lse, lse ? 4 * b * s.new_tokens * s.heads : 0, 4, true},
        {workspace, need, 16, true}};
    if (spans[7].bytes > 0 && overlaps_itself(rows, s.o_stride, 3, s.d_head))
        return CS_ERR_INVALID_ARG;
    return check_spans(spans, 10);
}

cs_status check_write_shape(const cs_write_shape* s) {
    if (!s) return CS_ERR_INVALID_ARG;
    if (s->batch < 0 || s->new_tokens < 0 || s->kv_heads < 1 || s->d_head < 1 ||
        s->page_size < 1 || s->num_pages < 0)
        return CS_ERR_DIM_MISMATCH;
    if (s->d_head > cs::kPagedMaxDHead) return CS_ERR_OOM;
    if (s->d_head % 8 != 0) return CS_ERR_INVALID_ARG;
    const int64_t tokens = static_cast<int64_t>(s->batch) * s->new_tokens;
    if (s->kv_heads > cs::kFattnMaxHeads || tokens > (1 << 30)) return CS_ERR_DIM_MISMATCH;
    return CS_OK;
}

// Whether a call may write these pages: rows that share no element, and keys
// and values that share none, also side by side in one buffer.
bool separate_pages(const int64_t* dim, const int64_t* k_stride, const int64_t* v_stride,
                    const uint16_t* k, const uint16_t* v, int64_t k_bytes, int64_t v_bytes,
                    int32_t d) {
    if (overlaps_itself(dim, k_stride, 3, d) || overlaps_itself(dim, v_stride, 3, d)) return false;
    if (!ranges_overlap(k, k_bytes, v, v_bytes)) return true;
    for (int i = 0; i < 3; ++i)
        if (dim[i] > 1 && k_stride[i] != v_stride[i]) return false;
    const int64_t apart = k < v ? v - k : k - v;
    const int64_t dims[4] = {dim[0], dim[1], dim[2], 2};
    const int64_t strides[4] = {k_stride[0], k_stride[1], k_stride[2], apart};
    return !overlaps_itself(dims, strides, 4, d);
}

}  // namespace

extern "C" {

cs_status cs_check_args(const float* logits, const float* out, int64_t batch,
                        int32_t num_classes, float entropy_bound, float t_min,
                        float t_max, int32_t max_iter, const float* t_out) {
    return check_forward_args(logits, out, batch, num_classes, entropy_bound,
                              t_min, t_max, max_iter, t_out, 4);
}

cs_status cs_check_args_bf16(const uint16_t* logits, const float* out,
                             int64_t batch, int32_t num_classes,
                             float entropy_bound, float t_min, float t_max,
                             int32_t max_iter, const float* t_out) {
    return check_forward_args(logits, out, batch, num_classes, entropy_bound,
                              t_min, t_max, max_iter, t_out, 2);
}

cs_status cs_plan_host(int64_t batch, int32_t num_classes,
                       const cs_options* options, int32_t sm_count,
                       int32_t smem_per_block_optin, int32_t smem_per_sm,
                       int32_t max_cluster, cs_plan* plan) {
    if (!plan) return CS_ERR_INVALID_ARG;
    if (batch < 0 || num_classes < 1) return CS_ERR_DIM_MISMATCH;
    if (num_classes > CS_MAX_NUM_CLASSES) return CS_ERR_OOM;
    if (sm_count < 1 || smem_per_block_optin < 1 || smem_per_sm < 1 ||
        max_cluster < 1)
        return CS_ERR_INVALID_ARG;
    if (max_cluster > cs::kMaxCluster) max_cluster = cs::kMaxCluster;
    cs_options o = options ? *options : cs_options{};
    if (o.variant == CS_VARIANT_AUTO) {
        if (o.param != 0) return CS_ERR_INVALID_ARG;
        o.variant = num_classes <= kAutoRowgroupMaxClassesFwd ? CS_VARIANT_ROWGROUP
                                                              : CS_VARIANT_CLUSTER;
    }
    if (o.variant == CS_VARIANT_ROWGROUP) {
        if (o.threads != 0 || (o.strict != 0 && o.strict != 1))
            return CS_ERR_INVALID_ARG;
        return plan_rowgroup(batch, num_classes, o.param, plan);
    }
    if (o.variant == CS_VARIANT_CLUSTER)
        return plan_cluster(batch, num_classes, o, sm_count,
                            smem_per_block_optin, smem_per_sm, max_cluster,
                            plan);
    return CS_ERR_INVALID_ARG;
}

cs_status cs_plan_launch(int64_t batch, int32_t num_classes,
                         const cs_options* options, cs_plan* plan) {
    DeviceInfo* d = nullptr;
    const cs_status st = device_info(&d);
    if (st != CS_OK) return st;
    return cs_plan_host(batch, num_classes, options, d->sm_count,
                        d->smem_optin, d->smem_per_sm, d->max_cluster, plan);
}

cs_status cs_constrained_softmax_ex(const float* logits, float* out,
                                    int64_t batch, int32_t num_classes,
                                    float entropy_bound, float t_min,
                                    float t_max, int32_t max_iter,
                                    float* t_out, const cs_options* options,
                                    void* stream) {
    return forward(logits, false, out, batch, num_classes, entropy_bound,
                   t_min, t_max, max_iter, t_out, options, stream);
}

cs_status cs_constrained_softmax(const float* logits, float* out,
                                 int64_t batch, int32_t num_classes,
                                 float entropy_bound, float t_min, float t_max,
                                 int32_t max_iter, float* t_out, void* stream) {
    return forward(logits, false, out, batch, num_classes, entropy_bound,
                   t_min, t_max, max_iter, t_out, nullptr, stream);
}

cs_status cs_constrained_softmax_bf16_ex(const uint16_t* logits, float* out,
                                         int64_t batch, int32_t num_classes,
                                         float entropy_bound, float t_min,
                                         float t_max, int32_t max_iter,
                                         float* t_out,
                                         const cs_options* options,
                                         void* stream) {
    return forward(logits, true, out, batch, num_classes, entropy_bound,
                   t_min, t_max, max_iter, t_out, options, stream);
}

cs_status cs_constrained_softmax_bf16(const uint16_t* logits, float* out,
                                      int64_t batch, int32_t num_classes,
                                      float entropy_bound, float t_min,
                                      float t_max, int32_t max_iter,
                                      float* t_out, void* stream) {
    return forward(logits, true, out, batch, num_classes, entropy_bound,
                   t_min, t_max, max_iter, t_out, nullptr, stream);
}

cs_status cs_get_error(int32_t* code_mask, void* stream) {
    if (!code_mask) return CS_ERR_INVALID_ARG;
    DeviceInfo* d = nullptr;
    const cs_status st = device_info(&d);
    if (st != CS_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int h = 0;
    // Read and clear in one atomic exchange on the device, so that a bit a
    // launch on another stream sets at the same time is never dropped.
    std::lock_guard<std::mutex> lock(d->take_mu);
    if (cs::launch_take_error(d->err, d->err_taken, s) != cudaSuccess ||
        cudaMemcpyAsync(&h, d->err_taken, sizeof(h), cudaMemcpyDeviceToHost,
                        s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    *code_mask = static_cast<int32_t>(h);
    return CS_OK;
}

cs_status cs_check_backward_args(const float* probs, const float* grad_out,
                                 const float* t, const float* grad_in,
                                 int64_t batch, int32_t num_classes) {
    if (batch < 0 || num_classes < 1) return CS_ERR_DIM_MISMATCH;
    if (num_classes > CS_MAX_NUM_CLASSES) return CS_ERR_OOM;
    if (batch > INT64_MAX / 4 / num_classes) return CS_ERR_DIM_MISMATCH;
    if (batch == 0) return CS_OK;
    if (!probs || !grad_out || !t || !grad_in) return CS_ERR_INVALID_ARG;
    const int64_t bytes = batch * num_classes * 4;
    if (grad_in != probs && ranges_overlap(grad_in, bytes, probs, bytes))
        return CS_ERR_INVALID_ARG;
    if (grad_in != grad_out && ranges_overlap(grad_in, bytes, grad_out, bytes))
        return CS_ERR_INVALID_ARG;
    if (ranges_overlap(t, batch * 4, grad_in, bytes)) return CS_ERR_INVALID_ARG;
    return CS_OK;
}

cs_status cs_plan_backward_host(int64_t batch, int32_t num_classes,
                                const cs_options* options, int32_t sm_count,
                                int32_t smem_per_block_optin,
                                int32_t smem_per_sm, int32_t max_cluster,
                                cs_plan* plan) {
    if (!plan) return CS_ERR_INVALID_ARG;
    if (batch < 0 || num_classes < 1) return CS_ERR_DIM_MISMATCH;
    if (num_classes > CS_MAX_NUM_CLASSES) return CS_ERR_OOM;
    if (sm_count < 1 || smem_per_block_optin < 1 || smem_per_sm < 1 ||
        max_cluster < 1)
        return CS_ERR_INVALID_ARG;
    if (max_cluster > cs::kMaxCluster) max_cluster = cs::kMaxCluster;
    cs_options o = options ? *options : cs_options{};
    if (o.strict != 0 || o.evals_out) return CS_ERR_INVALID_ARG;
    if (o.variant == CS_VARIANT_AUTO) {
        if (o.param != 0 || o.threads != 0) return CS_ERR_INVALID_ARG;
        o.variant = num_classes <= kAutoRowgroupMaxClasses ? CS_VARIANT_ROWGROUP
                                                           : CS_VARIANT_CLUSTER;
    }
    if (o.variant == CS_VARIANT_ROWGROUP) {
        if (o.threads != 0) return CS_ERR_INVALID_ARG;
        return plan_backward_rowgroup(batch, num_classes, o.param, plan);
    }
    if (o.variant == CS_VARIANT_CLUSTER)
        return plan_backward_cluster(batch, num_classes, o, sm_count,
                                     smem_per_block_optin, smem_per_sm,
                                     max_cluster, plan);
    return CS_ERR_INVALID_ARG;
}

cs_status cs_plan_backward_launch(int64_t batch, int32_t num_classes,
                                  const cs_options* options, cs_plan* plan) {
    DeviceInfo* d = nullptr;
    const cs_status st = device_info(&d);
    if (st != CS_OK) return st;
    return cs_plan_backward_host(batch, num_classes, options, d->sm_count,
                                 d->smem_optin, d->smem_per_sm,
                                 d->max_cluster, plan);
}

cs_status cs_constrained_softmax_backward_ex(const float* probs,
                                             const float* grad_out,
                                             const float* t, float* grad_in,
                                             int64_t batch,
                                             int32_t num_classes,
                                             const cs_options* options,
                                             void* stream) {
    cs_status st = cs_check_backward_args(probs, grad_out, t, grad_in, batch,
                                          num_classes);
    if (st != CS_OK) return st;
    if (batch == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs_plan p;
    st = cs_plan_backward_host(batch, num_classes, options, d->sm_count,
                               d->smem_optin, d->smem_per_sm, d->max_cluster,
                               &p);
    if (st != CS_OK) return st;
    cs::BwdTask task;
    task.probs = probs;
    task.grad_out = grad_out;
    task.t = t;
    task.grad_in = grad_in;
    task.batch = batch;
    task.num_classes = num_classes;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.variant == CS_VARIANT_ROWGROUP) {
        e = cs::launch_backward_rowgroup(task, p.lanes_per_row,
                                         p.elems_per_lane, s);
    } else {
        e = cs::launch_backward_cluster(task, p.cluster_size, p.slice_len,
                                        p.threads_per_cta, p.smem_bytes,
                                        p.staged_tensors == 2, p.grid_ctas, s);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

cs_status cs_constrained_softmax_backward(const float* probs,
                                          const float* grad_out,
                                          const float* t, float* grad_in,
                                          int64_t batch, int32_t num_classes,
                                          void* stream) {
    return cs_constrained_softmax_backward_ex(probs, grad_out, t, grad_in,
                                              batch, num_classes, nullptr,
                                              stream);
}

cs_status cs_check_attention_args(const float* scores, const float* out,
                                  const float* mask, int32_t batch,
                                  int32_t heads, int32_t seq_len,
                                  int32_t causal) {
    if (batch < 0 || heads < 0 || seq_len < 0) return CS_ERR_DIM_MISMATCH;
    if (causal != 0 && causal != 1) return CS_ERR_INVALID_ARG;
    if (seq_len > CS_MAX_SEQ_LEN) return CS_ERR_OOM;
    const int64_t rows = static_cast<int64_t>(batch) * heads * seq_len;
    if (rows == 0) return CS_OK;
    if (rows > INT64_MAX / 4 / seq_len) return CS_ERR_DIM_MISMATCH;
    if (!scores || !out) return CS_ERR_INVALID_ARG;
    const int64_t bytes = rows * seq_len * 4;
    if (out != scores && ranges_overlap(out, bytes, scores, bytes))
        return CS_ERR_INVALID_ARG;
    if (mask && ranges_overlap(mask, static_cast<int64_t>(batch) * seq_len * 4,
                               out, bytes))
        return CS_ERR_INVALID_ARG;
    return CS_OK;
}

cs_status cs_plan_attention_host(int32_t batch, int32_t heads,
                                 int32_t seq_len, int32_t aligned,
                                 const cs_options* options, int32_t sm_count,
                                 int32_t smem_per_block_optin,
                                 int32_t smem_per_sm, cs_plan* plan) {
    if (!plan) return CS_ERR_INVALID_ARG;
    if (batch < 0 || heads < 0 || seq_len < 1) return CS_ERR_DIM_MISMATCH;
    if (seq_len > CS_MAX_SEQ_LEN) return CS_ERR_OOM;
    if (aligned != 0 && aligned != 1) return CS_ERR_INVALID_ARG;
    if (sm_count < 1 || smem_per_block_optin < 1 || smem_per_sm < 1)
        return CS_ERR_INVALID_ARG;
    const cs_options o = options ? *options : cs_options{};
    return plan_attention(batch, heads, seq_len, aligned, o, sm_count,
                          smem_per_block_optin, smem_per_sm, plan);
}

cs_status cs_plan_attention_launch(int32_t batch, int32_t heads,
                                   int32_t seq_len, int32_t aligned,
                                   const cs_options* options, cs_plan* plan) {
    DeviceInfo* d = nullptr;
    const cs_status st = device_info(&d);
    if (st != CS_OK) return st;
    return cs_plan_attention_host(batch, heads, seq_len, aligned, options,
                                  d->sm_count, d->smem_optin, d->smem_per_sm,
                                  plan);
}

cs_status cs_attention_softmax_ex(const float* scores, float* out,
                                  const float* mask, int32_t batch,
                                  int32_t heads, int32_t seq_len,
                                  int32_t causal, const cs_options* options,
                                  void* stream) {
    cs_status st = cs_check_attention_args(scores, out, mask, batch, heads,
                                           seq_len, causal);
    if (st != CS_OK) return st;
    const int64_t rows = static_cast<int64_t>(batch) * heads * seq_len;
    if (rows == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    const bool aligned = seq_len % 4 == 0 &&
                         (reinterpret_cast<uintptr_t>(scores) & 15) == 0 &&
                         (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    cs_plan p;
    st = cs_plan_attention_host(batch, heads, seq_len, aligned ? 1 : 0,
                                options, d->sm_count, d->smem_optin,
                                d->smem_per_sm, &p);
    if (st != CS_OK) return st;
    cs::AttnTask task;
    task.scores = scores;
    task.out = out;
    task.mask = mask;
    task.err = d->err;
    task.rows = rows;
    task.heads = heads;
    task.seq_len = seq_len;
    task.causal = causal;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.variant == CS_VARIANT_ROWGROUP)
        e = cs::launch_attention_rowgroup(task, p.lanes_per_row,
                                          p.elems_per_lane, s);
    else
        e = cs::launch_attention_cta(task, p.threads_per_cta, p.smem_bytes,
                                     p.grid_ctas, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

cs_status cs_attention_softmax(const float* scores, float* out,
                               const float* mask, int32_t batch,
                               int32_t heads, int32_t seq_len,
                               int32_t causal, void* stream) {
    return cs_attention_softmax_ex(scores, out, mask, batch, heads, seq_len,
                                   causal, nullptr, stream);
}

cs_status cs_check_biencoder_args(const float* query,
                                  const float* context_keys,
                                  const float* context_values,
                                  const float* output, int32_t batch_size,
                                  int32_t query_len, int32_t context_len,
                                  int32_t d_head, int32_t num_heads,
                                  float scale, float entropy_bound,
                                  float t_min, float t_max, int32_t max_iter,
                                  const float* attn_out, const float* t_out) {
    if (batch_size < 0 || query_len < 0 || num_heads < 0 || context_len < 1 ||
        d_head < 1)
        return CS_ERR_DIM_MISMATCH;
    if (context_len > cs::kBiencMaxContext || d_head > cs::kBiencMaxDHead)
        return CS_ERR_OOM;
    if (d_head % 4 != 0) return CS_ERR_INVALID_ARG;
    if (!isfinite(scale)) return CS_ERR_INVALID_ARG;
    // The search parameters, as for cs_constrained_softmax.
    const cs_status st = cs_check_args(nullptr, nullptr, 0, context_len,
                                       entropy_bound, t_min, t_max, max_iter,
                                       nullptr);
    if (st != CS_OK) return st;
    const int64_t bh = static_cast<int64_t>(batch_size) * num_heads;
    const int64_t rows = bh * query_len;
    if (rows == 0) return CS_OK;
    if (!query || !context_keys || !context_values || !output)
        return CS_ERR_INVALID_ARG;
    const void* ptrs[4] = {query, context_keys, context_values, output};
    for (const void* ptr : ptrs)
        if (reinterpret_cast<uintptr_t>(ptr) & 15) return CS_ERR_INVALID_ARG;
    const int64_t qb = rows * d_head * 4;
    const int64_t kb = bh * context_len * d_head * 4;
    if (ranges_overlap(output, qb, query, qb) ||
        ranges_overlap(output, qb, context_keys, kb) ||
        ranges_overlap(output, qb, context_values, kb))
        return CS_ERR_INVALID_ARG;
    const int64_t ab = rows * context_len * 4;
    if (attn_out && (ranges_overlap(attn_out, ab, output, qb) ||
                     ranges_overlap(attn_out, ab, query, qb) ||
                     ranges_overlap(attn_out, ab, context_keys, kb) ||
                     ranges_overlap(attn_out, ab, context_values, kb)))
        return CS_ERR_INVALID_ARG;
    if (t_out && (ranges_overlap(t_out, rows * 4, output, qb) ||
                  ranges_overlap(t_out, rows * 4, query, qb) ||
                  ranges_overlap(t_out, rows * 4, context_keys, kb) ||
                  ranges_overlap(t_out, rows * 4, context_values, kb) ||
                  (attn_out && ranges_overlap(t_out, rows * 4, attn_out, ab))))
        return CS_ERR_INVALID_ARG;
    return CS_OK;
}

cs_status cs_plan_biencoder_host(int32_t batch_size, int32_t query_len,
                                 int32_t context_len, int32_t d_head,
                                 int32_t num_heads, const cs_options* options,
                                 int32_t smem_per_block_optin, cs_plan* plan) {
    if (!plan) return CS_ERR_INVALID_ARG;
    if (batch_size < 0 || query_len < 0 || num_heads < 0 || context_len < 1 ||
        d_head < 1)
        return CS_ERR_DIM_MISMATCH;
    if (context_len > cs::kBiencMaxContext || d_head > cs::kBiencMaxDHead)
        return CS_ERR_OOM;
    if (d_head % 4 != 0) return CS_ERR_INVALID_ARG;
    const cs_options o = options ? *options : cs_options{};
    if (o.threads != 0 || o.strict != 0 || o.evals_out) return CS_ERR_INVALID_ARG;
    // G lanes a query row, each holding `keys` context items: by default
    // sixteen (the fewest lanes, so the fewest copies of each row's search
    // bookkeeping); a forced G holds eight when that covers the context.
    int G = 0;
    if (o.variant == CS_VARIANT_AUTO ||
        (o.variant == CS_VARIANT_FUSED && o.param == 0)) {
        if (o.param != 0) return CS_ERR_INVALID_ARG;
        G = 1;
        while (16 * G < context_len) G <<= 1;
    } else if (o.variant == CS_VARIANT_ROWGROUP || o.variant == CS_VARIANT_FUSED) {
        G = o.param;
        if (G < 1 || G > kRowgroupMaxLanes || (G & (G - 1)))
            return CS_ERR_INVALID_ARG;
        if (16 * G < context_len) return CS_ERR_OOM;
    } else {
        return CS_ERR_INVALID_ARG;
    }
    const int keys = (o.variant == CS_VARIANT_AUTO ||
                      (o.variant == CS_VARIANT_FUSED && o.param == 0) ||
                      8 * G < context_len) ? 16 : 8;
    // Step 3 on the tensor cores (a second kernel) unless forced fused:
    // for head sizes up to kPvMaxD and contexts no longer than the head, so
    // that the weights fit in the output's own rows when attn_out is not
    // requested.
    const bool tc = o.variant != CS_VARIANT_FUSED && d_head <= cs::kPvMaxD &&
                    context_len <= d_head &&
                    cs::pv_smem_bytes(context_len, d_head) <= smem_per_block_optin;
    const int64_t smem = tc ? cs::bienc_search_smem_bytes(context_len, d_head, G)
                            : cs::bienc_smem_bytes(context_len, d_head, G);
    if (smem > smem_per_block_optin) return CS_ERR_OOM;
    const int64_t rows_per_tile = cs::bienc_threads(G) / G;
    const int64_t tiles = ceil_div(query_len, rows_per_tile);
    const int64_t per = cs::bienc_tiles_per_cta(query_len, G);
    const int64_t grid = static_cast<int64_t>(batch_size) * num_heads *
                         ceil_div(tiles, per);
    if (grid > kMaxGridX) return CS_ERR_DIM_MISMATCH;
    *plan = cs_plan{};
    plan->variant = CS_VARIANT_ROWGROUP;
    plan->lanes_per_row = G;
    plan->elems_per_lane = keys;
    plan->threads_per_cta = cs::bienc_threads(G);
    plan->smem_bytes = static_cast<int32_t>(smem);
    plan->grid_ctas = grid;
    plan->staged_tensors = tc ? 2 : 3;
    plan->tensor_cores = tc ? 1 : 0;
    return CS_OK;
}

cs_status cs_biencoder_attention_ex(const float* query,
                                    const float* context_keys,
                                    const float* context_values,
                                    float* output, int32_t batch_size,
                                    int32_t query_len, int32_t context_len,
                                    int32_t d_head, int32_t num_heads,
                                    float scale, float entropy_bound,
                                    float t_min, float t_max,
                                    int32_t max_iter, float* attn_out,
                                    float* t_out, const cs_options* options,
                                    void* stream) {
    cs_status st = cs_check_biencoder_args(
        query, context_keys, context_values, output, batch_size, query_len,
        context_len, d_head, num_heads, scale, entropy_bound, t_min, t_max,
        max_iter, attn_out, t_out);
    if (st != CS_OK) return st;
    const int64_t bh = static_cast<int64_t>(batch_size) * num_heads;
    if (bh * query_len == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs_plan p;
    st = cs_plan_biencoder_host(batch_size, query_len, context_len, d_head,
                                num_heads, options, d->smem_optin, &p);
    if (st != CS_OK) return st;
    cs::BiencTask task;
    task.q = query;
    task.k = context_keys;
    task.v = context_values;
    task.out = output;
    task.attn_out = attn_out;
    task.t_out = t_out;
    task.err = d->err;
    task.BH = static_cast<int32_t>(bh);
    task.Q = query_len;
    task.K = context_len;
    task.D = d_head;
    task.scale = scale;
    task.entropy_bound = entropy_bound;
    task.t_min = t_min;
    task.hi0 = t_max < 1.0f ? t_max : 1.0f;
    task.max_iter = max_iter;
    task.p_out = nullptr;
    task.p_stride = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.tensor_cores) {
        // Steps 1-2 write the weights (to attn_out, or to the first
        // context_len floats of each output row), then the tensor-core
        // kernel turns them into the output on the same stream.
        task.p_out = attn_out ? attn_out : output;
        task.p_stride = attn_out ? context_len : d_head;
        e = cs::launch_bienc(task, p.lanes_per_row, p.elems_per_lane, p.smem_bytes, s);
        if (e == cudaSuccess) {
            cs::PvTask pv;
            pv.p = task.p_out;
            pv.p_stride = task.p_stride;
            pv.v = context_values;
            pv.out = output;
            pv.err = d->err;
            pv.BH = task.BH;
            pv.Q = query_len;
            pv.K = context_len;
            pv.D = d_head;
            pv.wait_limit_cycles = cs::kWaitLimitCycles;
            e = cs::launch_bienc_pv(pv, d->sm_count, s);
        }
    } else {
        e = cs::launch_bienc(task, p.lanes_per_row, p.elems_per_lane, p.smem_bytes, s);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

cs_status cs_biencoder_attention(const float* query,
                                 const float* context_keys,
                                 const float* context_values, float* output,
                                 int32_t batch_size, int32_t query_len,
                                 int32_t context_len, int32_t d_head,
                                 int32_t num_heads, float scale,
                                 float entropy_bound, void* stream) {
    return cs_biencoder_attention_ex(query, context_keys, context_values,
                                     output, batch_size, query_len,
                                     context_len, d_head, num_heads, scale,
                                     entropy_bound, 0.01f, 10.0f, 20, nullptr,
                                     nullptr, nullptr, stream);
}

cs_status cs_check_fused_attention_args(const uint16_t* query,
                                        const uint16_t* keys,
                                        const uint16_t* values,
                                        const uint16_t* out, const float* lse,
                                        const uint8_t* mask,
                                        const cs_attention_shape* shape) {
    const cs_status st = check_attention_shape(shape);
    if (st != CS_OK) return st;
    const cs_attention_shape& s = *shape;
    const int64_t rows = static_cast<int64_t>(s.batch) * s.heads * s.query_len;
    const Span spans[6] = {
        {query, heads_extent(s, s.heads, s.query_len, s.q_stride), 16, false},
        {keys, heads_extent(s, s.kv_heads, s.key_len, s.k_stride), 16, false},
        {values, heads_extent(s, s.kv_heads, s.key_len, s.v_stride), 16, false},
        {mask, mask_extent(s, mask), 1, false},
        {out, heads_extent(s, s.heads, s.query_len, s.o_stride, true), 16, true},
        {lse, lse ? rows * 4 : 0, 4, true}};
    return check_spans(spans, 6);
}

cs_status cs_fused_attention(const uint16_t* query, const uint16_t* keys,
                             const uint16_t* values, uint16_t* out,
                             float* lse, const uint8_t* mask,
                             const cs_attention_shape* shape, void* stream) {
    cs_status st = cs_check_fused_attention_args(query, keys, values, out, lse,
                                                 mask, shape);
    if (st != CS_OK) return st;
    if (shape->batch == 0 || shape->query_len == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs::FattnTask t = attention_task(*shape, mask, *d);
    t.q = query;
    t.k = keys;
    t.v = values;
    t.out = out;
    t.lse = lse;
    if (cs::launch_fattn_forward(t, static_cast<cudaStream_t>(stream)) !=
        cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

int64_t cs_fused_attention_backward_workspace(const cs_attention_shape* shape) {
    if (check_attention_shape(shape) != CS_OK) return -1;
    return 4 * cs::fattn_workspace_floats(shape->batch, shape->heads,
                                          shape->query_len);
}

cs_status cs_check_fused_attention_backward_args(
    const uint16_t* query, const uint16_t* keys, const uint16_t* values,
    const uint16_t* out, const float* lse, const uint16_t* grad_out,
    const uint16_t* grad_query, const uint16_t* grad_keys,
    const uint16_t* grad_values, const uint8_t* mask,
    const cs_attention_shape* shape, const void* workspace,
    int64_t workspace_bytes) {
    const cs_status st = check_attention_shape(shape);
    if (st != CS_OK) return st;
    const cs_attention_shape& s = *shape;
    const int64_t rows = static_cast<int64_t>(s.batch) * s.heads * s.query_len;
    const int64_t need = cs_fused_attention_backward_workspace(shape);
    if (workspace_bytes < need) return CS_ERR_INVALID_ARG;
    const Span spans[11] = {
        {query, heads_extent(s, s.heads, s.query_len, s.q_stride), 16, false},
        {keys, heads_extent(s, s.kv_heads, s.key_len, s.k_stride), 16, false},
        {values, heads_extent(s, s.kv_heads, s.key_len, s.v_stride), 16, false},
        {out, heads_extent(s, s.heads, s.query_len, s.o_stride), 16, false},
        {grad_out, heads_extent(s, s.heads, s.query_len, s.go_stride), 16, false},
        {lse, rows * 4, 4, false},
        {mask, mask_extent(s, mask), 1, false},
        {grad_query, heads_extent(s, s.heads, s.query_len, s.dq_stride, true), 16, true},
        {grad_keys, heads_extent(s, s.kv_heads, s.key_len, s.dk_stride, true), 16, true},
        {grad_values, heads_extent(s, s.kv_heads, s.key_len, s.dv_stride, true), 16, true},
        {workspace, need, 16, true}};
    return check_spans(spans, 11);
}

cs_status cs_fused_attention_backward(
    const uint16_t* query, const uint16_t* keys, const uint16_t* values,
    const uint16_t* out, const float* lse, const uint16_t* grad_out,
    uint16_t* grad_query, uint16_t* grad_keys, uint16_t* grad_values,
    const uint8_t* mask, const cs_attention_shape* shape, void* workspace,
    int64_t workspace_bytes, void* stream) {
    cs_status st = cs_check_fused_attention_backward_args(
        query, keys, values, out, lse, grad_out, grad_query, grad_keys,
        grad_values, mask, shape, workspace, workspace_bytes);
    if (st != CS_OK) return st;
    if (shape->batch == 0 || (shape->query_len == 0 && shape->key_len == 0))
        return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs::FattnTask t = attention_task(*shape, mask, *d);
    t.q = query;
    t.k = keys;
    t.v = values;
    t.out = const_cast<uint16_t*>(out);
    t.lse = const_cast<float*>(lse);
    t.go = grad_out;
    t.dq = grad_query;
    t.dk = grad_keys;
    t.dv = grad_values;
    t.rows = static_cast<float*>(workspace);
    if (cs::launch_fattn_backward(t, static_cast<cudaStream_t>(stream)) !=
        cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

int64_t cs_paged_attention_workspace(const cs_paged_shape* shape) {
    if (check_paged_shape(shape) != CS_OK) return -1;
    // Two parts a CTA, of 16 heads: the (maximum, sum) pairs, the outputs.
    const int64_t heads = paged_groups(*shape, kPagedMaxSms) * paged_rows(*shape) * 2 * 16;
    return heads * 8 + heads * shape->d_head * 4;
}

cs_status cs_check_paged_attention_args(
    const uint16_t* query, const uint16_t* key_pages,
    const uint16_t* value_pages, const int32_t* page_table,
    const int32_t* lengths, const uint16_t* out, const float* lse,
    const cs_paged_shape* shape, const void* workspace,
    int64_t workspace_bytes) {
    const cs_status st = check_paged_shape(shape);
    if (st != CS_OK) return st;
    const cs_paged_shape& s = *shape;
    if (s.batch == 0) return CS_OK;
    // Steps and CTAs are counted in 32 bits.
    if (paged_steps(s) * s.batch > (1 << 30) || paged_rows(s) * s.batch > (1 << 30))
        return CS_ERR_DIM_MISMATCH;
    const int64_t need = cs_paged_attention_workspace(shape);
    if (workspace_bytes < need) return CS_ERR_INVALID_ARG;
    if (s.batch > 1 && (s.table_stride < s.max_pages || s.table_stride > kMaxRowStride))
        return CS_ERR_INVALID_ARG;
    const int64_t rows[2] = {s.batch, s.heads};
    const int64_t pages[3] = {s.num_pages, s.page_size, s.kv_heads};
    const int64_t table = s.max_pages == 0 ? 0
        : 4 * ((s.batch > 1 ? (s.batch - 1) * s.table_stride : 0) + s.max_pages);
    const Span spans[8] = {
        {query, strided_extent(rows, s.q_stride, 2, s.d_head), 16, false},
        {key_pages, strided_extent(pages, s.k_stride, 3, s.d_head), 16, false},
        {value_pages, strided_extent(pages, s.v_stride, 3, s.d_head), 16, false},
        {page_table, table, 4, false},
        {lengths, 4 * static_cast<int64_t>(s.batch), 4, false},
        {out, strided_extent(rows, s.o_stride, 2, s.d_head), 16, true},
        {lse, lse ? 4 * static_cast<int64_t>(s.batch) * s.heads : 0, 4, true},
        {workspace, need, 16, true}};
    if (spans[5].bytes > 0 && overlaps_itself(rows, s.o_stride, 2, s.d_head))
        return CS_ERR_INVALID_ARG;
    return check_spans(spans, 8);
}

cs_status cs_paged_attention(const uint16_t* query, const uint16_t* key_pages,
                             const uint16_t* value_pages,
                             const int32_t* page_table,
                             const int32_t* lengths, uint16_t* out,
                             float* lse, const cs_paged_shape* shape,
                             void* workspace, int64_t workspace_bytes,
                             void* stream) {
    cs_status st = cs_check_paged_attention_args(
        query, key_pages, value_pages, page_table, lengths, out, lse, shape,
        workspace, workspace_bytes);
    if (st != CS_OK) return st;
    const cs_paged_shape& s = *shape;
    if (s.batch == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs::PagedTask t{};
    t.q = query;
    t.k_pages = key_pages;
    t.v_pages = value_pages;
    t.page_table = page_table;
    t.lengths = lengths;
    t.out = out;
    t.lse = lse;
    t.err = d->err;
    for (int i = 0; i < 2; ++i) {
        t.q_stride[i] = s.q_stride[i];
        t.o_stride[i] = s.o_stride[i];
    }
    for (int i = 0; i < 3; ++i) {
        t.k_stride[i] = s.k_stride[i];
        t.v_stride[i] = s.v_stride[i];
    }
    t.table_stride = s.table_stride;
    t.batch = s.batch;
    t.heads = s.heads;
    t.kv_heads = s.kv_heads;
    t.d_head = s.d_head;
    t.page_size = s.page_size;
    t.num_pages = s.num_pages;
    t.max_pages = s.max_pages;
    t.head_tiles = paged_head_tiles(s);
    t.groups = static_cast<int32_t>(
        paged_groups(s, d->sm_count < kPagedMaxSms ? d->sm_count : kPagedMaxSms));
    t.split = t.groups > 0;
    t.fp16 = s.fp16;
    t.scale = s.scale;
    if (t.split) {
        t.part_stats = static_cast<float2*>(workspace);
        t.part_out = reinterpret_cast<float*>(t.part_stats +
                                              t.groups * paged_rows(s) * 2 * 16);
    }
    if (cs::launch_paged(t, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

cs_status cs_check_paged_extend_args(
    const int32_t* page_table, const int32_t* lengths, const int32_t* new_lengths,
    const int32_t* held, const int32_t* free_pages, const int32_t* cursor, const int64_t* slots,
    const int32_t* totals, const int32_t* held_out, const int32_t* cursor_out,
    const cs_extend_shape* shape) {
    if (!shape) return CS_ERR_INVALID_ARG;
    const cs_extend_shape& s = *shape;
    if (s.batch < 0 || s.max_new < 0 || s.max_pages < 0 || s.page_size < 1 || s.num_free < 0 ||
        s.batch > cs::kFattnMaxBatch || s.max_new > kPagedMaxTokens ||
        static_cast<int64_t>(s.max_pages) * s.page_size > kPagedMaxTokens ||
        static_cast<int64_t>(s.batch) * s.max_new > (int64_t(1) << 40))
        return CS_ERR_DIM_MISMATCH;
    if (s.batch > 1 && (s.table_stride < s.max_pages || s.table_stride > kMaxRowStride))
        return CS_ERR_INVALID_ARG;
    const int64_t b = s.batch;
    const int64_t table = b == 0 || s.max_pages == 0 ? 0
        : 4 * ((b > 1 ? (b - 1) * s.table_stride : 0) + s.max_pages);
    const Span spans[10] = {
        {page_table, table, 4, true},
        {lengths, 4 * b, 4, false},
        {new_lengths, 4 * b, 4, false},
        {held, held ? 4 * b : 0, 4, false},
        {free_pages, 4 * static_cast<int64_t>(s.num_free), 4, false},
        {cursor, cursor ? 4 : 0, 4, false},
        {slots, 8 * b * s.max_new, 8, true},
        {totals, 4 * b, 4, true},
        {held_out, 4 * b, 4, true},
        {cursor_out, 4, 4, true}};
    return check_spans(spans, 10);
}

cs_status cs_paged_extend(int32_t* page_table, const int32_t* lengths,
                          const int32_t* new_lengths, const int32_t* held,
                          const int32_t* free_pages, const int32_t* cursor, int64_t* slots,
                          int32_t* totals, int32_t* held_out, int32_t* cursor_out,
                          const cs_extend_shape* shape, void* stream) {
    cs_status st = cs_check_paged_extend_args(page_table, lengths, new_lengths, held, free_pages,
                                              cursor, slots, totals, held_out, cursor_out, shape);
    if (st != CS_OK) return st;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    const cs_extend_shape& s = *shape;
    cs::ExtendTask t{};
    t.page_table = page_table;
    t.lengths = lengths;
    t.new_lengths = new_lengths;
    t.held = held;
    t.free_pages = free_pages;
    t.cursor = cursor;
    t.slots = reinterpret_cast<long long*>(slots);
    t.sm_count = d->sm_count;
    t.totals = totals;
    t.held_out = held_out;
    t.cursor_out = cursor_out;
    t.err = d->err;
    t.table_stride = s.table_stride;
    t.batch = s.batch;
    t.max_new = s.max_new;
    t.max_pages = s.max_pages;
    t.page_size = s.page_size;
    t.num_free = s.num_free;
    if (cs::launch_extend(t, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

cs_status cs_check_paged_write_args(const uint16_t* keys, const uint16_t* values,
                                    const int64_t* slots, const uint16_t* key_pages,
                                    const uint16_t* value_pages, const cs_write_shape* shape) {
    const cs_status st = check_write_shape(shape);
    if (st != CS_OK) return st;
    const cs_write_shape& s = *shape;
    const int64_t in[3] = {s.batch, s.new_tokens, s.kv_heads};
    const int64_t pages[3] = {s.num_pages, s.page_size, s.kv_heads};
    if (s.batch == 0 || s.new_tokens == 0) return CS_OK;
    if (s.batch > 1 && (s.slot_stride < s.new_tokens || s.slot_stride > kMaxRowStride))
        return CS_ERR_INVALID_ARG;
    const int64_t slot_bytes =
        8 * ((s.batch > 1 ? (s.batch - 1) * s.slot_stride : 0) + s.new_tokens);
    const int64_t kb = strided_extent(pages, s.k_stride, 3, s.d_head);
    const int64_t vb = strided_extent(pages, s.v_stride, 3, s.d_head);
    const Span keys_of[4] = {{keys, strided_extent(in, s.key_stride, 3, s.d_head), 16, false},
                             {values, strided_extent(in, s.value_stride, 3, s.d_head), 16, false},
                             {slots, slot_bytes, 8, false},
                             {key_pages, kb, 16, true}};
    const Span values_of[4] = {keys_of[0], keys_of[1], keys_of[2], {value_pages, vb, 16, true}};
    cs_status r = check_spans(keys_of, 4);
    if (r == CS_OK) r = check_spans(values_of, 4);
    if (r == CS_OK && kb > 0 &&
        !separate_pages(pages, s.k_stride, s.v_stride, key_pages, value_pages, kb, vb, s.d_head))
        r = CS_ERR_INVALID_ARG;
    return r;
}

cs_status cs_paged_write(const uint16_t* keys, const uint16_t* values, const int64_t* slots,
                         uint16_t* key_pages, uint16_t* value_pages,
                         const cs_write_shape* shape, void* stream) {
    cs_status st = cs_check_paged_write_args(keys, values, slots, key_pages, value_pages, shape);
    if (st != CS_OK) return st;
    const cs_write_shape& s = *shape;
    if (s.batch == 0 || s.new_tokens == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs::WriteTask t{};
    t.keys = keys;
    t.values = values;
    t.slots = slots;
    t.k_pages = key_pages;
    t.v_pages = value_pages;
    t.err = d->err;
    for (int i = 0; i < 3; ++i) {
        t.key_stride[i] = s.key_stride[i];
        t.value_stride[i] = s.value_stride[i];
        t.k_stride[i] = s.k_stride[i];
        t.v_stride[i] = s.v_stride[i];
    }
    t.slot_stride = s.slot_stride;
    t.num_slots = static_cast<int64_t>(s.num_pages) * s.page_size;
    t.new_tokens = s.new_tokens;
    t.page_size = s.page_size;
    t.head_units = s.d_head / 8;
    t.units = s.kv_heads * t.head_units;
    t.tokens = s.batch * s.new_tokens;
    t.sm_count = d->sm_count;
    if (cs::launch_write(t, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

int64_t cs_paged_tree_attention_workspace(const cs_tree_shape* shape) {
    if (check_tree_shape(shape) != CS_OK) return -1;
    return tree_workspace(*shape, tree_plan(*shape, kPagedMaxSms));
}

cs_status cs_check_paged_tree_attention_args(
    const uint16_t* query, const uint16_t* key_pages, const uint16_t* value_pages,
    const int32_t* page_table, const int32_t* lengths, const int32_t* new_lengths,
    const uint8_t* mask, const uint16_t* out, const float* lse, const cs_tree_shape* shape,
    const void* workspace, int64_t workspace_bytes) {
    TreePlan p;
    return check_tree(query, key_pages, value_pages, page_table, lengths, new_lengths, mask, out,
                      lse, shape, workspace, workspace_bytes, p);
}

cs_status cs_paged_tree_attention(const uint16_t* query, const uint16_t* key_pages,
                                  const uint16_t* value_pages, const int32_t* page_table,
                                  const int32_t* lengths, const int32_t* new_lengths,
                                  const uint8_t* mask, uint16_t* out, float* lse,
                                  const cs_tree_shape* shape, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
    TreePlan p;
    cs_status st = check_tree(query, key_pages, value_pages, page_table, lengths, new_lengths, mask,
                              out, lse, shape, workspace, workspace_bytes, p);
    if (st != CS_OK) return st;
    const cs_tree_shape& s = *shape;
    if (s.batch == 0 || s.new_tokens == 0) return CS_OK;
    DeviceInfo* d = nullptr;
    st = device_info(&d);
    if (st != CS_OK) return st;
    cs::TreeTask t{};
    t.q = query;
    t.k_pages = key_pages;
    t.v_pages = value_pages;
    t.page_table = page_table;
    t.lengths = lengths;
    t.new_lengths = new_lengths;
    t.mask = mask;
    t.out = out;
    t.lse = lse;
    t.err = d->err;
    for (int i = 0; i < 3; ++i) {
        t.q_stride[i] = s.q_stride[i];
        t.o_stride[i] = s.o_stride[i];
        t.k_stride[i] = s.k_stride[i];
        t.v_stride[i] = s.v_stride[i];
    }
    t.table_stride = s.table_stride;
    t.mask_stride[0] = s.mask_stride[0];
    t.mask_stride[1] = s.mask_stride[1];
    t.batch = s.batch;
    t.new_tokens = s.new_tokens;
    t.heads = s.heads;
    t.kv_heads = s.kv_heads;
    t.group = s.heads / s.kv_heads;
    t.d_head = s.d_head;
    t.page_size = s.page_size;
    t.num_pages = s.num_pages;
    t.max_pages = s.max_pages;
    if (d->sm_count < kPagedMaxSms) p = tree_plan(s, d->sm_count);
    t.unit_rows = p.unit_rows;
    t.part_rows = p.part_rows;
    t.width = p.width;
    t.bundles = static_cast<int32_t>(p.units / p.width);
    t.groups = p.groups;
    t.split = p.groups > 0;
    t.fp16 = s.fp16;
    t.scale = s.scale;
    t.wait_limit_cycles = cs::kWaitLimitCycles;
    if (t.split) {
        t.part_stats = static_cast<float2*>(workspace);
        t.part_out = reinterpret_cast<float*>(
            t.part_stats + static_cast<int64_t>(p.groups) * p.width * 2 * p.part_rows);
    }
    if (cs::launch_tree(t, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

int32_t cs_probe_ex2_sink_floats(void) {
    DeviceInfo* d = nullptr;
    if (device_info(&d) != CS_OK) return -1;
    return d->sm_count * kProbeBlocksPerSm * kProbeThreads;
}

cs_status cs_probe_ex2(float* sink, int32_t iters, int64_t* ex2_count,
                       void* stream) {
    if (!sink || !ex2_count || iters < 1) return CS_ERR_INVALID_ARG;
    DeviceInfo* d = nullptr;
    const cs_status st = device_info(&d);
    if (st != CS_OK) return st;
    const int blocks = d->sm_count * kProbeBlocksPerSm;
    const cudaError_t e = cs::launch_probe_ex2(
        sink, iters, blocks, kProbeThreads, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    *ex2_count = static_cast<int64_t>(blocks) * kProbeThreads * iters *
                 cs::probe_chains();
    return CS_OK;
}

cs_status cs_test_wait_timeout(int64_t limit_ns, void* stream) {
    if (limit_ns < 1 || limit_ns > 10000000000ll) return CS_ERR_INVALID_ARG;
    DeviceInfo* d = nullptr;
    const cs_status st = device_info(&d);
    if (st != CS_OK) return st;
    // The wait is bounded in SM cycles; 2.07 cycles per ns at GB300's
    // maximum clock (a lower clock only lengthens the wait).
    const uint64_t cycles = static_cast<uint64_t>(limit_ns) * 207 / 100;
    const cudaError_t e = cs::launch_wait_timeout(
        d->err, cycles, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return CS_ERR_CUDA;
    }
    return CS_OK;
}

const char* cs_version(void) { return "1.0.0 sm_103a"; }

const char* cs_status_string(cs_status status) {
    switch (status) {
        case CS_OK: return "success";
        case CS_ERR_NAN_INPUT: return "NaN in input";
        case CS_ERR_INF_INPUT: return "Inf in input";
        case CS_ERR_ENTROPY_OVERFLOW: return "entropy bound unsatisfiable";
        case CS_ERR_DIM_MISMATCH: return "dimension mismatch";
        case CS_ERR_OOM: return "row does not fit the shared-memory plan";
        case CS_ERR_INVALID_ARG: return "invalid argument";
        case CS_ERR_CUDA: return "CUDA error";
        case CS_ERR_TIMEOUT: return "device wait timed out";
        case CS_ERR_BAD_PAGE: return "page or length out of range";
        case CS_ERR_OUT_OF_PAGES: return "no free page left";
        default: return "unknown status";
    }
}

}  // extern "C"
