// Pages and slots for new tokens of a paged key-value cache, and the write of
// their keys and values.
#include "cs_device.cuh"
#include "cs_pages.h"

namespace cs {
namespace {

using namespace csd;

// ------------------------------------------------------------------- extend
// For sequence b with n = lengths[b] tokens, w = new_lengths[b] more and h =
// held[b] pages:
//   need_b = max(0, ceil((n + w) / page) - h),   first_b = sum of need before b,
//   got_b = what of need_b the free list still has from cursor + first_b on,
// the pages of the list's entries cursor + first_b .. go to the table's entries
// h .., and token n + i gets slot table[(n + i) / page] * page + (n + i) % page.
//
// Bound by the slots that it writes, and, for few, by latency: lengths, then
// table entries, then slots are three trips to memory.  Every CTA adds up the
// needs of the sequences before its own, by itself (from caches: nothing waits
// for another CTA, and one launch is enough), and takes the pages straight from
// the free list where another CTA writes them into the table.  On the GPU: one
// token for each of 32 sequences 2.7 us, trees of up to 61 for 256 of them 3.1,
// 512 prompts of up to 4096 tokens, 17 MB of slots, 9.3 (1.8 TB/s: the needs
// before a CTA and the three trips, about 3, and then the instructions of a slot, a
// lookup, a wide multiplication and a store of 8 bytes: the ALU pipe is 51% busy).
constexpr int kExThreads = 256;
constexpr int kExSlots = 2048;
constexpr int kExCtasPerSm = 4;

__device__ __forceinline__ Claim claim_of(const ExtendTask& t, int b) {
    return cs::claim_of(t.lengths[b], t.new_lengths[b], t.held != nullptr,
                        t.held ? t.held[b] : 0, t.max_new, t.max_pages, t.page_size);
}

__global__ void __launch_bounds__(kExThreads) extend_kernel(const ExtendTask t) {
    constexpr int kWarps = kExThreads / 32;
    __shared__ int64_t scan[kWarps];
    struct Row {
        int len, held, total;   // total: tokens with a slot after the call
        int taken, got;         // of the free list: the entry of page `held`
    };
    __shared__ Row rows[kExThreads];
    // Launched while the kernel before ends, as the next one may be.
    allow_next_kernel();
    wait_for_previous_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b0 = blockIdx.y * t.sequences;
    const int nb = min(t.sequences, t.batch - b0);

    // The needs before sequence b0, then those of its own.
    int64_t before = 0;
    for (int b = threadIdx.x; b < b0; b += kExThreads) before += claim_of(t, b).need;
    Claim c{};
    if (threadIdx.x < nb) c = claim_of(t, b0 + threadIdx.x);
    int64_t up = c.need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    __shared__ int64_t own[kWarps];
    if (lane == 31) {
        scan[warp] = before;
        own[warp] = up;
    }
    __syncthreads();
    int64_t first = up - c.need, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        first += scan[w] + (w < warp ? own[w] : 0);
        all += scan[w] + own[w];
    }
    int cursor = t.cursor ? *t.cursor : 0;
    const bool bad_cursor = cursor < 0 || cursor > t.num_free;
    cursor = min(max(cursor, 0), t.num_free);
    const int64_t left = t.num_free - cursor;
    if (threadIdx.x < nb) {
        const int64_t rest = left - first;
        const int got = static_cast<int>(rest < 0 ? 0 : rest < c.need ? rest : c.need);
        const int have = c.held + got;
        const int64_t room = static_cast<int64_t>(have) * t.page_size;
        const int64_t want = static_cast<int64_t>(c.len) + c.fresh;
        Row r;
        r.len = c.len;
        r.held = c.held;
        r.total = static_cast<int>(c.fresh == 0 ? c.len : want < room ? want : room);
        r.taken = cursor + static_cast<int>(first < left ? first : left);
        r.got = got;
        rows[threadIdx.x] = r;
        if (blockIdx.x == 0) {
            t.totals[b0 + threadIdx.x] = r.total;
            t.held_out[b0 + threadIdx.x] = have;
            unsigned int bits = c.bad || bad_cursor ? kBitBadPage : 0u;
            if (got < c.need) bits |= kBitOutOfPages;
            raise_error(t.err, bits);
        }
    }
    if (blockIdx.x == 0 && b0 + nb == t.batch && threadIdx.x == 0)
        *t.cursor_out = cursor + static_cast<int>(all < left ? all : left);
    __syncthreads();

    // The new pages into the table: a warp a sequence, its CTAs in turn.
    for (int y = warp; y < nb; y += kWarps) {
        const Row r = rows[y];
        for (int i = 32 * blockIdx.x + lane; i < r.got; i += 32 * gridDim.x)
            t.page_table[(b0 + y) * t.table_stride + r.held + i] = t.free_pages[r.taken + i];
    }
    const int i0 = blockIdx.x * t.span;
    const int span = min(t.span, t.max_new - i0);
    // 2^bits threads to a sequence, which step through its places by additions;
    // four places at a time: their pages are all under way before one is used.
    const int step = 1 << t.lane_bits;
    const int skip = step / t.page_size, rest = step - skip * t.page_size;
    for (int y = threadIdx.x >> t.lane_bits; y < nb; y += kExThreads >> t.lane_bits) {
        const Row r = rows[y];
        const int32_t* table = t.page_table + (b0 + y) * t.table_stride;
        const int32_t* fresh = t.free_pages + r.taken;
        long long* out = t.slots + static_cast<int64_t>(b0 + y) * t.max_new + i0;
        const int there = min(r.total - r.len - i0, span);   // places with a slot
        int i = threadIdx.x & (step - 1);
        // (Places past the last slot may lie past 2^31; nothing is read there.)
        const uint32_t place = static_cast<uint32_t>(r.len) + static_cast<uint32_t>(i0 + i);
        const uint32_t size = t.page_size;
        uint32_t entry = place / size;
        uint32_t at = place - entry * size;
        while (i < span) {
            int page[4];
            uint32_t slot[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                page[x] = -1;
                slot[x] = at;
                if (i + x * step < there) {
                    const int e = static_cast<int>(entry);
                    page[x] = e < r.held ? table[e] : fresh[e - r.held];
                }
                entry += skip;
                at += rest;
                if (at >= size) {
                    at -= size;
                    ++entry;
                }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x, i += step) {
                if (i >= span) break;
                if (i < there && page[x] < 0) raise_error(t.err, kBitBadPage);
                __stcs(out + i, page[x] < 0 ? -1ll
                                            : static_cast<long long>(page[x]) * t.page_size +
                                                  slot[x]);
            }
        }
    }
}

// -------------------------------------------------------------------- write
// cache[slots[b][i]] = keys[b][i], values[b][i].  Bound by the bytes of both,
// read and written once.  A CTA takes some tokens, whose rows it looks up first,
// a thread each, and then copies units of 16 bytes, of the key and the value at
// the same place, two at a time, past the caches (nothing is read again here).
// Small CTAs of several rounds: 32 prompts of up to 4096 tokens, 8 heads of 128,
// 403 MB, take 64 us (6.3 TB/s, 93% of a plain copy); one round of 1024 units 74,
// through the caches 81.  A small call has no CTAs to spare for rounds (7 x 333
// tokens of 12 heads of 80, 11 MB: 4.2 us, with four rounds 6.8).
constexpr int kWrThreads = 128;
constexpr int kWrUnroll = 2;
constexpr int kWrUnits = kWrThreads * kWrUnroll;
constexpr int kWrRounds = 4;
constexpr int kWrCtasPerSm = 16;   // from which on rounds are taken

__global__ void __launch_bounds__(kWrThreads) write_kernel(const WriteTask t) {
    // Where a token's rows begin, in elements; dst_k -1: passed over.
    struct Rows {
        int64_t src_k, src_v, dst_k, dst_v;
    };
    __shared__ Rows rows[kWrThreads];
    allow_next_kernel();
    wait_for_previous_kernel();
    const int token0 = blockIdx.x * t.cta_tokens;
    const int n = min(t.cta_tokens, t.tokens - token0);
    if (threadIdx.x < n) {
        const int token = token0 + threadIdx.x;
        const int b = token / t.new_tokens, i = token - b * t.new_tokens;
        const int64_t slot = t.slots[b * t.slot_stride + i];
        Rows r;
        r.dst_k = -1;
        if (slot >= 0 && slot < t.num_slots) {
            int64_t page, at;
            if (t.num_slots <= 0xffffffffll) {   // a division of 32 bits
                const uint32_t x = static_cast<uint32_t>(slot) / static_cast<uint32_t>(t.page_size);
                page = x;
                at = static_cast<uint32_t>(slot) - x * static_cast<uint32_t>(t.page_size);
            } else {
                page = slot / t.page_size;
                at = slot - page * t.page_size;
            }
            r.src_k = b * t.key_stride[0] + i * t.key_stride[1];
            r.src_v = b * t.value_stride[0] + i * t.value_stride[1];
            r.dst_k = page * t.k_stride[0] + at * t.k_stride[1];
            r.dst_v = page * t.v_stride[0] + at * t.v_stride[1];
        } else if (slot >= 0 && blockIdx.y == 0) {
            raise_error(t.err, kBitBadPage);
        }
        rows[threadIdx.x] = r;
    }
    __syncthreads();
    // A token's units, all or (long ones) a slice of them.
    const int u0 = blockIdx.y * t.cta_units;
    const int units = min(t.cta_units, t.units - u0);
    const int total = n * units;
    for (int e0 = threadIdx.x; e0 < total; e0 += kWrUnits) {
        uint4 k[kWrUnroll], v[kWrUnroll];
        int64_t dk[kWrUnroll], dv[kWrUnroll];
#pragma unroll
        for (int x = 0; x < kWrUnroll; ++x) {
            const int e = e0 + x * kWrThreads;
            dk[x] = -1;
            if (e >= total) continue;
            const int y = e / units, unit = u0 + e - y * units;
            const Rows r = rows[y];
            if (r.dst_k < 0) continue;
            const int head = unit / t.head_units, d = 8 * (unit - head * t.head_units);
            k[x] = __ldcs(reinterpret_cast<const uint4*>(t.keys + r.src_k +
                                                         head * t.key_stride[2] + d));
            v[x] = __ldcs(reinterpret_cast<const uint4*>(t.values + r.src_v +
                                                         head * t.value_stride[2] + d));
            dk[x] = r.dst_k + head * t.k_stride[2] + d;
            dv[x] = r.dst_v + head * t.v_stride[2] + d;
        }
#pragma unroll
        for (int x = 0; x < kWrUnroll; ++x) {
            if (dk[x] < 0) continue;
            __stcs(reinterpret_cast<uint4*>(t.k_pages + dk[x]), k[x]);
            __stcs(reinterpret_cast<uint4*>(t.v_pages + dv[x]), v[x]);
        }
    }
}

}  // namespace

cudaError_t launch_extend(ExtendTask t, cudaStream_t stream) {
    // The slots of a CTA: one a thread, and more only where the device is full of
    // CTAs (each adds up the needs before it).
    int64_t slots = static_cast<int64_t>(t.batch) * t.max_new / (kExCtasPerSm * t.sm_count);
    slots = slots < kExThreads ? kExThreads : slots > kExSlots ? kExSlots : slots;
    const int most = static_cast<int>(slots);
    t.span = t.max_new < most ? (t.max_new > 0 ? t.max_new : 1) : most;
    t.lane_bits = 0;
    while ((1 << t.lane_bits) < t.span && (1 << t.lane_bits) < kExThreads) ++t.lane_bits;
    const int per = most / t.span;
    t.sequences = per < 1 ? 1 : per > kExThreads ? kExThreads : per;
    // (One CTA at least: it passes the cursor on.)
    const dim3 grid(t.max_new > 0 ? (t.max_new + t.span - 1) / t.span : 1,
                    t.batch > 0 ? (t.batch + t.sequences - 1) / t.sequences : 1);
    return launch_shaped(extend_kernel, {grid, kExThreads, 0, stream, true, 1}, t);
}

cudaError_t launch_write(WriteTask t, cudaStream_t stream) {
    // (A launch has at most 65535 slices of a token.)
    const int slice = (t.units + 65534) / 65535;
    t.cta_units = slice > kWrUnits ? slice : t.units < kWrUnits ? t.units : kWrUnits;
    const int64_t once = static_cast<int64_t>(t.tokens) * t.units / kWrUnits;
    const int rounds = once >= static_cast<int64_t>(kWrRounds) * kWrCtasPerSm * t.sm_count
                           ? kWrRounds : 1;
    t.cta_tokens = rounds * kWrUnits / t.cta_units;
    if (t.cta_tokens > kWrThreads) t.cta_tokens = kWrThreads;
    if (t.cta_tokens < 1) t.cta_tokens = 1;
    const dim3 grid((t.tokens + t.cta_tokens - 1) / t.cta_tokens,
                    (t.units + t.cta_units - 1) / t.cta_units);
    return launch_shaped(write_kernel, {grid, kWrThreads, 0, stream, true, 1}, t);
}

}  // namespace cs
