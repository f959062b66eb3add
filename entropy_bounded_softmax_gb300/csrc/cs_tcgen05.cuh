// Inline-PTX wrappers for the 5th-generation tensor cores of sm_103a
// (tcgen05): tensor-memory allocation, the MMA with operands in shared
// memory and the accumulator in tensor memory, its completion on an
// mbarrier, loads of the accumulator into registers, and tensor copies
// from global into shared memory.  Used by the attn . V step of
// biencoder_attention (k_bienc_pv.cu), by the fused attention kernels
// (k_fattn_fwd.cu, k_fattn_bwd.cu) and by attention of several new tokens over
// a paged cache (k_tree.cu).
#pragma once

#include <stdint.h>

#include "cs_device.cuh"

namespace csd {

// Allocates ncols (a power of two, 32..512) columns of tensor memory for
// the CTA; executed by one whole warp.  The tensor-memory address is
// written to the shared word at dst.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(dst)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

// Frees what tmem_alloc allocated; executed by the same warp.
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 :: "r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tc_fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Makes this thread's ordinary shared-memory stores visible to the tensor
// cores (the async proxy).
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Rounds an fp32 to the nearest TF32 (10 stored mantissa bits), returned as
// the fp32 with the low 13 bits zero.
__device__ __forceinline__ float to_tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return __uint_as_float(r);
}

// Shared-memory matrix descriptor, no swizzle (the canonical "interleaved"
// layout of 8-row x 16-byte core matrices): start address, the byte offset
// between core matrices adjacent along K (leading) and along M or N
// (stride), and the descriptor version of this architecture.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo,
                                              uint32_t sbo) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
           (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) |
           (1ull << 46);
}

// Instruction descriptor of a dense kind::tf32 MMA with an fp32
// accumulator, both operands TF32 and K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_tf32(int M, int N) {
    return (1u << 4)                                   // D: fp32
         | (2u << 7)                                   // A: TF32
         | (2u << 10)                                  // B: TF32
         | (static_cast<uint32_t>(N >> 3) << 17)
         | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] . B[smem]^T, issued by one thread.
__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint64_t a_desc,
                                         uint64_t b_desc, uint32_t idesc,
                                         bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n}"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc),
           "r"(accumulate ? 1u : 0u) : "memory");
}

// The mbarrier at bar receives one arrival when every tcgen05 operation
// this thread issued before has completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
        :: "r"(smem_addr(bar)) : "memory");
}

// 16 consecutive 32-bit columns of this thread's tensor-memory lane (the
// warp's quarter of the lanes: lane base 32 (warp % 4)).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    // The load and its wait in one statement, so that no use of the
    // registers can be scheduled between them.
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 2-D tiled copy by the tensor-memory-access unit: the box of the tensor
// map at element coordinates (x, y) into shared memory at sdst (laid out
// and swizzled as the map says), counted in bytes on the mbarrier at bar.
__device__ __forceinline__ void tma_load_2d(void* sdst, const void* tmap, int x,
                                            int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];"
        :: "r"(smem_addr(sdst)), "l"(tmap), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// Shared-memory matrix descriptor of a K-major operand in the 128-byte
// swizzled layout: 8-row groups of 128-byte rows (1024-byte atoms, each
// row's 16-byte units permuted by the row index mod 8), atoms stacked
// along M or N every sbo bytes; the start address may step through an
// atom's row in 32-byte (one K = 8 tf32) increments.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr, uint32_t sbo) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
           (static_cast<uint64_t>(1u) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) |
           (1ull << 46) |
           (2ull << 61);
}

// Instruction descriptor of a dense kind::f16 MMA on bf16 or fp16 operands
// with an fp32 accumulator, M x N; A K-major, B K-major or (b_mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_half(int M, int N, bool b_mn, bool fp16) {
    return (1u << 4)                                   // D: fp32
         | (fp16 ? 0u : 1u << 7)                       // A: fp16 or bf16
         | (fp16 ? 0u : 1u << 10)                      // B
         | (b_mn ? 1u << 16 : 0u)
         | (static_cast<uint32_t>(N >> 3) << 17)
         | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) {
    return idesc_half(M, N, b_mn, false);
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_lane() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}

// The low word of the descriptors of 128-byte swizzled operands whose 8-row
// atoms lie 1024 bytes apart: the address, which steps by plain additions, and
// the leading offset (bytes; K-major operands have none).  Their high word is
// kDescHigh: the atoms' distance, this architecture's version, the swizzle.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
    // (In a cluster an address has bits above the 18 that name a byte of the
    // CTA's shared memory, which would fall into the offset.)
    return ((saddr & 0x3ffffu) >> 4) | ((lbo ? lbo >> 4 : 1u) << 16);
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

// D[tmem] (+)= A[smem] . B[smem], K = 16, of descriptors with these low words.
// Called by the whole warp, issued by the lane where `leader` is true: the
// operands are then the same in every lane and stay in uniform registers,
// where a branch around the call would move each of them there for every
// instruction (an issuing thread that did so took 97 to 150 cycles an
// instruction of 64).
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low,
                                            uint32_t idesc, bool accumulate, bool leader) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 a, b;\n"
        " setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " mov.b64 a, {%1, %6};\n mov.b64 b, {%2, %6};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}"
        :: "r"(d_tmem), "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate ? 1u : 0u),
           "r"(leader ? 1u : 0u), "r"(kDescHigh) : "memory");
}

// The same with A in tensor memory: row m in lane m, two bf16 to a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low,
                                            uint32_t idesc, bool accumulate, bool leader) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 b;\n"
        " setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " mov.b64 b, {%2, %6};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}"
        :: "r"(d_tmem), "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate ? 1u : 0u),
           "r"(leader ? 1u : 0u), "r"(kDescHigh) : "memory");
}

// mma_commit by the leader of a warp that issues as mma_bf16_ss.
__device__ __forceinline__ void mma_commit(uint64_t* bar, bool leader) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
        :: "r"(smem_addr(bar)), "r"(leader ? 1u : 0u) : "memory");
}

// 32 consecutive columns of this thread's lane, without the wait: the
// registers are valid after tmem_wait_ld() on them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
          "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr) : "memory");
}

// Waits for this thread's tensor-memory loads.  The empty statements tie the
// N registers to a point after the wait, so that no use is scheduled before.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The same of 16 columns.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// 32 registers into 32 consecutive columns of this thread's lane; complete
// after tmem_wait_st().
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
        "%23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        :: "r"(taddr),
           "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
           "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
           "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
           "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
           "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
           "r"(r[30]), "r"(r[31]) : "memory");
}

// 16 registers into 16 consecutive columns, as tmem_st32.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, "
        "%9, %10, %11, %12, %13, %14, %15, %16};"
        :: "r"(taddr),
           "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
           "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
           "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
           "r"(r[15]) : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 4-D tiled copy, as tma_load_2d.
__device__ __forceinline__ void tma_load_4d(void* sdst, const void* tmap, int x, int y,
                                            int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        :: "r"(smem_addr(sdst)), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w),
           "r"(smem_addr(bar)) : "memory");
}

// Fetches a box into L2 alone.
__device__ __forceinline__ void tma_prefetch_4d(const void* tmap, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];"
                 :: "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Fetches a tensor map ahead of its first use.
__device__ __forceinline__ void prefetch_tmap(const void* tmap) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(tmap) : "memory");
}

// Untiled copy of `bytes` (a multiple of 16; both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(void* sdst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1], %2, [%3];"
        :: "r"(smem_addr(sdst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

// Two fp32 to a packed bf16 pair (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace csd
