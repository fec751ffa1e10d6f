// ott_tcgen.cuh -- the tcgen05, tensor memory and mbarrier instructions of the
// kernels that multiply tiles (ott_chunk_tiles.cu, ott_byte_tiles.cu).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ott_chunk.cuh"

namespace ott {
namespace {

__device__ __forceinline__ void bar_init(uint64_t *b, int n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(ch_smem(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(ch_smem(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(ch_smem(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
// Bounded wait: gives up after four seconds, or once another role has. A role
// whose wait gave up goes on (every later wait then ends at once, every
// address stays what it would have been), so that warps stay together and
// all roles reach the end; the status word tells the host.
__device__ __forceinline__ void bar_wait(uint64_t *b, uint32_t parity, volatile int *gave_up) {   // whole warps
    if (!bar_try(b, parity)) {
        const unsigned long long end = now_ns() + 4000000000ull;
        for (int k = 0; !bar_try(b, parity); ++k) {
            if (k & 63) continue;
            if (*gave_up) break;
            if (now_ns() > end) *gave_up = 1;
        }
    }
    __syncwarp();
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(ch_smem(b)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The registers of the loads before it are valid from here on: `tie` keeps
// the compiler from moving their uses above the wait.
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tie16(float *f) {
    asm volatile("" : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]),
                      "+f"(f[8]), "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]), "+f"(f[15]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tm_ld16(uint32_t at, float *f) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
#pragma unroll
    for (int x = 0; x < 16; ++x) f[x] = __uint_as_float(r[x]);
}
__device__ __forceinline__ void tm_st16(uint32_t at, const float *f) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]), "f"(f[8]), "f"(f[9]),
        "f"(f[10]), "f"(f[11]), "f"(f[12]), "f"(f[13]), "f"(f[14]), "f"(f[15])
        : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Shared-memory matrix descriptor: K-major, swizzled rows of 128 bytes (kind
// 2), 8-row groups `group` bytes apart. (Value tiles in 32-byte rows, one
// group of tokens each, measured 127 cycles per product of 16 tokens instead
// of 64: those are read 32 bytes at a time.) The low word holds the
// address in 16-byte units (and a field that swizzled layouts ignore), so
// that a step along the operand is an addition to it.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr >> 4) & 0x3fff) | (1u << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t group, uint32_t kind) {
    return (group >> 4) | (1u << 14) | (kind << 29);
}
// fp16 x fp16 -> fp32, M = 128, both operands K-major
__host__ __device__ constexpr uint32_t instr_desc(int n) {
    return (1u << 4) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(128 / 16) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n setp.ne.u32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t at, uint32_t b, uint32_t hi, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %3};\n setp.ne.u32 p, %5, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}" ::"r"(d),
        "r"(at), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// Order of a group's 16 tokens in its tile rows (keys) and 32-byte columns
// (values), and of 8 channels among the rows of a value tile: 2i, 2i + 1,
// 2i + 8, 2i + 9 are adjacent, which is what a lane of an mma fragment holds,
// and the channels' low bits are rotated, so that 16 lanes of an 8-byte store
// meet all banks.
__device__ __forceinline__ int slot_of(int t) { return 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1); }
__host__ __device__ constexpr int vrow(int r) { return ((r << 1) & 6) | (r >> 2); }

__device__ __forceinline__ float max16(const float *x) {   // short chains of three-way maxima
    float g[3] = {x[0], x[1], x[2]};
#pragma unroll
    for (int c = 3; c < 15; c += 6)
#pragma unroll
        for (int y = 0; y < 3; ++y) g[y] = fmaxf(fmaxf(g[y], x[c + 2 * y]), x[c + 2 * y + 1]);
    return fmaxf(fmaxf(g[0], g[1]), fmaxf(g[2], x[15]));
}

}  // namespace
}  // namespace ott
