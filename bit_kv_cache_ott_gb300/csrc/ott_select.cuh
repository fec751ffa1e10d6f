// ott_select.cuh -- the selection of the best-bounded blocks that the Top-K
// forms of decoding share (ott_topk.cu, ott_byte_rows.cu).
#pragma once

#include <math_constants.h>
#include <stdint.h>

namespace ott {
namespace {

constexpr int SORT_THREADS = 512;   // selection CTA: at most

// fp32 -> uint32 whose unsigned order is the float order
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t x = __float_as_uint(f);
    return (x & 0x80000000u) ? ~x : (x | 0x80000000u);
}

constexpr uint32_t EMPTY = 0xffffffffu;           // key of an empty block

// The selection among n bounds (-inf: an empty block), by a CTA of whole warps:
// the first min(K, non-empty) under (bound descending, index ascending), into
// out[0 .. Kc) in ascending order, -1 behind them. An exact radix select: key_j
// = the bit-inverted ordered bound (smallest key = largest bound). The bits
// above the highest one in which keys differ are known (bounds are of one
// magnitude: a first histogram over sign and exponent would put all keys into a
// few bins, whose atomics go one after another). Rounds over 8-bit digits below
// them, each a histogram of the keys that match the digits found so far, end
// when every key that still matches is selected. Then threads count, in four
// keys each, those below the last prefix and those equal to it; the sums over
// the threads before give each selected block its place. Latency bounds all of
// it (2,047 bounds, 256 selected, in cycles: bounds and common bits 2,000, a
// round 1,400, places 1,000); loops unrolled four and eight times cost a 131K
// layer's call 0.4 us, a key at a time with votes for the places 1.5 us.
// The bounds: the largest of bd[j], bd[stride + j] .. of `groups` of them.
// key: n words of shared memory and up to the next multiple of four.
__device__ __forceinline__ void pick_blocks(const float *bd, int groups, int stride, int n, int K, int Kc, int32_t *out, uint32_t *key) {
    __shared__ __align__(16) int hist[256];
    __shared__ uint32_t red[3][SORT_THREADS / 32], tot[2][SORT_THREADS / 32];
    __shared__ int4 found;   // a round's digit, the keys below it, those that have it
    const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, wid = tid >> 5, n4 = (n + 3) / 4;
    const uint4 *const key4 = reinterpret_cast<const uint4 *>(key);
    for (int i = tid; i < 256; i += nth) hist[i] = 0;
    uint32_t all = EMPTY, any = 0;
    int ne = 0;
    constexpr int BATCH = 4;   // bounds in flight per thread
#pragma unroll 1
    for (int j0 = tid; j0 < 4 * n4; j0 += BATCH * nth) {
        float f[BATCH];
#pragma unroll
        for (int x = 0; x < BATCH; ++x) f[x] = j0 + x * nth < n ? bd[j0 + x * nth] : -CUDART_INF_F;
#pragma unroll 1
        for (int y = 1; y < groups; ++y) {
            float v[BATCH];
#pragma unroll
            for (int x = 0; x < BATCH; ++x) v[x] = j0 + x * nth < n ? bd[(size_t)y * stride + j0 + x * nth] : -CUDART_INF_F;
#pragma unroll
            for (int x = 0; x < BATCH; ++x) f[x] = v[x] > f[x] ? v[x] : f[x];
        }
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
            uint32_t k = EMPTY;
            if (f[x] != -CUDART_INF_F) {
                k = ~ordered(f[x]);   // a finite bound never maps to EMPTY
                all &= k;
                any |= k;
                ++ne;
            }
            if (j0 + x * nth < 4 * n4) key[j0 + x * nth] = k;
        }
    }
    all = __reduce_and_sync(0xffffffffu, all);
    any = __reduce_or_sync(0xffffffffu, any);
    ne = __reduce_add_sync(0xffffffffu, ne);
    if (lane == 0) {
        red[0][wid] = all;
        red[1][wid] = any;
        red[2][wid] = (uint32_t)ne;
    }
    __syncthreads();
    const bool has = lane < nth / 32;
    all = __reduce_and_sync(0xffffffffu, has ? red[0][lane] : EMPTY);
    any = __reduce_or_sync(0xffffffffu, has ? red[1][lane] : 0u);
    ne = __reduce_add_sync(0xffffffffu, has ? (int)red[2][lane] : 0);
    const int want = min(K, ne);
    int left = 32 - __clz(all ^ any);   // bits that are not known yet
    uint32_t mask = left == 32 ? 0u : 0xffffffffu << left, prefix = all & mask;
    // the first `need` of the `cnt` keys that match the prefix are selected, and all keys below it
    int need = want, cnt = ne;
    while (left > 0 && need < cnt) {
        const int bits = min(8, left), shift = left - bits;
        const uint32_t digit = (1u << bits) - 1u;
#pragma unroll 1
        for (int j = tid; j < n; j += 4 * nth) {
            uint32_t k[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) k[x] = j + x * nth < n ? key[j + x * nth] : EMPTY;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (k[x] != EMPTY && (k[x] & mask) == prefix) atomicAdd(&hist[(k[x] >> shift) & digit], 1);
        }
        __syncthreads();
        if (wid == 0) {
            // lane l owns digits 8l .. 8l+7, and clears them for the next round
            int4 *const h = reinterpret_cast<int4 *>(hist) + 2 * lane;
            const int4 ha = h[0], hb = h[1];
            h[0] = h[1] = make_int4(0, 0, 0, 0);
            const int c[8] = {ha.x, ha.y, ha.z, ha.w, hb.x, hb.y, hb.z, hb.w};
            const int sum = ha.x + ha.y + ha.z + ha.w + hb.x + hb.y + hb.z + hb.w;
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int run = incl - sum, x = 0, n_x = c[0];
            const bool mine = run < need && need <= incl;   // one lane's
#pragma unroll
            for (int y = 0; y < 7; ++y) {   // its first digit that reaches `need`
                const bool next = run + c[y] < need && x == y;
                run += next ? c[y] : 0;
                x += next;
                n_x = next ? c[y + 1] : n_x;
            }
            if (mine) found = make_int4(8 * lane + x, run, n_x, 0);
        }
        __syncthreads();
        const int4 f = found;
        prefix |= (uint32_t)f.x << shift;
        mask |= digit << shift;
        need -= f.y;
        cnt = f.z;
        left = shift;
    }
    int lt0 = 0, eq0 = 0;   // below the prefix, equal to it, so far
#pragma unroll 1
    for (int c0 = 0, turn = 0; c0 < n4; c0 += nth, turn ^= 1) {
        const int j = c0 + tid;
        const uint4 k4 = j < n4 ? key4[j] : make_uint4(EMPTY, EMPTY, EMPTY, EMPTY);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        bool lt[4], eq[4];
        uint32_t own = 0;   // low half: below; high half: equal
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            lt[x] = k[x] != EMPTY && (k[x] & mask) < prefix;
            eq[x] = k[x] != EMPTY && (k[x] & mask) == prefix;
            own += (lt[x] ? 1u : 0u) + (eq[x] ? 0x10000u : 0u);
        }
        uint32_t incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) tot[turn][wid] = incl;
        __syncthreads();
        const uint32_t t = lane < nth / 32 ? tot[turn][lane] : 0u;
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < wid ? t : 0u) + incl - own;
        int nl = lt0 + (int)(before & 0xffffu), nq = eq0 + (int)(before >> 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (lt[x] || (eq[x] && nq < need)) out[nl + min(nq, need)] = 4 * j + x;
            nl += lt[x];
            nq += eq[x];
        }
        const uint32_t more = __reduce_add_sync(0xffffffffu, t);
        lt0 += (int)(more & 0xffffu);
        eq0 += (int)(more >> 16);
    }
    for (int i = want + tid; i < Kc; i += nth) out[i] = -1;
}

}  // namespace
}  // namespace ott
