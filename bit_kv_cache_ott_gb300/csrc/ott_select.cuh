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
// when every key that still matches is selected. Then 32 keys at a time give
// way to two masks (below the last prefix, equal to it) and their counts, whose
// prefix sums give each selected block its place. The bounds: the largest of
// bd[j], bd[stride + j] .. of `groups` of them. key: n words of shared memory.
__device__ __forceinline__ void pick_blocks(const float *bd, int groups, int stride, int n, int K, int Kc, int32_t *out, uint32_t *key) {
    __shared__ int hist[256];
    __shared__ uint32_t red[3][SORT_THREADS / 32];
    __shared__ int s_digit, s_below, s_count;
    const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, wid = tid >> 5, nseg = (n + 31) / 32;
    // masks and counts of segment x take the place of its keys, the last one's, which may be fewer than four, a place of their own
    __shared__ uint32_t tail[4];
    auto seg = [&](int x) { return x + 1 < nseg ? key + 32 * x : tail; };
    uint32_t all = EMPTY, any = 0;
    int ne = 0;
    constexpr int BATCH = 8;   // bounds in flight per thread
    for (int j0 = tid; j0 < n; j0 += BATCH * nth) {
        float f[BATCH];
#pragma unroll
        for (int x = 0; x < BATCH; ++x) f[x] = j0 + x * nth < n ? bd[j0 + x * nth] : -CUDART_INF_F;
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
            if (j0 + x * nth < n) key[j0 + x * nth] = k;
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
        for (int i = tid; i < 256; i += nth) hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int j = tid; j < n; j += nth) {
            const uint32_t k = key[j];
            if (k != EMPTY && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1);
        }
        __syncthreads();
        if (wid == 0) {
            // lane l owns digits 8l .. 8l+7
            int c[8], sum = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                c[x] = hist[8 * lane + x];
                sum += c[x];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int run = incl - sum;
            if (run < need && need <= incl) {   // exactly one lane
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (run < need && need <= run + c[x]) {
                        s_digit = 8 * lane + x;
                        s_below = run;
                        s_count = c[x];
                    }
                    run += c[x];
                }
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        mask |= digit << shift;
        need -= s_below;
        cnt = s_count;
        left = shift;
    }
    // (all threads of a warp together: nth and the segments are multiples of 32)
#pragma unroll 4
    for (int j = tid; j < 32 * nseg; j += nth) {
        const uint32_t k = j < n ? key[j] : EMPTY, m = k & mask;
        const unsigned lt = __ballot_sync(0xffffffffu, k != EMPTY && m < prefix), eq = __ballot_sync(0xffffffffu, k != EMPTY && m == prefix);
        if (lane == 0) {   // (behind the votes all lanes have read their keys)
            uint32_t *w = seg(j / 32);
            w[0] = lt;
            w[1] = eq;
            w[2] = __popc(lt);
            w[3] = __popc(eq);
        }
    }
    __syncthreads();
    if (wid == 0) {
        int lt0 = 0, eq0 = 0;
        for (int x = 0; x < nseg; x += 32) {
            const bool in = x + lane < nseg;
            uint32_t *w = seg(in ? x + lane : nseg - 1);
            const int lt = in ? (int)w[2] : 0, eq = in ? (int)w[3] : 0;
            int a = lt, b = eq;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, a, o), z = __shfl_up_sync(0xffffffffu, b, o);
                if (lane >= o) {
                    a += y;
                    b += z;
                }
            }
            if (in) {
                w[2] = lt0 + a - lt;
                w[3] = eq0 + b - eq;
            }
            lt0 += __shfl_sync(0xffffffffu, a, 31);
            eq0 += __shfl_sync(0xffffffffu, b, 31);
        }
    }
    __syncthreads();
    const unsigned before = (1u << lane) - 1u;
#pragma unroll 4
    for (int j = tid; j < 32 * nseg; j += nth) {
        const uint32_t *w = seg(j / 32);
        const unsigned lt = w[0], eq = w[1];
        const int nl = (int)w[2] + __popc(lt & before), nq = (int)w[3] + __popc(eq & before);
        if ((lt >> lane & 1u) || ((eq >> lane & 1u) && nq < need)) out[nl + min(nq, need)] = j;
    }
    for (int i = want + tid; i < Kc; i += nth) out[i] = -1;
}

}  // namespace
}  // namespace ott
