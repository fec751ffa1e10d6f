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

// Exclusive prefix sum of v over the threads of the CTA (in thread order);
// `total` receives the sum over all threads. ws: 32 ints of shared memory.
__device__ __forceinline__ int block_exscan(int v, int *ws, int &total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) ws[wid] = x;
    __syncthreads();
    if (wid == 0) {
        int t = lane < nw ? ws[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        ws[lane] = t;
    }
    __syncthreads();
    total = ws[nw - 1];
    const int r = (wid > 0 ? ws[wid - 1] : 0) + x - v;
    __syncthreads();   // ws is reused by the next call
    return r;
}

// The selection among n bounds (-inf: an empty block), by a CTA: the first min(K,
// non-empty) into out[0 .. Kc), -1 behind them, by an exact radix select: key_j = the bit-inverted ordered
// bound (smallest key = largest bound). Four rounds over 8-bit digits, most
// significant first, each a histogram of the keys that still match the
// digits found so far, give the key tau of the need-th smallest key and the
// number `take` of keys equal to tau that belong to the selection. The
// selection is every key below tau and the `take` lowest-indexed keys equal
// to tau: exactly the first min(K, non-empty) blocks under (bound
// descending, index ascending). A prefix count gives each its slot in
// ascending block order.
constexpr uint32_t EMPTY = 0xffffffffu;           // key of an empty block

// key: n words of shared memory.
__device__ __forceinline__ void pick_blocks(const float *bd, int n, int K, int Kc, int32_t *out, uint32_t *key) {
    __shared__ int hist[256];
    __shared__ int ws[32];
    __shared__ int s_digit, s_below;
    const int tid = threadIdx.x, nth = blockDim.x;
    // a contiguous chunk of blocks per thread, so that prefix counts follow block order
    const int chunk = (n + nth - 1) / nth, jb = min(n, tid * chunk), je = min(n, jb + chunk);
    int ne_local = 0;
    for (int j = jb; j < je; ++j) {
        const float f = bd[j];
        const bool nonempty = f != -CUDART_INF_F;
        key[j] = nonempty ? ~ordered(f) : EMPTY;   // a finite bound never maps to EMPTY
        ne_local += nonempty;
    }
    int ne;
    block_exscan(ne_local, ws, ne);
    const int want = min(K, ne);
    uint32_t prefix = 0, mask = 0;
    int need = want;
    for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
        for (int i = tid; i < 256; i += nth) hist[i] = 0;
        __syncthreads();
        for (int j = jb; j < je; ++j) {
            const uint32_t k = key[j];
            if (k != EMPTY && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (tid < 32) {
            // lane l owns digits 8l .. 8l+7
            int cnt[8], sum = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                cnt[x] = hist[8 * tid + x];
                sum += cnt[x];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += y;
            }
            const int excl = incl - sum;
            if (excl < need && need <= incl) {   // exactly one lane
                int c = excl, dg = 8 * tid;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    if (c + cnt[x] >= need) {
                        dg = 8 * tid + x;
                        break;
                    }
                    c += cnt[x];
                }
                s_digit = dg;
                s_below = c;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        mask |= 255u << shift;
        need -= s_below;
        __syncthreads();
    }
    // keys equal to tau = prefix: the `need` lowest-indexed ones are taken
    int eq_local = 0;
    for (int j = jb; j < je; ++j) eq_local += want > 0 && key[j] != EMPTY && key[j] == prefix;
    int eq_total;
    int eq_before = block_exscan(eq_local, ws, eq_total);
    int sel_local = 0;
    for (int j = jb; j < je; ++j) {
        const uint32_t k = key[j];
        const bool ok = want > 0 && k != EMPTY;
        const bool take = ok && (k < prefix || (k == prefix && eq_before++ < need));
        key[j] = take ? 1u : 0u;                   // reused as the selection mark
        sel_local += take;
    }
    int nsel;
    int pos = block_exscan(sel_local, ws, nsel);
    for (int j = jb; j < je; ++j)
        if (key[j]) out[pos++] = j;
    for (int i = nsel + tid; i < Kc; i += nth) out[i] = -1;
}

}  // namespace
}  // namespace ott
