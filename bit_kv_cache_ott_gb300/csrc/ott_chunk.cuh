// ott_chunk.cuh -- what the kernels of ott_chunk_attn and
// ott_decode_attn_window share: the launch's arguments, the table of its
// sequences, the visibility rule, small device helpers.
#pragma once

#include <math_constants.h>

#include "ott_internal.cuh"

namespace ott {

// Tokens whose weighted values the tensor cores add up on their own. They
// truncate each product to the sum's last place, so a sum of values of one
// sign shrinks by 5.9e-9 of itself per token (tcgen05; measured, 8,192 rows of
// 8 heads over 2^20 tokens: 3.8e-3 of the output when runs were as long as the
// plan made them), and by 2.4 to 4.8e-9 with mma.sync. Sums end here and are
// merged in fp32: 1.5e-4 at any length, a third of the output's largest
// rounding. 2,048 tokens over 131K: 3.35 ms, and 3.29 with sums of 57,344
// tokens (3.4e-4).
constexpr int SUM_TOKENS = 25088;

// One sequence of a launch.
struct ChunkSeq {
    long long base;    // its first work item; entry [nseq] holds the total
    int ubase;         // its first work unit
    int S;             // slices of query rows per kv head (0: no queries)
    int T;             // tokens in the cache
    int pos0;          // position of its first query
    int nq;            // query tokens
    int nnew;          // new tokens behind the cache's: nq, or 0 for a decode step
    int nf, jlo;       // blocks; blocks j >= jlo may hold tokens of the window
    int nsink;         // slots of the list of blocks j < jlo that hold one of the first tokens
    int ntail, npool, ring_start;
    int Sf, Iu;        // fp16 work items, all work items of a unit
};
// A kernel parameter: 64 sequences (4 KB) per launch; a table of 256 made
// every launch of a small batch about a microsecond longer.
constexpr int CHUNK_SEQS = 64;
struct ChunkTable {
    ChunkSeq e[CHUNK_SEQS + 1];
};

struct ChunkArgs {
    const uint8_t *blk;
    long long blk_bytes;
    const int32_t *bidx, *bcnt, *bt, *sel, *pidx, *cidx;
    const int *cmeta;
    const __half *rk, *rv, *pk, *pv, *ck, *cv;
    const __half *q, *k, *v;   // [B][Hq][n][d], [B][Hkv][n][d]
    __half *out;
    float *part;
    int *ctl;
    int n, B0, nseq;           // rows of room per sequence; the launch's sequences B0 .. B0 + nseq - 1
    int Hq, Hkv, g, NB, G, P, C, ring;
    int jfull;                 // blocks j >= jfull hold G tokens (norm criterion)
    int CPB;                   // chunks (CHUNK_TILES tiles) per block
    int spi;           // rows mode: slots of the list of first tokens' blocks per work item
    int window, sinks;         // window 0: no limit
    long long W;               // work items
    int ctas;                  // CTAs
    int NWp, MAXU, RV;         // active warps, units a warp's range can touch, rows of a partial
    float sl2;                 // log2(e) / sqrt(d)
};

// Valid tokens of block j of unit u.
__device__ __forceinline__ int chunk_block_cnt(const ChunkArgs &a, int u, int j) {
    if (a.bcnt) return __ldg(a.bcnt + (size_t)u * a.NB + j);
    return j >= a.jfull ? a.G : block_count(a.P, a.G, j);
}

// Position of fp16 token f of a unit: residual ring (oldest first), pool,
// cold pool (oldest first), new tokens.
__device__ __forceinline__ int chunk_fp16_pos(const ChunkArgs &a, const ChunkSeq &s, int u, int f, int ncold, int chead) {
    if (f < s.ntail) return s.T - s.ntail + f;
    f -= s.ntail;
    if (f < s.npool) return __ldg(a.pidx + (size_t)u * a.P + f);
    f -= s.npool;
    if (f < ncold) {
        int x = chead + f;
        if (x >= a.C) x -= a.C;
        return __ldg(a.cidx + (size_t)u * a.C + x);
    }
    return s.T + f - ncold;
}
__device__ __forceinline__ const __half *chunk_fp16_row(const ChunkArgs &a, const ChunkSeq &s, int b, int hkv, int u,
                                                        int f, int ncold, int chead, bool val, int D) {
    if (f < s.ntail) {
        int x = s.ring_start + f;
        if (x >= a.ring) x -= a.ring;
        return (val ? a.rv : a.rk) + ((size_t)u * a.ring + x) * D;
    }
    f -= s.ntail;
    if (f < s.npool) return (val ? a.pv : a.pk) + ((size_t)u * a.P + f) * D;
    f -= s.npool;
    if (f < ncold) {
        int x = chead + f;
        if (x >= a.C) x -= a.C;
        return (val ? a.cv : a.ck) + ((size_t)u * a.C + x) * D;
    }
    return (val ? a.v : a.k) + (((size_t)b * a.Hkv + hkv) * a.n + (f - ncold)) * D;
}

// The token at t is seen from position p, whose window starts at lo.
__device__ __forceinline__ bool chunk_sees(int t, int p, int lo, int sinks) { return t <= p && (t >= lo || t < sinks); }

// What a row's output is multiplied by: one over the sum L of its weights (NaN
// stays). A row of a chunk sees at least its own token, so that L = 0 means
// that every score was -inf: NaN. A step may also see nothing (a policy has
// discarded every token of its window): zeros, unless its query q is not finite.
__device__ __forceinline__ float chunk_norm(float L, bool step, const __half *q, int D) {
    if (L != 0.0f) return 1.0f / L;
    bool finite = step;
    for (int c = 0; finite && c < D; ++c) finite = fabsf(__half2float(q[c])) < CUDART_INF_F;
    return finite ? 0.0f : CUDART_NAN_F;
}

__device__ __forceinline__ uint32_t ch_smem(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ float ch_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t ch_h2(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 ch_as_h2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }

// Dequantization in fp16x2 registers. The two codes at position p of a word
// (w8 = w >> 8 serves p >= 4) are ORed into the mantissa of 2^(10-2c), c = p
// mod 4, whose unit in the last place they are counted in: an exact fp16
// 2^(10-2c) + code. One subtraction gives code - 1 (keys) or code (values),
// exactly. Magic holds the four 2^(10-2c) in registers, so that extraction is
// one three-input operation (it takes one immediate, the mask).
struct Magic {
    uint32_t m[4];
    __device__ __forceinline__ Magic() {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            m[c] = (uint32_t)((25 - 2 * c) << 10) * 0x10001u;
            asm volatile("" : "+r"(m[c]));   // a register's value from here on
        }
    }
};
__device__ __forceinline__ uint32_t ch_raw(const Magic &mg, uint32_t w, uint32_t w8, int p) {
    const int c = p & 3;
    uint32_t d;   // (w & mask) | magic, as one operation
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(p < 4 ? w : w8), "r"(0x00030003u << (2 * c)), "r"(mg.m[c]));
    return d;
}
__device__ __forceinline__ uint32_t ch_const(int p, int less) {   // -(2^(10-2c) + less) in both halves
    const __half h = __float2half_rn(-(float)((1 << (10 - 2 * (p & 3))) + less));
    return (uint32_t)__half_as_ushort(h) * 0x10001u;
}
// s * (code - 1): exact (a scale, its negative, zero or twice it)
__device__ __forceinline__ uint32_t ch_key(const Magic &mg, uint32_t w, uint32_t w8, int p, uint32_t s2) {
    const __half2 c1 = __hadd2(ch_as_h2(ch_raw(mg, w, w8, p)), ch_as_h2(ch_const(p, 1)));
    return ch_h2(__hmul2(c1, ch_as_h2(s2)));
}
// z + s * code, one rounding
__device__ __forceinline__ uint32_t ch_val(const Magic &mg, uint32_t w, uint32_t w8, int p, uint32_t s2, uint32_t z2) {
    const __half2 c = __hadd2(ch_as_h2(ch_raw(mg, w, w8, p)), ch_as_h2(ch_const(p, 0)));
    return ch_h2(__hfma2(c, ch_as_h2(s2), ch_as_h2(z2)));
}
// A scale of 32,768 or more (a channel that spans more than 98,256) has no
// 2 s in fp16. A block with one takes half of every scale (exact but for the
// last bit of subnormal ones), and its scores twice. Looking for such scales
// costs 1 to 2% (mixed paged batch 350 -> 356 us, 8 rows 185 -> 188).
__device__ __forceinline__ bool ch_wide(uint32_t s) { return (s & 0xffffu) >= 0x7800u; }   // (scales are positive)
// fp16x2 hi + lo = s + z exactly up to lo's rounding (the two-sum of both halves)
__device__ __forceinline__ void ch_offset(uint32_t s2, uint32_t z2, uint32_t &hi, uint32_t &lo) {
    const __half2 s = ch_as_h2(s2), z = ch_as_h2(z2);
    const __half2 h = __hadd2_rn(z, s), b = __hsub2_rn(h, z);
    lo = ch_h2(__hadd2_rn(__hsub2_rn(z, __hsub2_rn(h, b)), __hsub2_rn(s, b)));
    hi = ch_h2(h);
}

// Items split over warps as evenly as integers allow (the decode kernel's rule).
__device__ __forceinline__ long long ch_range_start(long long W, int NWp, long long w) {
    const unsigned long long num = (unsigned long long)w * (unsigned long long)W;
    if (num <= 0xffffffffull) return (long long)((unsigned)num / (unsigned)NWp);
    return (long long)(num / (unsigned long long)NWp);
}
__device__ __forceinline__ int ch_warp_of(long long W, int NWp, long long x) {
    return (int)(((unsigned long long)(x + 1) * (unsigned long long)NWp + (unsigned long long)W - 1) /
                 (unsigned long long)W) - 1;
}
// Rounded to fp16, a weight loses its last bits below 2^-14 and is gone below
// 2^-25, while the sum of the weights, in fp32, counts all of it. A row's
// reference lies at most GROW (log2) below its largest score, so weights are
// taken LIFT higher: the largest is at most 2^(GROW + LIFT), inside fp16, and
// what is lost lies 2^LIFT lower. The factor 2^LIFT is in sums and outputs
// alike and cancels.
constexpr float GROW = 8.0f, LIFT = 7.0f;

// Entry that holds work item x (x < W): the last one whose base is <= x.
__device__ __forceinline__ int ch_entry_of(const ChunkTable &st, int nseq, long long x) {
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (st.e[mid].base <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ott_decode.cu: the decode kernel in rows mode, gs rows per slice
cudaError_t launch_decode_rows(const ott_cache *c, const ChunkArgs &a, const ChunkTable &st, int gs, int ipb, cudaStream_t s);
cudaError_t set_decode_rows_attributes(int d, int smem_max);
// ott_chunk_tiles.cu
cudaError_t set_tiles_attributes(int d);
bool plan_tiles(const ott_cache *c, ChunkArgs &a, ChunkTable &st, int &nC, bool &whole, size_t &part_floats);
cudaError_t launch_tiles(const ott_cache *c, const ChunkArgs &a, const ChunkTable &st, int nC, bool whole, cudaStream_t s);

}  // namespace ott
