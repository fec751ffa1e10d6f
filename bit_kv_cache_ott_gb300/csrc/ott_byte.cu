// ott_byte.cu -- the cache held in 8 bits: its calls (argument and state
// checks, the host's counts), and the kernels that write it and read it back.
//
// Writing. A CTA quantizes the keys or the values of one block: it holds them
// in registers, finds each channel's smallest and largest value (the keys' are
// stored for the Top-K bounds), from them a = max |x|, and stores the codes in
// the pieces that the attention kernels load. It reads a token's 4 d bytes and
// writes 2 d once each; HBM bounds it (32 prompts of 4,096 tokens, 32 heads, d
// = 128, written and read back, 6.5 GB: 984 us, 6.6 TB/s).
// The quotient 127 x / a (or 448 x / a) decides a rounding, so it has to fall
// on the right side of every tie: 127 x is exact in fp32; the quotient differs
// from a tie by 0 or by more than 2^-20 of itself (both are ratios of integers
// of at most 18 and 11 bits); and a product with 1 / a, corrected once by its
// exact residual (Markstein's division), is off by less than 2^-23, and exact
// where the quotient is a number that fp32 holds.
//
// Reading back. A warp takes a group of 16 tokens: codes times the scale in
// fp32, rounded to fp16, to rows in shared memory (the values transposed by
// movmatrix on the way), from there whole rows to memory.
#include <algorithm>
#include <climits>
#include <cstdlib>
#include <cstring>
#include <new>

#include "ott_byte.cuh"

using namespace ott;

namespace {

constexpr int READ_WARPS = 8;
// Threads of an append CTA: eight 16-byte pieces of one block each. (With four,
// and scalar arithmetic, a thread's fixed work was half of its instructions:
// 131K tokens of 8 units in blocks of 64 took 136 us, now 118, in blocks of 32
// 100 us per 400 MB, now 60.)
__host__ __device__ constexpr int app_threads(int d, int g) { return g * d / 64; }

struct AppendArgs {
    uint8_t *blk;
    ByteRec *rec;
    __half2 *dig;
    __half *tk, *tv;
    int32_t *bt;                // null: slot u * NB + j
    const int32_t *fstack;
    const __half *k, *v;        // [entries][Hkv][n][d]
    int n, B0, nseq, Hkv, NB;
    int top;                    // free slots before the call (paged)
};
// Entry e: sequence B0 + e, which holds T tokens and receives m. Its CTAs
// start at base (one per unit and block that becomes complete, at least one
// per unit); its blocks take the free slots from number `taken` on.
struct AppendTable {
    int base[CHUNK_SEQS + 1], T[CHUNK_SEQS], m[CHUNK_SEQS], taken[CHUNK_SEQS];
};

__device__ __forceinline__ uint32_t h2min(uint32_t a, uint32_t b) { return ch_h2(__hmin2(ch_as_h2(a), ch_as_h2(b))); }
__device__ __forceinline__ uint32_t h2max(uint32_t a, uint32_t b) { return ch_h2(__hmax2(ch_as_h2(a), ch_as_h2(b))); }

// Two codes of x0, x1 (fp16): in the low bytes of the result.
template <int FMT>
__device__ __forceinline__ uint32_t encode2(uint32_t x, float a, float inv) {
    constexpr float TOP = FMT == OTT_BYTE_INT ? 127.0f : 448.0f;
    const float2 p = __fmul2_rn(__half22float2(ch_as_h2(x)), make_float2(TOP, TOP)), i2 = make_float2(inv, inv);
    const float2 q = __fmul2_rn(p, i2);
    // p - q a: exact
    const float2 r = __ffma2_rn(__ffma2_rn(q, make_float2(-a, -a), p), i2, q);
    if constexpr (FMT == OTT_BYTE_INT) {
        // r + 1.5 * 2^23 + 128: the sum rounds r to an integer (ties to even), its low byte is 128 + code
        const float2 c = __fadd2_rn(r, make_float2(12583040.0f, 12583040.0f));
        return __byte_perm(__float_as_uint(c.x), __float_as_uint(c.y), 0x0040);
    } else {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(r.y), "f"(r.x));
        return c;
    }
}

template <int D, int G, int FMT>
__global__ void __launch_bounds__(app_threads(D, G))
    k_byte_append(const __grid_constant__ AppendArgs a, const __grid_constant__ AppendTable t) {
    constexpr int APP_THREADS = app_threads(D, G);
    constexpr int CPR = D / 8;                          // 16-byte pieces of a token
    constexpr int PER = G * CPR / APP_THREADS;          // pieces per thread: tokens TPI apart, the same channels
    constexpr int TPI = APP_THREADS / CPR, WARPS = APP_THREADS / 32;
    static_assert(PER * APP_THREADS == G * CPR && TPI * CPR == APP_THREADS && WARPS * 32 == APP_THREADS, "whole pieces");
    constexpr float TOP = FMT == OTT_BYTE_INT ? 127.0f : 448.0f;
    constexpr int RS = D + 4;                           // row of codes in shared memory
    __shared__ uint32_t rng[2][WARPS][D / 2];           // smallest and largest, by warp
    __shared__ float amax[WARPS];
    __shared__ uint32_t rows[G * RS / 4];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int e = 0, hi = a.nseq;
    while (hi - e > 1) {
        const int mid = (e + hi) >> 1;
        if (t.base[mid] <= (int)blockIdx.x) e = mid;
        else hi = mid;
    }
    const int T = t.T[e], end = T + t.m[e], j0 = T / G, nblk = end / G - j0, per = max(nblk, 1);
    const int rel = (int)blockIdx.x - t.base[e], head = rel / per, x = rel % per;
    const bool val = blockIdx.y != 0;
    const int u = (a.B0 + e) * a.Hkv + head;
    const __half *const src = (val ? a.v : a.k) + ((size_t)e * a.Hkv + head) * a.n * D;
    __half *const open = (val ? a.tv : a.tk) + (size_t)u * G * D;
    const int ch8 = tid % CPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (x < nblk) {
        uint4 v[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int tok = tid / CPR + TPI * p, at = (j0 + x) * G + tok;
            v[p] = *reinterpret_cast<const uint4 *>((at < T ? open + tok * D : src + (size_t)(at - T) * D) + 8 * ch8);
        }
        size_t slot = (size_t)u * a.NB + j0 + x;
        if (a.bt) {
            const int s = a.fstack[a.top - 1 - (t.taken[e] + rel)];
            if (tid == 0 && !val) a.bt[slot] = s;
            slot = (size_t)s;
        }
        // the channels' ranges: over the thread's tokens, the warp's, the CTA's
        uint32_t lo[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, up[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int p = 1; p < PER; ++p) {
            const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                lo[y] = h2min(lo[y], w[y]);
                up[y] = h2max(up[y], w[y]);
            }
        }
#pragma unroll
        for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                lo[y] = h2min(lo[y], __shfl_xor_sync(0xffffffffu, lo[y], o));
                up[y] = h2max(up[y], __shfl_xor_sync(0xffffffffu, up[y], o));
            }
        if (lane < CPR) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                rng[0][warp][4 * lane + y] = lo[y];
                rng[1][warp][4 * lane + y] = up[y];
            }
        }
        __syncthreads();
        float m = 0.0f;
        for (int z = tid; z < D / 2; z += APP_THREADS) {
            uint32_t l = rng[0][0][z], h = rng[1][0][z];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) {
                l = h2min(l, rng[0][w][z]);
                h = h2max(h, rng[1][w][z]);
            }
            if (!val)
                *reinterpret_cast<uint2 *>(a.dig + slot * D + 2 * z) =
                    make_uint2(__byte_perm(l, h, 0x5410), __byte_perm(l, h, 0x7632));
            const float2 fl = __half22float2(ch_as_h2(l)), fh = __half22float2(ch_as_h2(h));
            m = fmaxf(m, fmaxf(fmaxf(fabsf(fl.x), fabsf(fl.y)), fmaxf(fabsf(fh.x), fabsf(fh.y))));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) amax[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) m = fmaxf(m, amax[w]);
        const float inv = m > 0.0f ? __frcp_rn(m) : 0.0f;
        uint8_t *const dst = a.blk + slot * (2 * G * D);
        uint2 c[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            c[p].x = __byte_perm(encode2<FMT>(v[p].x, m, inv), encode2<FMT>(v[p].y, m, inv), 0x5410);
            c[p].y = __byte_perm(encode2<FMT>(v[p].z, m, inv), encode2<FMT>(v[p].w, m, inv), 0x5410);
        }
        if (!val) {
            constexpr int CPL = D / 4;   // channels per lane i
            const int i = 8 * ch8 / CPL, in = 8 * ch8 % CPL, rot = D == 128 ? i >> 1 : 0;
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int tok = tid / CPR + TPI * p, piece = in / 16 + (D / 64) * (tok >> 3 & 1);
                *reinterpret_cast<uint2 *>(dst + (tok >> 4) * (32 * D) + (piece * 32 + 4 * (tok & 7) + i) * 16 +
                                           8 * ((in >> 3 & 1) ^ rot)) = c[p];
            }
            if (tid == 0) a.rec[slot].ks = __fdiv_rn(m, TOP);
        } else {
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                uint32_t *w = rows + ((tid / CPR + TPI * p) * RS + 8 * ch8) / 4;
                w[0] = c[p].x;
                w[1] = c[p].y;
            }
            if (tid == 0) {
                const float vs = __fdiv_rn(m, TOP);
                a.rec[slot].vs = vs;
                a.rec[slot].lv = vs > 0.0f ? log2f(vs) : -40.0f;
                a.rec[slot].iv = vs > 0.0f ? __fdiv_rn(1.0f, vs) : 1099511627776.0f;
            }
            __syncthreads();
            // four channels of lane column i: 4 x 4 bytes turned, four times
            for (int z = tid; z < G * D / 64; z += APP_THREADS) {
                const int i = z & 3, rq = z >> 2 & 1, cc = (z >> 3) % (D / 32), grp = (z >> 3) / (D / 32);
                uint32_t out[4][4];   // [channel of the four][w]
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t b[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        b[y] = rows[((16 * grp + 2 * i + (y & 1) + 8 * (y >> 1)) * RS + 32 * cc + 8 * w + 4 * rq) / 4];
                    const uint32_t p0 = __byte_perm(b[0], b[1], 0x5140), p1 = __byte_perm(b[0], b[1], 0x7362),
                                   p2 = __byte_perm(b[2], b[3], 0x5140), p3 = __byte_perm(b[2], b[3], 0x7362);
                    out[0][w] = __byte_perm(p0, p2, 0x5410);
                    out[1][w] = __byte_perm(p0, p2, 0x7632);
                    out[2][w] = __byte_perm(p1, p3, 0x5410);
                    out[3][w] = __byte_perm(p1, p3, 0x7632);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<uint4 *>(dst + grp * (32 * D) + 16 * D + (cc * 32 + 4 * (4 * rq + y) + i) * 16) =
                        make_uint4(out[y][0], out[y][1], out[y][2], out[y][3]);
            }
        }
    }
    if (x != 0) return;
    // The unit's first CTA copies the tokens that stay open. They may take the
    // rows that it has read above (its barriers lie between).
    const int from = max(T, end / G * G);
    for (int z = tid; z < (end - from) * CPR; z += APP_THREADS) {
        const int at = from + z / CPR;
        *reinterpret_cast<uint4 *>(open + (size_t)(at % G) * D + 8 * (z % CPR)) =
            *reinterpret_cast<const uint4 *>(src + (size_t)(at - T) * D + 8 * (z % CPR));
    }
}

struct ReadArgs {
    const uint8_t *blk;
    const ByteRec *rec;
    const int32_t *bt;
    const __half *tk, *tv;
    __half *K, *V;
    int n, start, Hkv, NB, G, groups, ctas;   // groups of 16 tokens from start / 16 on, CTAs per unit
};
struct ReadTable {
    int T[BYTE_MAX_SEQS];
};

template <int D, int FMT>
__global__ void __launch_bounds__(READ_WARPS * 32)
    k_byte_read(const __grid_constant__ ReadArgs a, const __grid_constant__ ReadTable t) {
    constexpr int CPR = D / 8, RS = D + 8, PP = D / 64;
    __shared__ __align__(16) __half rows[READ_WARPS][16 * RS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, i = lane & 3;
    const int u = (int)(blockIdx.x / (unsigned)a.ctas), x = (int)(blockIdx.x % (unsigned)a.ctas) * READ_WARPS + warp;
    const int T = t.T[u / a.Hkv], stop = (int)min((long long)a.start + a.n, (long long)T);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (x >= a.groups) return;
    const int t0 = (a.start / 16 + x) * 16;   // the group's first token
    if (t0 >= stop) return;
    const int held = T / a.G * a.G;
    __half *const sm = rows[warp];
    const uint8_t *src = nullptr;
    ByteRec rec = {};
    if (t0 < held) {
        const int j = t0 / a.G;
        const size_t own = (size_t)u * a.NB + j, slot = a.bt ? (size_t)a.bt[own] : own;
        src = a.blk + slot * (2 * (size_t)a.G * D) + (t0 % a.G) / 16 * (32 * D);
        const float4 f = *reinterpret_cast<const float4 *>(a.rec + slot);
        rec.ks = f.x;
        rec.vs = f.y;
    }
#pragma unroll
    for (int val = 0; val < 2; ++val) {
        const float s = val ? rec.vs : rec.ks;
        auto scaled = [&](uint32_t h) {
            const float2 f = __half22float2(ch_as_h2(h));
            return ch_h2(__floats2half2_rn(f.x * s, f.y * s));
        };
        if (src) {
            uint4 p[2 * PP];
#pragma unroll
            for (int y = 0; y < 2 * PP; ++y) p[y] = reinterpret_cast<const uint4 *>(src + val * 16 * D)[y * 32 + lane];
#pragma unroll
            for (int y = 0; y < 2 * PP; ++y) {
                const uint32_t w[4] = {p[y].x, p[y].y, p[y].z, p[y].w};
                uint32_t h[8];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    byte_unpack<FMT>(w[z], h[2 * z], h[2 * z + 1]);
                    h[2 * z] = scaled(h[2 * z]);
                    h[2 * z + 1] = scaled(h[2 * z + 1]);
                }
                if (!val) {
                    const int rot = D == 128 ? 8 * (i >> 1) : 0;
                    __half *row = sm + (r + 8 * (y / PP)) * RS + (D / 4) * i + 16 * (y % PP);
                    *reinterpret_cast<uint4 *>(row + rot) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(row + (8 ^ rot)) = make_uint4(h[4], h[5], h[6], h[7]);
                } else {
#pragma unroll
                    for (int z = 0; z < 8; ++z) {   // word z / 2, tokens 2i or 2i + 8
                        uint32_t m;
                        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(m) : "r"(h[z]));
                        *reinterpret_cast<uint32_t *>(sm + (r + 8 * (z & 1)) * RS + 32 * y + 8 * (z >> 1) + 2 * i) = m;
                    }
                }
            }
            __syncwarp();
        }
        const __half *open = (val ? a.tv : a.tk) + ((size_t)u * a.G + (t0 - held)) * D;   // (used where t0 >= held)
        __half *out = val ? a.V : a.K;
#pragma unroll
        for (int y = 0; y < 16 * CPR / 32; ++y) {
            const int row = (y * 32 + lane) / CPR, ch = 8 * (lane % CPR), at = t0 + row;
            if (at >= a.start && at < stop)
                *reinterpret_cast<uint4 *>(out + ((size_t)u * a.n + (at - a.start)) * D + ch) =
                    src ? *reinterpret_cast<const uint4 *>(sm + row * RS + ch)
                        : *reinterpret_cast<const uint4 *>(open + (size_t)row * D + ch);
        }
        __syncwarp();
    }
}

// Free slots: all of them (b < 0), or those of sequence b behind the free ones.
__global__ void k_byte_release(int32_t *fstack, const int32_t *bt, int NB, int Hkv, int b, int nb, int top, int all) {
    const long long n = b < 0 ? all : (long long)nb * Hkv;
    for (long long z = (long long)blockIdx.x * blockDim.x + threadIdx.x; z < n; z += (long long)gridDim.x * blockDim.x)
        fstack[top + z] = b < 0 ? (int32_t)z : bt[((size_t)b * Hkv + z / nb) * NB + z % nb];
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int fail_cuda(ott_byte_cache *c, cudaError_t e) {
    if (e == cudaSuccess) return OTT_OK;
    c->poisoned = 1;
    return OTT_ERR_CUDA;
}

// The cache's device has to be the current one.
int device_of(const ott_byte_cache *c) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return OTT_ERR_CUDA;
    return dev == c->device ? OTT_OK : OTT_ERR_STATE;
}
// The checks of every call, before anything else is looked at.
int state_of(const ott_byte_cache *c) { return c->poisoned ? OTT_ERR_STATE : device_of(c); }

template <int D, int G>
cudaError_t append_t(const AppendArgs &a, const AppendTable &t, int format, int ctas, cudaStream_t s) {
    auto *kern = format == OTT_BYTE_INT ? k_byte_append<D, G, OTT_BYTE_INT> : k_byte_append<D, G, OTT_BYTE_FLOAT>;
    return launch_pdl(kern, dim3((unsigned)ctas, 2), app_threads(D, G), 0, s, a, t);
}

// Sequences [b0, b0 + nb): m[x] tokens each from k, v [nb][Hkv][n][d]; m null: n.
int append(ott_byte_cache *c, int b0, int nb, const __half *k, const __half *v, int n, const int *m, cudaStream_t s) {
    long long blocks = 0;
    bool any = false;
    for (int x = 0; x < nb; ++x) {
        const int T = c->T[b0 + x], mx = m ? m[x] : n;
        if (mx > c->max_tokens - T) return OTT_ERR_CAPACITY;
        blocks += (long long)((T + mx) / c->G - T / c->G) * c->Hkv;
        any |= mx > 0;
    }
    if (c->paged && blocks > c->free_blocks) return OTT_ERR_CAPACITY;
    if (!any) return OTT_OK;
    AppendArgs a;
    a.blk = c->blk;
    a.rec = c->rec;
    a.dig = c->dig;
    a.tk = c->tk;
    a.tv = c->tv;
    a.bt = c->paged ? c->bt : nullptr;
    a.fstack = c->fstack;
    a.n = n;
    a.Hkv = c->Hkv;
    a.NB = c->NB;
    for (int x0 = 0; x0 < nb; x0 += CHUNK_SEQS) {
        AppendTable t;
        a.B0 = b0 + x0;
        a.nseq = std::min(nb - x0, CHUNK_SEQS);
        a.k = k + (size_t)x0 * c->Hkv * n * c->d;
        a.v = v + (size_t)x0 * c->Hkv * n * c->d;
        a.top = (int)c->free_blocks;
        int ctas = 0;
        long long taken = 0;
        for (int y = 0; y < a.nseq; ++y) {
            const int T = c->T[a.B0 + y], mx = m ? m[x0 + y] : n, nblk = (T + mx) / c->G - T / c->G;
            t.base[y] = ctas;
            t.T[y] = T;
            t.m[y] = mx;
            t.taken[y] = (int)taken;
            taken += (long long)nblk * c->Hkv;
            ctas += mx > 0 ? std::max(nblk, 1) * c->Hkv : 0;
        }
        t.base[a.nseq] = ctas;
        if (ctas == 0) continue;
        cudaError_t e = cudaErrorInvalidValue;
#define OTT_APP(D_, G_) \
    if (c->d == D_ && c->G == G_) e = append_t<D_, G_>(a, t, c->format, ctas, s);
        OTT_APP(128, 32) OTT_APP(128, 64) OTT_APP(128, 128) OTT_APP(64, 32) OTT_APP(64, 64) OTT_APP(64, 128)
#undef OTT_APP
        if (e != cudaSuccess) return fail_cuda(c, e);
        if (c->paged) c->free_blocks -= taken;
        for (int y = 0; y < a.nseq; ++y) c->T[a.B0 + y] += t.m[y];
    }
    return OTT_OK;
}

bool lens_ok(const ott_byte_cache *c, int n, const int *lens) {
    for (int b = 0; lens && b < c->B; ++b)
        if (lens[b] < 0 || lens[b] > n) return false;
    return true;
}

int attend(ott_byte_cache *c, const ByteCall &call, void *stream) {
    for (int b = 0; b < c->B; ++b)
        if (c->T[b] > INT_MAX - call.n) return OTT_ERR_INVALID;
    cudaError_t e;
    const int rc = run_byte_attn(c, call, static_cast<cudaStream_t>(stream), e);
    return rc == OTT_ERR_CUDA ? fail_cuda(c, e) : rc;
}

int most_blocks(const ott_byte_cache *c) {
    int t = 0;
    for (int b = 0; b < c->B; ++b) t = std::max(t, c->T[b]);
    return t / c->G;
}

}  // namespace

extern "C" {

int ott_byte_create(int B, int Hq, int Hkv, int d, int G, int format, int max_tokens, long long pool_blocks,
                    ott_byte_cache **out) {
    if (!out) return OTT_ERR_INVALID;
    *out = nullptr;
    if (B < 1 || B > BYTE_MAX_SEQS || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || max_tokens < 0 || (d != 64 && d != 128) ||
        (G != 32 && G != 64 && G != 128) || (format != OTT_BYTE_INT && format != OTT_BYTE_FLOAT) || pool_blocks < 0 ||
        pool_blocks > INT_MAX)
        return OTT_ERR_INVALID;
    const long long NB = max_tokens / G;
    // units, query rows and blocks are counted in 32 bits
    if ((long long)B * Hq > INT_MAX / 512 || (long long)B * Hkv * (NB + 1) > INT_MAX / 8) return OTT_ERR_INVALID;
    int dev = 0, sms = 0, optin = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return OTT_ERR_CUDA;
    ott_byte_cache *c = new (std::nothrow) ott_byte_cache();
    if (!c) return OTT_ERR_OOM;
    c->B = B; c->Hq = Hq; c->Hkv = Hkv; c->d = d; c->G = G;
    c->format = format;
    c->max_tokens = max_tokens;
    c->U = B * Hkv;
    c->g = Hq / Hkv;
    c->NB = (int)NB;
    c->blk_bytes = 2LL * G * d;
    c->device = dev;
    c->sm_count = sms;
    c->smem_optin = optin;
    c->paged = pool_blocks > 0;
    c->pool_blocks = c->free_blocks = pool_blocks;
    try {
        c->T.assign(B, 0);
    } catch (...) {
        delete c;
        return OTT_ERR_OOM;
    }
    const size_t slots = c->paged ? (size_t)pool_blocks : (size_t)c->U * NB;
    // partials of one call on a batch of moderate size; larger ones use stream-ordered scratch
    c->part_floats = (size_t)sms * 16 * 2 * 8 * (d + 2);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = round_up(off + bytes, 256);
        return at;
    };
    const size_t o_blk = take(slots * (size_t)c->blk_bytes), o_rec = take(slots * sizeof(ByteRec)),
                 o_dig = take(slots * d * sizeof(__half2)), o_tk = take((size_t)c->U * G * d * 2),
                 o_tv = take((size_t)c->U * G * d * 2), o_bt = take(c->paged ? (size_t)c->U * NB * 4 : 0),
                 o_fs = take(c->paged ? slots * 4 : 0), o_part = take(c->part_floats * 4), o_ctl = take(64);
    c->mem_bytes = off;
    // host-side fault injection for tests, as in ott_create
    const char *fault = std::getenv("OTT_FAULT");
    void *mem = nullptr;
    if ((fault && std::strcmp(fault, "alloc") == 0) || cudaMalloc(&mem, c->mem_bytes) != cudaSuccess) {
        cudaGetLastError();
        delete c;
        return OTT_ERR_OOM;
    }
    c->mem = mem;
    uint8_t *base = static_cast<uint8_t *>(mem);
    c->blk = base + o_blk;
    c->rec = reinterpret_cast<ByteRec *>(base + o_rec);
    c->dig = reinterpret_cast<__half2 *>(base + o_dig);
    c->tk = reinterpret_cast<__half *>(base + o_tk);
    c->tv = reinterpret_cast<__half *>(base + o_tv);
    c->bt = reinterpret_cast<int32_t *>(base + o_bt);
    c->fstack = reinterpret_cast<int32_t *>(base + o_fs);
    c->part = reinterpret_cast<float *>(base + o_part);
    c->ctl = reinterpret_cast<int *>(base + o_ctl);
    e = cudaMemset(mem, 0, c->mem_bytes);
    if (e == cudaSuccess) e = set_byte_attributes(c);
    if (e == cudaSuccess && c->paged) {
        k_byte_release<<<256, 256>>>(c->fstack, c->bt, c->NB, Hkv, -1, 0, 0, (int)pool_blocks);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaFree(mem);
        delete c;
        return OTT_ERR_CUDA;
    }
    *out = c;
    return OTT_OK;
}

int ott_byte_destroy(ott_byte_cache *c) {
    if (!c) return OTT_OK;
    // any device may be current: the cache's kernels run on its own
    int dev = c->device;
    cudaError_t e = cudaGetDevice(&dev);
    const bool away = dev != c->device;
    if (e == cudaSuccess && away) e = cudaSetDevice(c->device);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    const cudaError_t e2 = cudaFree(c->mem);
    if (e == cudaSuccess) e = e2;
    if (away) {
        const cudaError_t e3 = cudaSetDevice(dev);
        if (e == cudaSuccess) e = e3;
    }
    delete c;
    return e == cudaSuccess ? OTT_OK : OTT_ERR_CUDA;
}

int ott_byte_append(ott_byte_cache *c, const void *k, const void *v, int n, const int *lens, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    if (n < 0 || !lens_ok(c, n, lens)) return OTT_ERR_INVALID;
    if (n == 0) return OTT_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return OTT_ERR_INVALID;
    return append(c, 0, c->B, static_cast<const __half *>(k), static_cast<const __half *>(v), n, lens,
                  static_cast<cudaStream_t>(stream));
}

int ott_byte_append_seq(ott_byte_cache *c, int b, const void *k, const void *v, int n, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    if (b < 0 || b >= c->B || n < 0) return OTT_ERR_INVALID;
    if (n == 0) return OTT_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return OTT_ERR_INVALID;
    return append(c, b, 1, static_cast<const __half *>(k), static_cast<const __half *>(v), n, nullptr,
                  static_cast<cudaStream_t>(stream));
}

int ott_byte_read(ott_byte_cache *c, void *K, void *V, int start, int n, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    if (start < 0 || n < 0) return OTT_ERR_INVALID;
    if (n == 0) return OTT_OK;
    if (!K || !V || !aligned16(K) || !aligned16(V)) return OTT_ERR_INVALID;
    const size_t bytes = (size_t)c->U * n * c->d * 2;
    if (overlap(K, bytes, V, bytes)) return OTT_ERR_INVALID;
    ReadArgs a = {c->blk, c->rec, c->paged ? c->bt : nullptr, c->tk, c->tv, static_cast<__half *>(K),
                  static_cast<__half *>(V), n, start, c->Hkv, c->NB, c->G, 0, 0};
    ReadTable t;
    long long stop = 0;
    for (int b = 0; b < c->B; ++b) {
        t.T[b] = c->T[b];
        stop = std::max<long long>(stop, c->T[b]);
    }
    stop = std::min<long long>(stop, (long long)start + n);
    if (stop <= start) return OTT_OK;
    a.groups = (int)((stop - 1) / 16 - start / 16 + 1);
    a.ctas = (a.groups + READ_WARPS - 1) / READ_WARPS;
    auto *kern = c->d == 128 ? (c->format == OTT_BYTE_INT ? k_byte_read<128, OTT_BYTE_INT> : k_byte_read<128, OTT_BYTE_FLOAT>)
                             : (c->format == OTT_BYTE_INT ? k_byte_read<64, OTT_BYTE_INT> : k_byte_read<64, OTT_BYTE_FLOAT>);
    return fail_cuda(c, launch_pdl(kern, dim3((unsigned)(c->U * a.ctas)), READ_WARPS * 32, 0,
                                   static_cast<cudaStream_t>(stream), a, t));
}

int ott_byte_decode(ott_byte_cache *c, const void *q, void *out, int topk, int32_t *sel, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    for (int b = 0; b < c->B; ++b)
        if (c->T[b] == 0) return OTT_ERR_STATE;
    const size_t nq = (size_t)c->B * c->Hq * c->d * 2;
    if (topk < 0 || !q || !out || !aligned16(q) || !aligned16(out) || overlap(q, nq, out, nq)) return OTT_ERR_INVALID;
    if (topk > 0 && sel) {
        const size_t ns = (size_t)c->U * std::min(topk, most_blocks(c)) * 4;
        if ((reinterpret_cast<uintptr_t>(sel) & 3u) || overlap(sel, ns, q, nq) || overlap(sel, ns, out, nq))
            return OTT_ERR_INVALID;
    }
    ByteCall call = {static_cast<const __half *>(q), nullptr, nullptr, static_cast<__half *>(out), 1, nullptr, topk, sel};
    return attend(c, call, stream);
}

int ott_byte_attn(ott_byte_cache *c, const void *q, const void *k, const void *v, void *out, int n, const int *lens,
                  int topk, int32_t *sel, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    if (n < 0 || topk < 0 || !lens_ok(c, n, lens)) return OTT_ERR_INVALID;
    if (n == 0) return OTT_OK;
    if (!q || !k || !v || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return OTT_ERR_INVALID;
    const size_t nq = (size_t)c->B * c->Hq * n * c->d * 2, nk = (size_t)c->U * n * c->d * 2;
    if (overlap(out, nq, q, nq) || overlap(out, nq, k, nk) || overlap(out, nq, v, nk)) return OTT_ERR_INVALID;
    if (topk > 0 && sel) {
        const size_t ns = (size_t)c->U * n * std::min(topk, most_blocks(c)) * 4;
        if ((reinterpret_cast<uintptr_t>(sel) & 3u) || overlap(sel, ns, q, nq) || overlap(sel, ns, k, nk) ||
            overlap(sel, ns, v, nk) || overlap(sel, ns, out, nq))
            return OTT_ERR_INVALID;
    }
    ByteCall call = {static_cast<const __half *>(q), static_cast<const __half *>(k), static_cast<const __half *>(v),
                     static_cast<__half *>(out), n, lens, topk, sel};
    return attend(c, call, stream);
}

int ott_byte_release(ott_byte_cache *c, int b, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    if (b < 0 || b >= c->B) return OTT_ERR_INVALID;
    const int nb = c->T[b] / c->G;
    if (c->paged && nb > 0) {
        k_byte_release<<<(unsigned)std::min(256LL, ((long long)nb * c->Hkv + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(
            c->fstack, c->bt, c->NB, c->Hkv, b, nb, (int)c->free_blocks, 0);
        if (const int rc = fail_cuda(c, cudaGetLastError())) return rc;
        c->free_blocks += (long long)nb * c->Hkv;
    }
    c->T[b] = 0;
    return OTT_OK;
}

int ott_byte_reset(ott_byte_cache *c, void *stream) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = state_of(c)) return rc;
    if (c->paged && c->free_blocks < c->pool_blocks) {
        k_byte_release<<<256, 256, 0, static_cast<cudaStream_t>(stream)>>>(c->fstack, c->bt, c->NB, c->Hkv, -1, 0, 0,
                                                                          (int)c->pool_blocks);
        if (const int rc = fail_cuda(c, cudaGetLastError())) return rc;
        c->free_blocks = c->pool_blocks;
    }
    std::fill(c->T.begin(), c->T.end(), 0);
    return OTT_OK;
}

int ott_byte_counts(const ott_byte_cache *c, int b, long long *T, int *blocks) {
    if (!c || b < -1 || b >= c->B) return OTT_ERR_INVALID;
    const int t = b < 0 ? *std::max_element(c->T.begin(), c->T.end()) : c->T[b];
    if (T) *T = t;
    if (blocks) *blocks = t / c->G;
    return OTT_OK;
}

long long ott_byte_free_blocks(const ott_byte_cache *c) { return c && c->paged ? c->free_blocks : -1; }

int ott_byte_check(ott_byte_cache *c) {
    if (!c) return OTT_ERR_INVALID;
    if (const int rc = device_of(c)) return rc;
    int flag = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&flag, c->ctl + 1, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return fail_cuda(c, e);
    if (!flag) return OTT_OK;
    c->poisoned = 1;
    return OTT_ERR_DEVICE;
}

long long ott_byte_bytes(const ott_byte_cache *c) { return c ? (long long)c->mem_bytes : 0; }

}  // extern "C"
