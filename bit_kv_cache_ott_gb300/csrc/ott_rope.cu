// ott_rope.cu -- rotary positions with one to four axes, for the queries and
// keys of a decode step or of a chunk, before they are attended and stored.
//
// Pair i of a head's channels turns by the angle pos[axis(i)] * f_i with
// f_i = base^-e_i. The angle of a far position (10^6 radians and more) has
// no fractional digits left in 32 bits, so it is never formed: with
// F_i = 2^64 f_i / 2 pi, cut to a whole number, the 64-bit product pos * F_i,
// wrapped modulo 2^64, is the turn's fraction in units of 2^-64, whole turns
// dropped exactly. Its upper 32 bits, as a signed number of half turns in
// [-1, 1), go to sincospif. The products and sums of a pair are taken in 32 bits and
// rounded once to fp16.
//
// The pass reads and writes every element once and nothing else of size, so
// HBM bounds it. A thread keeps the cosines and sines of 8 pairs of one
// token in registers and walks a run of heads with them, 16 bytes per load,
// ROPE_UNROLL heads in flight: the trigonometry is paid once per run.
// With many tokens a run is all heads; with few (a decode step), runs are
// cut until the threads cover the GPU.
// Measured on one GB300: 40 heads of 32,767 tokens, d = 128 (672 MB read and
// written), 109 us, 6.1 TB/s, 90% of the copy bandwidth; a decode step of 32
// sequences with 32 + 32 heads (1 MB) 3.4 us, launch included.
#include <climits>
#include <cmath>
#include <cstring>

#include "ott_internal.cuh"

namespace ott {
namespace {

constexpr int ROPE_MAX_PAIRS = 128;   // d <= 256
constexpr int ROPE_THREADS = 256;
constexpr int ROPE_UNROLL = 4;        // heads in flight per thread

struct RopeArgs {
    const __half *x[2];      // queries, keys: [B][H][n][d]
    __half *y[2];
    int H[2];
    const int32_t *pos;      // [axes][B][n]
    int B, n, d, half;       // half: rotated pairs
    int interleaved;
    int run;                 // heads per thread
    int runs;                // runs covering all heads
    int groups;              // pair groups per token, then groups of channels left alone
    int rot_groups;
    long long tokens;        // B * n
    uint64_t F[ROPE_MAX_PAIRS];
    uint8_t axis[ROPE_MAX_PAIRS];
};

__device__ __forceinline__ void rope_angle(const RopeArgs &a, int pair, long long tok, float &c, float &s) {
    const long long p = __ldg(a.pos + (size_t)a.axis[pair] * a.tokens + tok);
    const uint64_t turn = (uint64_t)p * a.F[pair];
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }

// Two 16-byte vectors hold 8 pairs: (x0 of 8 pairs, x1 of 8 pairs) in the
// half-split order, 4 adjacent pairs each in the interleaved one.
template <bool IL>
__device__ __forceinline__ void rotate8(uint4 &u, uint4 &w, const float (&c)[8], const float (&s)[8]) {
    uint32_t *a = reinterpret_cast<uint32_t *>(&u), *b = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (IL) {
            const float2 p = unpack2(a[k]), q = unpack2(b[k]);
            a[k] = pack2(p.x * c[k] - p.y * s[k], p.x * s[k] + p.y * c[k]);
            b[k] = pack2(q.x * c[4 + k] - q.y * s[4 + k], q.x * s[4 + k] + q.y * c[4 + k]);
        } else {
            const float2 p = unpack2(a[k]), q = unpack2(b[k]);
            a[k] = pack2(p.x * c[2 * k] - q.x * s[2 * k], p.y * c[2 * k + 1] - q.y * s[2 * k + 1]);
            b[k] = pack2(p.x * s[2 * k] + q.x * c[2 * k], p.y * s[2 * k + 1] + q.y * c[2 * k + 1]);
        }
    }
}

// Pair counts that are multiples of 8: whole vectors. Thread = (token, group
// of 8 pairs or 16 channels left alone, run of heads), groups fastest.
template <bool IL>
__global__ void __launch_bounds__(ROPE_THREADS) k_rope_vec(const __grid_constant__ RopeArgs a) {
    const long long e = (long long)blockIdx.x * ROPE_THREADS + threadIdx.x;
    const int g = (int)(e % a.groups);
    const long long tr = e / a.groups, tok = tr % a.tokens;
    const int r = (int)(tr / a.tokens);
    if (r >= a.runs) return;
    const int b = (int)(tok / a.n), i = (int)(tok % a.n);
    const bool rot = g < a.rot_groups;
    float c[8], s[8];
    int o0, o1;   // the two vectors' channel offsets
    if (rot) {
#pragma unroll
        for (int k = 0; k < 8; ++k) rope_angle(a, 8 * g + k, tok, c[k], s[k]);
        o0 = IL ? 16 * g : 8 * g;
        o1 = IL ? 16 * g + 8 : a.half + 8 * g;
    } else {
        o0 = 2 * a.half + 16 * (g - a.rot_groups);
        o1 = o0 + 8;
    }
    // rows h0 .. h1-1 of the queries' heads followed by the keys'
    const int h0 = r * a.run, h1 = min(h0 + a.run, a.H[0] + a.H[1]);
    auto row = [&](int h, const __half *&src, __half *&dst) {
        const int t = h >= a.H[0];
        const size_t off = (((size_t)b * a.H[t] + (t ? h - a.H[0] : h)) * a.n + i) * a.d;
        src = a.x[t] + off;
        dst = a.y[t] + off;
    };
    for (int h = h0; h < h1; h += ROPE_UNROLL) {
        uint4 u[ROPE_UNROLL], w[ROPE_UNROLL];
#pragma unroll
        for (int k = 0; k < ROPE_UNROLL; ++k)
            if (h + k < h1) {
                const __half *src;
                __half *dst;
                row(h + k, src, dst);
                u[k] = *reinterpret_cast<const uint4 *>(src + o0);
                w[k] = *reinterpret_cast<const uint4 *>(src + o1);
            }
#pragma unroll
        for (int k = 0; k < ROPE_UNROLL; ++k)
            if (h + k < h1) {
                const __half *src;
                __half *dst;
                row(h + k, src, dst);
                if (rot) rotate8<IL>(u[k], w[k], c, s);
                *reinterpret_cast<uint4 *>(dst + o0) = u[k];
                *reinterpret_cast<uint4 *>(dst + o1) = w[k];
            }
    }
}

// Any pair count: thread = (token, pair of channels, run of heads).
__global__ void __launch_bounds__(ROPE_THREADS) k_rope_any(const __grid_constant__ RopeArgs a) {
    const long long e = (long long)blockIdx.x * ROPE_THREADS + threadIdx.x;
    const int g = (int)(e % a.groups);   // pairs, then pairs of channels left alone
    const long long tr = e / a.groups, tok = tr % a.tokens;
    const int r = (int)(tr / a.tokens);
    if (r >= a.runs) return;
    const int b = (int)(tok / a.n), i = (int)(tok % a.n);
    const bool rot = g < a.half;
    float c = 1.0f, s = 0.0f;
    if (rot) rope_angle(a, g, tok, c, s);
    const int o0 = rot && !a.interleaved ? g : 2 * g, o1 = rot && !a.interleaved ? a.half + g : 2 * g + 1;
    const int h1 = min(r * a.run + a.run, a.H[0] + a.H[1]);
    for (int h = r * a.run; h < h1; ++h) {
        const int t = h >= a.H[0];
        const size_t off = (((size_t)b * a.H[t] + (t ? h - a.H[0] : h)) * a.n + i) * a.d;
        const __half p = a.x[t][off + o0], q = a.x[t][off + o1];
        const float pf = __half2float(p), qf = __half2float(q);
        a.y[t][off + o0] = rot ? __float2half_rn(pf * c - qf * s) : p;
        a.y[t][off + o1] = rot ? __float2half_rn(pf * s + qf * c) : q;
    }
}

}  // namespace
}  // namespace ott

extern "C" int ott_rope(const void *q, void *q_out, int Hq, const void *k, void *k_out, int Hkv, const int32_t *pos,
                        int B, int n, int d, const ott_rope_plan *plan, void *stream) {
    using namespace ott;
    if (!plan || B < 1 || n < 0 || Hq < 0 || Hkv < 0 || (long long)Hq + Hkv < 1 || (long long)Hq + Hkv > INT_MAX)
        return OTT_ERR_INVALID;
    if (d < 16 || d % 16 != 0 || d > 2 * ROPE_MAX_PAIRS) return OTT_ERR_INVALID;
    if (plan->axes < 1 || plan->axes > 4 || !(plan->base >= 1.0) || !std::isfinite(plan->base)) return OTT_ERR_INVALID;
    int half = 0;
    for (int x = 0; x < plan->axes; ++x) {
        if (plan->sections[x] < 1 || plan->sections[x] > d / 2) return OTT_ERR_INVALID;
        half += plan->sections[x];
    }
    if (half > d / 2) return OTT_ERR_INVALID;
    if (n == 0) return OTT_OK;
    auto bad = [](const void *p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u); };
    if (!pos || (reinterpret_cast<uintptr_t>(pos) & 3u) || (Hq > 0 && (bad(q) || bad(q_out))) ||
        (Hkv > 0 && (bad(k) || bad(k_out))))
        return OTT_ERR_INVALID;
    // each output is its input (in place) or apart from it, and apart from everything else
    const size_t tok = (size_t)B * n * d * 2, nq = tok * Hq, nk = tok * Hkv, np = (size_t)plan->axes * B * n * 4;
    if (Hq > 0 && ((q != q_out && overlap(q, nq, q_out, nq)) || overlap(q_out, nq, pos, np))) return OTT_ERR_INVALID;
    if (Hkv > 0 && ((k != k_out && overlap(k, nk, k_out, nk)) || overlap(k_out, nk, pos, np))) return OTT_ERR_INVALID;
    if (Hq > 0 && Hkv > 0 && (overlap(q_out, nq, k, nk) || overlap(q_out, nq, k_out, nk) || overlap(q, nq, k_out, nk)))
        return OTT_ERR_INVALID;

    RopeArgs a = {};
    a.x[0] = static_cast<const __half *>(q);
    a.x[1] = static_cast<const __half *>(k);
    a.y[0] = static_cast<__half *>(q_out);
    a.y[1] = static_cast<__half *>(k_out);
    a.H[0] = Hq;
    a.H[1] = Hkv;
    a.pos = pos;
    a.B = B;
    a.n = n;
    a.d = d;
    a.half = half;
    a.interleaved = plan->interleaved != 0;
    a.tokens = (long long)B * n;
    // a plan's frequencies: up to 128 powers, found once per thread and plan
    struct Ladder {
        ott_rope_plan plan;
        bool set = false;
        uint64_t F[ROPE_MAX_PAIRS];
        uint8_t axis[ROPE_MAX_PAIRS];
    };
    static thread_local Ladder lad;
    bool same = lad.set && lad.plan.axes == plan->axes && lad.plan.base == plan->base &&
                (lad.plan.restart != 0) == (plan->restart != 0);
    for (int x = 0; same && x < plan->axes; ++x) same = lad.plan.sections[x] == plan->sections[x];
    if (!same) {
        int i = 0;
        for (int x = 0; x < plan->axes; ++x)
            for (int j = 0; j < plan->sections[x]; ++j, ++i) {
                const double e = plan->restart ? (double)j / plan->sections[x] : (double)i / half;
                lad.F[i] = (uint64_t)std::ldexp(std::pow(plan->base, -e) / 6.283185307179586476925, 64);
                lad.axis[i] = (uint8_t)x;
            }
        lad.plan = *plan;
        lad.set = true;
    }
    std::memcpy(a.F, lad.F, sizeof(uint64_t) * half);
    std::memcpy(a.axis, lad.axis, half);
    const bool vec = half % 8 == 0;
    a.rot_groups = vec ? half / 8 : half;
    a.groups = vec ? d / 16 : d / 2;
    const int H = Hq + Hkv;
    int sms = 152, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return OTT_ERR_CUDA;
    // Runs of all heads where the (token, group) threads cover the GPU; fewer
    // heads per run until they do. A decode step of 32 sequences, 64 heads:
    // 3.4 us by the rule, 20.6 with all heads in one run; 32,767 tokens of 40
    // heads: 109 us by the rule, 347 with a head per run.
    const long long per_run = a.tokens * a.groups, want = (long long)sms * 1024;
    long long runs = (want + per_run - 1) / per_run;
    runs = runs < 1 ? 1 : (runs > H ? H : runs);
    a.run = (int)((H + runs - 1) / runs);
    a.runs = (H + a.run - 1) / a.run;
    const long long blocks = (per_run * a.runs + ROPE_THREADS - 1) / ROPE_THREADS;
    if (blocks > INT_MAX) return OTT_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!vec)
        k_rope_any<<<(unsigned)blocks, ROPE_THREADS, 0, s>>>(a);
    else if (a.interleaved)
        k_rope_vec<true><<<(unsigned)blocks, ROPE_THREADS, 0, s>>>(a);
    else
        k_rope_vec<false><<<(unsigned)blocks, ROPE_THREADS, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? OTT_OK : OTT_ERR_CUDA;
}
