// ott_byte_tiles.cu -- attention of many query rows per kv head over the cache
// held in 8 bits, on the tcgen05 tensor cores.
//
// Mathematics: as in ott_byte_rows.cu. The key tile and the value tile of a
// step hold codes, which are exact in fp16 (or fp16 tokens); a group of 16
// tokens comes with its scales, and the softmax takes
//     z = s * (ks log2(e) / sqrt(d)) + log2(vs),  w = 2^(z - m),  sum += w / vs
// in the multiply-add that it makes anyway and once per group.
//
// A CTA (512 threads, one per SM) serves up to 256 rows of one (sequence, kv
// head), as two tiles of 128 rows (row v = token * g + head) that share every
// step of 112 tokens:
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread per row. S from TMEM,
//                   running maximum (the output is rescaled only when it has
//                   grown by 2^8), weights back into S's columns as fp16, those of
//                   four groups first, whose product starts under the others.
//   warps 8-14      producers: warp w turns group w of each step from codes into
//                   the swizzled key tile and value tile (V transposed; both
//                   K-major), the lanes' pieces being cut for stores that meet all banks.
//   warp 15         issues the products. Order on the tensor pipe:
//                   S0(j), O1(j-1), S1(j), O0(j): while one tile's weights are
//                   computed, the other tile's products run.
// TMEM: S0, S1 (fp32 128 columns, the weights overwrite the first 56), O0, O1.
// Work is cut into steps. Either every CTA gets an equal run of the steps of
// all tiles (a tile cut between CTAs leaves partials, merged by
// k_byte_tiles_combine), or a tile of its own, whichever is estimated to end
// first (plan_byte_tiles). After SUM_STEPS steps of a tile, whoever takes the
// next ones, its sums are carried over in fp32 (finish): the tensor cores
// truncate.
//
// What bounds it: 512 tokens of four sequences over 32K (8 kv heads, 4 heads
// each, d = 128) take 850 to 871 us, 1.27 to 1.31 PFLOP/s; 2,048 over 131K 3.12
// to 3.37 ms, 1.32 to 1.42 (the power limit: by the GPU and what ran before). A
// step is some 2,900 cycles, 1,920 of them products (a score product takes as
// long for 112 keys as for 128: its queries are read at 64 bytes a cycle). The
// rest is the chain that a tile goes through, since S(j+1) takes the place of
// P(j): softmax about 1,500, then O and S, 450 each, and the handing over; no
// part of it alone (with fewer products, no exponentials, no unpacking, or no
// stores of the producers the same call takes 3 to 7% less). Weights handed
// over in one part: 875 us. Not taken, all measured on that call: steps of 80
// tokens whose S(j+1) has columns of its own, so that the softmax never waits
// (1,040: a score product costs the same for 80 keys); that with a warp of
// products per tile (957); a warp of products per tile and six producers, with
// steps of 112 (988); exponentials of one group under the conversions of the
// one before (885: registers spill); loops over the groups (910 to 980).
#include <algorithm>
#include <climits>
#include <cmath>

#include "ott_byte.cuh"
#include "ott_tcgen.cuh"

namespace ott {
namespace {

constexpr int GRPS = 7;              // groups of 16 tokens per step
constexpr int STEP_TOK = 16 * GRPS;
constexpr int ROWS = 128;            // rows of a tile
constexpr int THREADS = 512;
constexpr int PROD0 = 8, MMA_WARP = 15;
constexpr int HALF = 4;              // groups whose weights are handed over first
constexpr int META = 4;              // steps of group metadata in flight
constexpr int HIDDEN = 1;            // its flag: some row does not see some token
constexpr int SUM_STEPS = SUM_TOKENS / STEP_TOK;   // steps whose products stay one sum in TMEM
constexpr int MIN_STEPS = 2;         // steps per CTA at least
constexpr int FIXED = 4;             // a tile's fixed cost (find it, queries, fill the pipeline, output) in steps of 2 us

template <int D>
struct TCfg {
    static constexpr int QB = ROWS * D * 2, KB = ROWS * D * 2, VB = 2 * D * 128;
    static constexpr int OFF_Q = 0, OFF_K = 2 * QB, OFF_V = OFF_K + 2 * KB;
    static constexpr int OFF_POS = OFF_V + 2 * VB;          // int pos[META][STEP_TOK]
    static constexpr int OFF_REC = OFF_POS + META * STEP_TOK * 4;   // ByteRec[META][GRPS], ks times log2(e) / sqrt(d)
    static constexpr int OFF_FLAG = OFF_REC + META * GRPS * 16;     // a byte of flag[META][8] per group
    static constexpr int OFF_STG = (OFF_FLAG + META * 8 + 1023) / 1024 * 1024;   // per producer: 16 fp16 rows
    static constexpr int OFF_BAR = OFF_STG + GRPS * 32 * D;    // barriers, tmem address, abort flag
    static constexpr int SMEM = OFF_BAR + 256 + 1024;       // + alignment to 1024
    static_assert(SMEM <= 227 * 1024, "shared memory");
    __host__ __device__ static constexpr uint32_t S(int t) { return 128u * t; }
    __host__ __device__ static constexpr uint32_t O(int t) { return 256u + (uint32_t)D * t; }
};

enum { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_SFULL = 8, B_PFULL = 10, B_PHALF = 12, B_OFULL = 14, B_COUNT = 15 };

struct TileArgs {
    ByteArgs a;
    int nC;           // CTAs
    long long W;      // places of all tiles: FIXED and its steps each
    float *part;      // [nC][2][D + 2][256]
    int whole;        // CTA i takes tile i whole, else an equal run of steps
};

// A tile pair of a (sequence, kv head): its rows, and the groups that they see.
struct Tile {
    int e, hkv, p;            // entry, kv head, pair
    int rows;                 // valid rows
    int gq, gf, gn;           // groups: of blocks, of the open block, of new tokens
    int sq, steps;            // steps of the blocks' groups, then of the others; all steps
};

__host__ __device__ inline void tile_extent(const ByteArgs &a, const ByteSeq &s, int p, Tile &t) {
    const int v0 = 256 * p, vend = s.nq * a.g;
    t.p = p;
    t.rows = vend - v0 < 256 ? vend - v0 : 256;
    const int last = (v0 + t.rows - 1) / a.g;   // token of the last row
    t.gq = s.T / a.G * (a.G / 16);
    t.gf = (s.T % a.G + 15) / 16;
    t.gn = a.k ? last / 16 + 1 : 0;
    t.sq = (t.gq + GRPS - 1) / GRPS;
    t.steps = t.sq + (t.gf + t.gn + GRPS - 1) / GRPS;
}

// The tile that holds place x, and the place's number in it: a tile has FIXED
// places, so that CTAs with many short tiles get fewer steps, and then its
// steps. Warp-collective.
__device__ __forceinline__ Tile tile_at(const TileArgs &ta, const ByteTable &st, long long x, int &step) {
    const ByteArgs &a = ta.a;
    Tile t;
    {
        int lo = 0, hi = a.nseq;   // the last entry whose base is <= x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (st.e[mid].base <= x) lo = mid;
            else hi = mid;
        }
        t.e = lo;
    }
    const ByteSeq &s = st.e[t.e];
    const unsigned rel = (unsigned)(x - s.base);
    t.hkv = (int)(rel / (unsigned)s.Iu);             // Iu: places of one kv head's tiles
    int left = (int)(rel % (unsigned)s.Iu);
    const int lane = threadIdx.x & 31;
    for (int p0 = 0;; p0 += 32) {                    // ends: s.S tiles hold Iu places
        int n = 0;
        if (p0 + lane < s.S) {
            Tile u;
            tile_extent(a, s, p0 + lane, u);
            n = u.steps + FIXED;
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > left && inc - n <= left);
        if (hit || p0 + 32 >= s.S) {
            const int l = hit ? __ffs(hit) - 1 : 0;
            step = left - __shfl_sync(0xffffffffu, inc - n, l);
            tile_extent(a, s, min(p0 + l, s.S - 1), t);
            return t;
        }
        left -= __shfl_sync(0xffffffffu, inc, 31);
    }
}

// Tile number i of the launch where every CTA takes one: an entry's last rows
// (of all its heads) first, since they see the most.
__device__ __forceinline__ Tile tile_number(const TileArgs &ta, const ByteTable &st, int i) {
    Tile t;
    int lo = 0, hi = ta.a.nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (st.e[mid].ubase <= i) lo = mid;
        else hi = mid;
    }
    const ByteSeq &s = st.e[lo];
    t.e = lo;
    t.hkv = (i - s.ubase) % ta.a.Hkv;
    tile_extent(ta.a, s, s.S - 1 - (i - s.ubase) / ta.a.Hkv, t);
    return t;
}

// The softmax warps and the product warp, each from its own place in the
// code: the tile's queries are in place, the last tile's output is read.
__device__ __forceinline__ void tile_sync() { asm volatile("barrier.sync 1, %0;" ::"n"(32 * (PROD0 + 1)) : "memory"); }

// ---------------------------------------------------------------- producers
// Channels stand in the key rows in their own order, tokens and value rows as
// slot_of and vrow say; outputs are put in order where they are read.
// 16-byte piece ch (8 channels from 8 * ch on) of a row of a key tile.
__device__ __forceinline__ uint32_t piece_at(int row, int ch) {
    return (uint32_t)((ch >> 3) * (ROWS * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}

// A tile's groups of blocks are made first, then the fp16 ones, each kind
// dealt to the 7 warps in runs, so that a warp walks through its blocks. In
// the first loop, round k makes a group while the next one's codes are on
// their way; round -1 only starts the first loads (one copy of the code).
template <int D, int FMT>
struct Producer {
    using C = TCfg<D>;
    static constexpr int PP = D / 64;
    static constexpr int CPR = D / 8, RPI = 32 / CPR;   // 16-byte pieces of an fp16 row, rows per load of a warp
    const TileArgs &ta;
    const ByteArgs &a;
    const ByteSeq &s;
    const Tile &t;
    uint8_t *const sm;
    uint64_t *const bar;
    volatile int *const gave_up;
    const int w, lane, r, i, u;
    uint32_t it;

    __device__ Producer(const TileArgs &ta_, const ByteSeq &s_, const Tile &t_, uint8_t *sm_, uint64_t *bar_,
                        volatile int *gave_up_, uint32_t it_)
        : ta(ta_), a(ta_.a), s(s_), t(t_), sm(sm_), bar(bar_), gave_up(gave_up_), w((threadIdx.x >> 5) - PROD0),
          lane(threadIdx.x & 31), r(lane >> 2), i(lane & 3), u((a.B0 + t.e) * a.Hkv + t.hkv), it(it_) {}
    __device__ void wait(int which) { bar_wait(&bar[which + (it & 1)], ((it >> 1) & 1u) ^ 1u, gave_up); }
    // The group's part of the key tile is written. place (of lane < 16's
    // token): -1: every row sees it, else its number among the new tokens
    // (INT_MAX: none); rec: its scales.
    __device__ void key_done(bool ask, int place, float4 rec) {
        bool hidden = false;
        if (ask) {
            hidden = __any_sync(0xffffffffu, lane < 16 && place > 256 * t.p / a.g);
            if (lane < 16)
                reinterpret_cast<volatile int *>(sm + C::OFF_POS)[(it % META) * STEP_TOK + 16 * w + slot_of(lane)] = place;
        }
        if (lane == 0) {
            *reinterpret_cast<volatile uint8_t *>(sm + C::OFF_FLAG + (it % META) * 8 + w) = hidden ? HIDDEN : 0;
            *reinterpret_cast<float4 *>(sm + C::OFF_REC + ((it % META) * GRPS + w) * 16) =
                make_float4(rec.x * a.sl2, rec.y, rec.z, rec.w);
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar[B_KFULL + (it & 1)]);
    }
    __device__ void value_done() {
        proxy_fence();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar[B_VFULL + (it & 1)]);
        ++it;
    }
    __device__ uint8_t *key_tile() const { return sm + C::OFF_K + (it & 1) * C::KB; }
    // this lane's place in the value tile's row vrow(r)
    __device__ uint8_t *value_at() const {
        return sm + C::OFF_V + (it & 1) * C::VB + (w / 4) * (D * 128) + vrow(r) * 128 +
               (((2 * (w & 3) + (i >> 1)) ^ vrow(r)) << 4) + 8 * (i & 1);
    }

    // Groups x .. x + n - 1 of the blocks (none from gq on).
    __device__ void quantized(int x, int n) {
        const int per = a.G / 16;
        uint4 kr[2 * PP], vr[2 * PP];
        float4 rec = make_float4(0.0f, 0.0f, 0.0f, 0.0f), recn = rec;
        bool have = false;
#pragma unroll 1
        for (int k = -1; k < n; ++k) {
            const int xn = x + k + 1;
            const bool next = k + 1 < n && xn < t.gq;
            const uint8_t *src = nullptr;
            if (next) {
                const size_t own = (size_t)u * a.NB + xn / per, slot = a.bt ? (size_t)a.bt[own] : own;
                src = a.blk + slot * a.blk_bytes + (size_t)(xn % per) * (32 * D);
                recn = *reinterpret_cast<const float4 *>(a.rec + slot);
            }
            if (k >= 0) {
                wait(B_KEMPTY);
                uint8_t *kb = key_tile();
                if (have) {
#pragma unroll
                    for (int th = 0; th < 2; ++th) {
                        const int row = 16 * w + slot_of(r + 8 * th);
#pragma unroll
                        for (int y = 0; y < PP; ++y) {
                            const uint4 c = kr[th * PP + y];
                            uint32_t h[8];
                            byte_unpack<FMT>(c.x, h[0], h[1]);
                            byte_unpack<FMT>(c.y, h[2], h[3]);
                            byte_unpack<FMT>(c.z, h[4], h[5]);
                            byte_unpack<FMT>(c.w, h[6], h[7]);
                            const int pp = PP == 2 ? y ^ (r & 1) : 0, rot = D == 128 ? i >> 1 : 0, ch = (D / 32) * i + 2 * pp;
                            *reinterpret_cast<uint4 *>(kb + piece_at(row, ch + rot)) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4 *>(kb + piece_at(row, ch + (1 ^ rot))) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                    }
                    key_done(false, 0, rec);
                } else {
                    zero_keys(kb);
                    key_done(true, INT_MAX, make_float4(1.0f, 1.0f, 0.0f, 1.0f));
                }
            }
            if (next) {   // in flight under the value tile
#pragma unroll
                for (int y = 0; y < 2 * PP; ++y) {
                    const int piece = PP == 2 ? (y & 2) + ((y & 1) ^ (r & 1)) : y;
                    kr[y] = reinterpret_cast<const uint4 *>(src)[piece * 32 + lane];
                }
            }
            if (k >= 0) {
                wait(B_VEMPTY);
                uint8_t *vb = value_at();
                if (have) {
#pragma unroll
                    for (int c = 0; c < 2 * PP; ++c) {
                        const uint32_t q[4] = {vr[c].x, vr[c].y, vr[c].z, vr[c].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint2 h;
                            byte_unpack<FMT>(q[y], h.x, h.y);
                            *reinterpret_cast<uint2 *>(vb + (32 * c + 8 * y) * 128) = h;
                        }
                    }
                } else {
                    zero_values(vb);
                }
                value_done();
            }
            if (next) {
#pragma unroll
                for (int y = 0; y < 2 * PP; ++y) vr[y] = reinterpret_cast<const uint4 *>(src + 16 * D)[y * 32 + lane];
            }
            have = next;
            rec = recn;
        }
    }

    // n groups from the x-th of the fp16 ones on: the open block's, then the
    // new tokens'; past them, nothing. Keys come through registers, values
    // through shared memory, both under one wait.
    __device__ void plain(int x, int n) {
        uint8_t *const stage = sm + C::OFF_STG + w * (32 * D);   // 16 rows, 16-byte chunks turned by the row
#pragma unroll 1
        for (int y = x; y < x + n; ++y) {
            const bool fresh = y >= t.gf;
            int f = 0, left = 0;   // first token (of the open block, or of the new ones), tokens left
            if (!fresh) {
                f = 16 * y;
                left = s.T % a.G - f;
            } else if (y < t.gf + t.gn) {
                f = 16 * (y - t.gf);
                left = s.nq - f;
            }
            const size_t at = (fresh ? (size_t)u * a.n + f : (size_t)u * a.G + f) * D;
            const __half *ksrc = (fresh ? a.k : a.tk) + at, *vsrc = (fresh ? a.v : a.tv) + at;
            uint4 kr[16 / RPI];
#pragma unroll
            for (int e = 0; e < 16 / RPI; ++e) {
                const int row = RPI * e + lane / CPR;
                kr[e] = make_uint4(0, 0, 0, 0);
                if (row < left) kr[e] = reinterpret_cast<const uint4 *>(ksrc + (size_t)row * D)[lane % CPR];
            }
#pragma unroll
            for (int e = 0; e < 16 / RPI; ++e) {
                const int row = RPI * e + lane / CPR, ch = lane % CPR;
                // no row: zeros (nothing is read)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ch_smem(stage + row * (2 * D) + ((ch ^ (row & 7)) << 4))),
                             "l"(row < left ? reinterpret_cast<const uint8_t *>(vsrc + (size_t)row * D + 8 * ch) : reinterpret_cast<const uint8_t *>(a.q)),
                             "r"(row < left ? 16 : 0)
                             : "memory");
            }
            const int place = lane < left ? (fresh ? f + lane : -1) : INT_MAX;
            wait(B_KEMPTY);
            uint8_t *kb = key_tile();
#pragma unroll
            for (int e = 0; e < 16 / RPI; ++e)
                *reinterpret_cast<uint4 *>(kb + piece_at(16 * w + slot_of(RPI * e + lane / CPR), lane % CPR)) = kr[e];
            key_done(true, place, make_float4(1.0f, 1.0f, 0.0f, 1.0f));
            asm volatile("cp.async.wait_all;" ::: "memory");
            wait(B_VEMPTY);   // (its __syncwarp covers the copies)
            uint8_t *vb = value_at();
            const int row = lane & 15, cb = lane >> 4;   // ldmatrix: the row and block that this lane names
#pragma unroll
            for (int c = 0; c < D / 8; c += 2) {
                uint32_t m[4];   // tokens 0..7 and 8..15 of channels 8c .., then of 8c + 8 ..
                asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                             : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
                             : "r"(ch_smem(stage + row * (2 * D) + (((c + cb) ^ (row & 7)) << 4)))
                             : "memory");
                *reinterpret_cast<uint2 *>(vb + 8 * c * 128) = make_uint2(m[0], m[1]);
                *reinterpret_cast<uint2 *>(vb + 8 * (c + 1) * 128) = make_uint2(m[2], m[3]);
            }
            value_done();
        }
    }

    __device__ void zero_keys(uint8_t *kb) const {
#pragma unroll 1
        for (int e = lane; e < 16 * CPR; e += 32)
            *reinterpret_cast<uint4 *>(kb + piece_at(16 * w + e / CPR, e % CPR)) = make_uint4(0, 0, 0, 0);
    }
    __device__ static void zero_values(uint8_t *vb) {
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint2 *>(vb + 8 * c * 128) = make_uint2(0u, 0u);
    }
};

template <int D, int FMT>
__device__ void produce(const TileArgs &ta, const ByteSeq &s, const Tile &t, uint8_t *sm, uint64_t *bar,
                        volatile int *gave_up, int j0, int j1, uint32_t it) {
    Producer<D, FMT> p(ta, s, t, sm, bar, gave_up, it);
    if (j0 < t.sq) p.quantized(p.w * t.sq + j0, min(j1, t.sq) - j0);
    if (j1 > t.sq) p.plain(p.w * (t.steps - t.sq) + max(j0 - t.sq, 0), j1 - max(j0, t.sq));
}

// ---------------------------------------------------------------- products
template <int D>
__device__ void multiply(uint8_t *sm, uint64_t *bar, volatile int *gave_up, uint32_t tmem, int nt, int steps, uint32_t it,
                         uint32_t c0, uint32_t c1) {
    using C = TCfg<D>;
    const uint32_t base = ch_smem(sm), dq = desc_lo(base + C::OFF_Q), dk = desc_lo(base + C::OFF_K),
                   dv = desc_lo(base + C::OFF_V);
    auto scores = [&](int t, int slot) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            constexpr uint32_t HI = desc_hi(1024, 2);
            const uint32_t off = ((k / 4) * (ROWS * 128) + (k & 3) * 32) / 16;
            mma_ss(tmem + C::S(t), dq + t * (C::QB / 16) + off, dk + slot * (C::KB / 16) + off, HI, instr_desc(STEP_TOK), k > 0);
        }
    };
    auto values = [&](int t, int slot, bool acc, int k0, int k1) {
#pragma unroll
        for (int k = k0; k < k1; ++k) {
            constexpr uint32_t HI = desc_hi(1024, 2);
            mma_ts(tmem + C::O(t), tmem + C::S(t) + 8 * k, dv + slot * (C::VB / 16) + ((k / 4) * (D * 128) + (k & 3) * 32) / 16, HI, instr_desc(D),
                   acc || k > 0);
        }
    };
    // the whole warp keeps the loop, so that the operands stay in uniform
    // registers; one lane issues
    for (int j = 0; j < steps; ++j, ++it) {
        const int slot = it & 1, prev = slot ^ 1;
        const uint32_t par = (it >> 1) & 1u;
        bar_wait(&bar[B_KFULL + slot], par, gave_up);
        tc_after();
        if (elect_one()) {
            scores(0, slot);
            tc_commit(&bar[B_SFULL]);
        }
        __syncwarp();
        if (nt == 2) {
            if (j > 0) {
                bar_wait(&bar[B_PHALF + 1], (c1 - 1) & 1u, gave_up);
                tc_after();
                if (elect_one()) values(1, prev, j > 1, 0, HALF);
                __syncwarp();
                bar_wait(&bar[B_PFULL + 1], (c1 - 1) & 1u, gave_up);
            }
            tc_after();
            if (elect_one()) {
                if (j > 0) {
                    values(1, prev, true, HALF, GRPS);
                    tc_commit(&bar[B_VEMPTY + prev]);
                }
                scores(1, slot);
                tc_commit(&bar[B_SFULL + 1]);
                tc_commit(&bar[B_KEMPTY + slot]);
            }
            ++c1;
        } else {
            if (elect_one()) tc_commit(&bar[B_KEMPTY + slot]);
        }
        __syncwarp();
        bar_wait(&bar[B_VFULL + slot], par, gave_up);
        bar_wait(&bar[B_PHALF], c0 & 1u, gave_up);
        tc_after();
        if (elect_one()) values(0, slot, j > 0, 0, HALF);
        __syncwarp();
        bar_wait(&bar[B_PFULL], c0 & 1u, gave_up);
        ++c0;
        tc_after();
        if (elect_one()) {
            values(0, slot, true, HALF, GRPS);
            if (nt == 1) tc_commit(&bar[B_VEMPTY + slot]);
        }
        __syncwarp();
    }
    const int last = (it - 1) & 1;
    if (nt == 2) {
        bar_wait(&bar[B_PHALF + 1], (c1 - 1) & 1u, gave_up);
        bar_wait(&bar[B_PFULL + 1], (c1 - 1) & 1u, gave_up);
    }
    tc_after();
    if (elect_one()) {
        if (nt == 2) {
            values(1, last, steps > 1, 0, GRPS);
            tc_commit(&bar[B_VEMPTY + last]);
        }
        tc_commit(&bar[B_OFULL]);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- softmax
// Scales of group k of a step: (ks log2(e) / sqrt(d), vs, log2(vs), 1 / vs).
__device__ __forceinline__ float4 rec_at(uint32_t at, int k) {
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(at + 16 * k));
    return r;
}
template <int D>
__device__ void softmax(const TileArgs &ta, const ByteSeq &s, const Tile &t, uint8_t *sm, uint64_t *bar,
                        volatile int *gave_up, uint32_t tmem, int tile, int steps, uint32_t it, uint32_t cnt, float &m_ref,
                        float &l) {
    using C = TCfg<D>;
    const ByteArgs &a = ta.a;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(32 * wq) << 16;
    const uint32_t ts = tmem + C::S(tile) + lanes, to = tmem + C::O(tile) + lanes;
    const int row = ROWS * tile + 32 * wq + lane;
    const int tok = (256 * t.p + min(row, t.rows - 1)) / a.g;
    m_ref = -CUDART_INF_F;
    l = 0.0f;
    for (int j = 0; j < steps; ++j, ++it, ++cnt) {
        bar_wait(&bar[B_SFULL + tile], cnt & 1u, gave_up);
        tc_after();
        // groups with a token that some row does not see: -inf into its scores
        const int ms = it % META;
        const uint32_t recs = ch_smem(sm + C::OFF_REC) + ms * GRPS * 16;
        unsigned long long flags = *reinterpret_cast<const volatile unsigned long long *>(sm + C::OFF_FLAG + ms * 8);
        if (flags) {
            const volatile int *tp = reinterpret_cast<volatile int *>(sm + C::OFF_POS) + ms * STEP_TOK;
#pragma unroll 1
            for (int k = 0; k < GRPS; ++k, flags >>= 8)
                if (flags & 0xff) {
                    float f[16];
                    tm_ld16(ts + 16 * k, f);
                    wait_ld();
                    tie16(f);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (tp[16 * k + c] > tok) f[c] = -CUDART_INF_F;
                    tm_st16(ts + 16 * k, f);
                }
            wait_st();
        }
        // The maximum: groups 4..6 first, then 0..3, which stay in registers
        // (64 of them; 4..6 are read again below, behind the weights of 0..3,
        // whose columns they do not share).
        float x[64];
#pragma unroll
        for (int k = 4; k < GRPS; ++k) tm_ld16(ts + 16 * k, x + 16 * (k - 4));
        wait_ld();
#pragma unroll
        for (int k = 0; k < 3; ++k) tie16(x + 16 * k);
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int k = 4; k < GRPS; ++k) {
            const float4 rc = rec_at(recs, k);
            mx = fmaxf(mx, fmaf(max16(x + 16 * (k - 4)), rc.x, rc.z));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) tm_ld16(ts + 16 * k, x + 16 * k);
        wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) tie16(x + 16 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 rc = rec_at(recs, k);
            mx = fmaxf(mx, fmaf(max16(x + 16 * k), rc.x, rc.z));
        }
        const bool grow = mx > m_ref + GROW && m_ref != -CUDART_INF_F;
        if (__any_sync(0xffffffffu, grow)) {
            // the previous step's products are complete (the scores were issued behind them)
            const float al = grow ? ch_ex2(m_ref - mx) : 1.0f;
            l *= al;
            if (grow) m_ref = mx;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                float o[16];
                tm_ld16(to + c, o);
                wait_ld();
                tie16(o);
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] *= al;
                tm_st16(to + c, o);
            }
        }
        if (m_ref == -CUDART_INF_F) m_ref = mx;   // the first token that the row sees: its output is zero so far
        const float mm = m_ref == -CUDART_INF_F ? 0.0f : m_ref - LIFT;
        auto weights = [&](int k, const float *y) {
            const float4 rc = rec_at(recs, k);
            const float2 ad = make_float2(rc.z - mm, rc.z - mm), sc = make_float2(rc.x, rc.x);
            float2 sum = make_float2(0.0f, 0.0f);
            uint32_t p8[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 v = __ffma2_rn(make_float2(y[2 * c], y[2 * c + 1]), sc, ad);
                const float2 p = make_float2(ch_ex2(v.x), ch_ex2(v.y));
                sum = __fadd2_rn(sum, p);
                p8[c] = ch_h2(__floats2half2_rn(p.x, p.y));
            }
            tm_st8(ts + 8 * k, p8);
            l = fmaf(sum.x + sum.y, rc.w, l);
        };
        weights(0, x);
        weights(1, x + 16);
        weights(2, x + 32);
        tm_ld16(ts + 64, x);
        tm_ld16(ts + 80, x + 16);
        tm_ld16(ts + 96, x + 32);
        weights(3, x + 48);
        wait_st();
        wait_ld();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar[B_PHALF + tile]);
        tie16(x);
        tie16(x + 16);
        tie16(x + 32);
        weights(4, x);
        weights(5, x + 16);
        weights(6, x + 32);
        wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&bar[B_PFULL + tile]);
    }
}

// The output of a tile's row, or its part of it (the reference of its weights,
// their sum, the output: a column of rows each). more: the part holds the
// sums of earlier steps, which these join. Warps of the softmax.
template <int D>
__device__ void finish(const TileArgs &ta, const Tile &t, uint32_t tmem, int tile, bool whole, bool more, int slot, float m,
                       float l) {
    using C = TCfg<D>;
    const ByteArgs &a = ta.a;
    const int wq = (threadIdx.x >> 5) & 3, row = ROWS * tile + 32 * wq + (threadIdx.x & 31), v = 256 * t.p + row;
    const uint32_t to = tmem + C::O(tile) + ((uint32_t)(32 * wq) << 16);
    float *pb = ta.part + ((size_t)blockIdx.x * 2 + slot) * (D + 2) * 256 + row;
    if (more) {
        const float mo = pb[0], M = fmaxf(mo, m), mr = M == -CUDART_INF_F ? 0.0f : M;
        const float sn = ch_ex2(m - mr), so = ch_ex2(mo - mr);
        l = fmaf(l, sn, pb[256] * so);
        const size_t at = (((size_t)(a.B0 + t.e) * a.Hq + t.hkv * a.g + v % a.g) * a.n + v / a.g) * D;
        const float inv = whole && row < t.rows ? 1.0f / l : 0.0f;
        pb[0] = M;
        pb[256] = l;
        constexpr int CH = 32;   // channels whose loads are in flight together
#pragma unroll 1
        for (int c = 0; c < D; c += CH) {
            float f[CH], o[CH];
#pragma unroll
            for (int y = 0; y < CH; ++y) o[y] = pb[(size_t)(2 + c + y) * 256];
            tm_ld16(to + c, f);
            tm_ld16(to + c + 16, f + 16);
            wait_ld();
            tie16(f);
            tie16(f + 16);
#pragma unroll
            for (int y = 0; y < CH; ++y) o[y] = fmaf(f[(y & 24) + vrow(y & 7)], sn, o[y] * so);
            if (!whole) {
#pragma unroll
                for (int y = 0; y < CH; ++y) pb[(size_t)(2 + c + y) * 256] = o[y];
            } else if (row < t.rows) {
#pragma unroll
                for (int y = 0; y < CH; y += 8)
                    *reinterpret_cast<uint4 *>(a.out + at + c + y) =
                        make_uint4(ch_h2(__floats2half2_rn(o[y] * inv, o[y + 1] * inv)), ch_h2(__floats2half2_rn(o[y + 2] * inv, o[y + 3] * inv)),
                                   ch_h2(__floats2half2_rn(o[y + 4] * inv, o[y + 5] * inv)), ch_h2(__floats2half2_rn(o[y + 6] * inv, o[y + 7] * inv)));
            }
        }
    } else if (whole) {
        const size_t at = (((size_t)(a.B0 + t.e) * a.Hq + t.hkv * a.g + v % a.g) * a.n + v / a.g) * D;
        const float inv = row < t.rows ? 1.0f / l : 0.0f;
        __half *o = a.out + at;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            float f[16];
            tm_ld16(to + c, f);
            wait_ld();
            tie16(f);
            uint32_t h[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {   // channels 2y, 2y + 1 of the 16, from their columns
                const int c0 = (2 * y & 8) + vrow(2 * y & 7), c1 = (2 * y & 8) + vrow((2 * y & 7) + 1);
                h[y] = ch_h2(__floats2half2_rn(f[c0] * inv, f[c1] * inv));
            }
            if (row < t.rows) {
                *reinterpret_cast<uint4 *>(o + c) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(o + c + 8) = make_uint4(h[4], h[5], h[6], h[7]);
            }
        }
    } else {
        pb[0] = m;
        pb[256] = l;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            float f[16];
            tm_ld16(to + c, f);
            wait_ld();
            tie16(f);
#pragma unroll
            for (int y = 0; y < 16; ++y) pb[(size_t)(2 + c + y) * 256] = f[(y & 8) + vrow(y & 7)];
        }
    }
    tc_before();
}

enum { SOFTMAX, MULTIPLY, PRODUCE };

// A CTA's run of steps, tile by tile, in one of its roles. The roles have
// loops of their own, so that each keeps to its own registers. The producers
// run on into the next tile while the last one's output is read and the next
// one's queries are fetched.
template <int D, int FMT, int ROLE>
__device__ void role_loop(const TileArgs &ta, const ByteTable &st, uint8_t *sm, uint64_t *bar, volatile int *gave_up,
                          uint32_t tmem) {
    using C = TCfg<D>;
    const ByteArgs &a = ta.a;
    // (places from the run's start on: fewer registers than the places)
    int done = 0;
    const long long x0 = ta.whole ? 0 : ch_range_start(ta.W, ta.nC, blockIdx.x);
    const int todo = ta.whole ? 1 : (int)(ch_range_start(ta.W, ta.nC, blockIdx.x + 1) - x0);
    uint32_t it = 0, ct[2] = {0, 0};   // steps done by the CTA, and by each tile
    for (uint32_t run = 0; done < todo;) {
        int at = 0;
        const Tile t = ta.whole ? tile_number(ta, st, blockIdx.x) : tile_at(ta, st, x0 + done, at);
        const ByteSeq &s = st.e[t.e];
        const int j0 = max(0, at - FIXED);
        const int end = ta.whole ? t.steps + FIXED : min(min(t.steps, j0 + SUM_STEPS) + FIXED, at + (todo - done));
        const int j1 = max(0, end - FIXED), n = j1 - j0;
        const int jf = ta.whole ? 0 : max(0, at - done - FIXED);   // the CTA's first step of the tile
        const int slot = done > at;   // a tile that the run starts in or with leaves its part in slot 0, a later one in slot 1
        done += ta.whole ? 1 : end - at;
        if (n == 0) continue;   // the run ends before the tile's steps
        const int nt = t.rows > ROWS ? 2 : 1;
        if constexpr (ROLE == SOFTMAX) {
            // queries into the swizzled tiles, rows past the last zero; a
            // warp takes rows 8 or 16 apart, its loads in flight together
            constexpr int CPR = D / 8, RPW = 32 / CPR, STEP = PROD0 * RPW, BATCH = 8;
            const int ch = threadIdx.x % CPR, r0 = threadIdx.x / CPR;
            const __half *const q0 = a.q + (size_t)(a.B0 + t.e) * a.Hq * a.n * D + (size_t)t.hkv * a.g * a.n * D + 8 * ch;
#pragma unroll 1
            for (int rr = j0 > jf ? nt * ROWS : r0; rr < nt * ROWS; rr += STEP * BATCH) {   // (still there for a tile's next steps)
                uint4 v[BATCH];
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    const int row = rr + STEP * y, vv = 256 * t.p + row, tk = vv / a.g;
                    v[y] = make_uint4(0, 0, 0, 0);
                    if (row < t.rows) v[y] = *reinterpret_cast<const uint4 *>(q0 + ((size_t)(vv - tk * a.g) * a.n + tk) * D);
                }
#pragma unroll
                for (int y = 0; y < BATCH; ++y) {
                    const int row = rr + STEP * y;
                    *reinterpret_cast<uint4 *>(sm + C::OFF_Q + row / ROWS * C::QB + piece_at(row % ROWS, ch)) = v[y];
                }
            }
            proxy_fence();
            tile_sync();
            const int tile = threadIdx.x / ROWS;
            if (tile < nt) {
                float m, l;
                softmax<D>(ta, s, t, sm, bar, gave_up, tmem, tile, n, it, ct[tile], m, l);
                bar_wait(&bar[B_OFULL], run & 1u, gave_up);
                tc_after();
                finish<D>(ta, t, tmem, tile, jf == 0 && j1 == t.steps, j0 > jf, slot, m, l);
            } else {
                bar_wait(&bar[B_OFULL], run & 1u, gave_up);   // its products may still read the queries
            }
        } else if constexpr (ROLE == MULTIPLY) {
            tile_sync();
            tc_after();
            multiply<D>(sm, bar, gave_up, tmem, nt, n, it, ct[0], ct[1]);
        } else {
            produce<D, FMT>(ta, s, t, sm, bar, gave_up, j0, j1, it);
        }
        it += (uint32_t)n;
        ct[0] += (uint32_t)n;
        if (nt == 2) ct[1] += (uint32_t)n;
        ++run;
    }
}

template <int D, int FMT>
__global__ void __launch_bounds__(THREADS, 1)
    k_byte_tiles(const __grid_constant__ TileArgs ta, const __grid_constant__ ByteTable st) {
    using C = TCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (ch_smem(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(sm + C::OFF_BAR + 192);
    volatile int *gave_up = reinterpret_cast<volatile int *>(sm + C::OFF_BAR + 196);
    const ByteArgs &a = ta.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int k = 0; k < 2; ++k) {
            bar_init(&bar[B_KFULL + k], GRPS);
            bar_init(&bar[B_VFULL + k], GRPS);
            bar_init(&bar[B_KEMPTY + k], 1);
            bar_init(&bar[B_VEMPTY + k], 1);
            bar_init(&bar[B_SFULL + k], 1);
            bar_init(&bar[B_PFULL + k], ROWS / 32);
            bar_init(&bar[B_PHALF + k], ROWS / 32);
        }
        bar_init(&bar[B_OFULL], 1);
        *gave_up = 0;
        for (int k = 0; k < META; ++k) *reinterpret_cast<unsigned long long *>(sm + C::OFF_FLAG + 8 * k) = 0;   // byte 7 stays
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ch_smem(tm)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tm, 0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp < PROD0) {
        role_loop<D, FMT, SOFTMAX>(ta, st, sm, bar, gave_up, tmem);
    } else {
        if (warp == MMA_WARP)
            role_loop<D, FMT, MULTIPLY>(ta, st, sm, bar, gave_up, tmem);
        else
            role_loop<D, FMT, PRODUCE>(ta, st, sm, bar, gave_up, tmem);
    }
    __syncthreads();
    if (*gave_up && threadIdx.x == 0) atomicExch(&a.ctl[1], 1);
    if (warp == MMA_WARP) {
        // after a wait that gave up, products may still be in flight: one more bounded wait for them
        if (*gave_up && lane == 0) {
            bar_init(&bar[B_COUNT], 1);
            tc_commit(&bar[B_COUNT]);
            const unsigned long long end = now_ns() + 1000000000ull;
            while (!bar_try(&bar[B_COUNT], 0) && now_ns() < end) {
            }
        }
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Merge the parts of the tiles that CTAs share: 32 rows per CTA, lane = row,
// D / 8 channels per warp.
template <int D>
__global__ void __launch_bounds__(256) k_byte_tiles_combine(const __grid_constant__ TileArgs ta, const __grid_constant__ ByteTable st) {
    const ByteArgs &a = ta.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the tile: x = (pair of the largest sequence, 32 rows), y = kv head, z = entry
    const ByteSeq &s = st.e[blockIdx.z];
    const int p = blockIdx.x / 8, row = 32 * (blockIdx.x % 8) + lane;
    // A CTA with nothing to merge leaves at once, but the first one, which
    // waits in any case: this grid ends behind the tiles.
    const bool first = (blockIdx.x | blockIdx.y | blockIdx.z) == 0;
    if (p >= s.S && !first) return;
    Tile t;
    long long ts = s.base + (long long)blockIdx.y * s.Iu;
    {
        long long before = 0;
        for (int q = lane; q < p; q += 32) {
            tile_extent(a, s, q, t);
            before += t.steps + FIXED;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        ts += before;
    }
    tile_extent(a, s, p, t);
    if (32 * (blockIdx.x % 8) >= t.rows && !first) return;
    const int c0 = ch_warp_of(ta.W, ta.nC, ts + FIXED), c1 = ch_warp_of(ta.W, ta.nC, ts + FIXED + t.steps - 1);
    const int slot0 = ch_range_start(ta.W, ta.nC, c0) < ts ? 1 : 0;
    if (c0 == c1 && !first) return;   // written whole
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c0 == c1 || p >= s.S || t.rows <= 0) return;
    constexpr int CH = D / 8;
    float M = -CUDART_INF_F, L = 0.0f, acc[CH];
#pragma unroll
    for (int y = 0; y < CH; ++y) acc[y] = 0.0f;
    constexpr int AHEAD = 4;   // parts whose loads are in flight together
    for (int c = c0; c <= c1; c += AHEAD) {
        float m[AHEAD], l[AHEAD], f[AHEAD][CH];
#pragma unroll
        for (int z = 0; z < AHEAD; ++z) {
            const int cc = min(c + z, c1);
            const float *pb = ta.part + ((size_t)cc * 2 + (cc == c0 ? slot0 : 0)) * (D + 2) * 256 + row;
            m[z] = c + z <= c1 ? pb[0] : -CUDART_INF_F;
            l[z] = pb[256];
#pragma unroll
            for (int y = 0; y < CH; ++y) f[z][y] = pb[(size_t)(2 + CH * warp + y) * 256];
        }
        float mn = M;
#pragma unroll
        for (int z = 0; z < AHEAD; ++z) mn = fmaxf(mn, m[z]);
        // (no maximum yet: nothing seen, or scores that are NaN, and then the sum, too, which stays)
        const float mr = mn == -CUDART_INF_F ? 0.0f : mn, so = ch_ex2(M - mr);
        L *= so;
#pragma unroll
        for (int y = 0; y < CH; ++y) acc[y] *= so;
#pragma unroll
        for (int z = 0; z < AHEAD; ++z) {
            const float sn = ch_ex2(m[z] - mr);
            L = fmaf(l[z], sn, L);
#pragma unroll
            for (int y = 0; y < CH; ++y) acc[y] = fmaf(f[z][y], sn, acc[y]);
        }
        M = mn;
    }
    if (row >= t.rows) return;
    const int vv = 256 * p + row;
    const size_t at = (((size_t)(a.B0 + blockIdx.z) * a.Hq + blockIdx.y * a.g + vv % a.g) * a.n + vv / a.g) * D;
    const float inv = 1.0f / L;   // a row sees a token at least: 0 only beside scores of -inf, then NaN
    __half *o = a.out + at + CH * warp;
#pragma unroll
    for (int y = 0; y < CH; y += 8)
        *reinterpret_cast<uint4 *>(o + y) = make_uint4(
            ch_h2(__floats2half2_rn(acc[y] * inv, acc[y + 1] * inv)), ch_h2(__floats2half2_rn(acc[y + 2] * inv, acc[y + 3] * inv)),
            ch_h2(__floats2half2_rn(acc[y + 4] * inv, acc[y + 5] * inv)), ch_h2(__floats2half2_rn(acc[y + 6] * inv, acc[y + 7] * inv)));
}

template <int D, int FMT>
cudaError_t launch_t(const TileArgs &ta, const ByteTable &st, int rows, cudaStream_t s) {
    cudaError_t e = launch_pdl(k_byte_tiles<D, FMT>, dim3((unsigned)ta.nC), THREADS, (size_t)TCfg<D>::SMEM, s, ta, st);
    if (e != cudaSuccess || ta.nC == 1 || ta.whole) return e;
    return launch_pdl(k_byte_tiles_combine<D>, dim3((unsigned)((rows + 31LL) / 32), (unsigned)ta.a.Hkv, (unsigned)ta.a.nseq), 256, 0, s, ta, st);
}

template <int D, int FMT>
cudaError_t attribute() {
    return cudaFuncSetAttribute(k_byte_tiles<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<D>::SMEM);
}

}  // namespace

cudaError_t set_byte_tiles_attributes(int d, int format) {
    if (format == OTT_BYTE_INT) return d == 128 ? attribute<128, OTT_BYTE_INT>() : attribute<64, OTT_BYTE_INT>();
    return d == 128 ? attribute<128, OTT_BYTE_FLOAT>() : attribute<64, OTT_BYTE_FLOAT>();
}

// The launch's table in tiles: S pairs of tiles per kv head, Iu their steps.
// false: the sizes do not fit the kernel's 32-bit counters.
bool plan_byte_tiles(const ott_byte_cache *c, ByteArgs &a, ByteTable &st, int &nC, bool &whole, size_t &part_floats) {
    if (a.Hkv > 65535) return false;   // a grid dimension of the merge
    long long base = 0, tiles = 0;
    int longest = 0;
    for (int x = 0; x < a.nseq; ++x) {
        ByteSeq &s = st.e[x];
        s.base = base;
        s.ubase = (int)tiles;
        s.S = (int)(((long long)s.nq * a.g + 255) / 256);
        long long steps = 0;
        if ((long long)s.T + s.nq > INT_MAX - 4096) return false;
        for (int p = 0; p < s.S; ++p) {
            Tile t;
            tile_extent(a, s, p, t);
            steps += t.steps + FIXED;
            longest = std::max(longest, t.steps);
            if (steps * a.Hkv > INT_MAX) return false;
        }
        s.Iu = (int)steps;
        base += steps * a.Hkv;
        tiles += (long long)s.S * a.Hkv;
        if (tiles > INT_MAX) return false;
    }
    st.e[a.nseq] = ByteSeq{};
    st.e[a.nseq].base = a.W = base;
    st.e[a.nseq].ubase = (int)tiles;
    const double sms = c->sm_count, W = (double)base, nT = (double)tiles;
    // Equal runs of places, or a tile per CTA: by their estimated times, as
    // plan_tiles of ott_chunk_tiles.cu (cut tiles and their merge cost 8 steps
    // and 0.1 per part of a tile).
    const double one = std::max<double>(FIXED + longest, std::min(W / sms + longest / 2.0, std::ceil(nT / sms) * (FIXED + longest)));
    double best = 1e30;
    for (int div = 1; div <= 4; div *= 2) {
        const long long n = std::max<long long>(1, std::min<long long>(c->sm_count, (base - FIXED * tiles) / MIN_STEPS) / div);
        const double run = W / n, cost = FIXED + run + (n > 1 ? 8 + 0.1 * (W / nT) / run : 0);
        if (div > 1 && run > INT_MAX / 2) break;   // a run's places are counted in 32 bits
        if (cost < best) {
            best = cost;
            nC = (int)n;
        }
    }
    whole = longest <= SUM_STEPS && one <= best;
    if (whole) nC = (int)tiles;
    part_floats = !whole && (nC > 1 || longest > SUM_STEPS) ? (size_t)nC * 2 * (c->d + 2) * 256 : 1;
    return true;
}

cudaError_t launch_byte_tiles(const ott_byte_cache *c, const ByteArgs &a, const ByteTable &st, int nC, bool whole,
                              cudaStream_t s) {
    TileArgs ta;
    ta.a = a;
    ta.nC = nC;
    ta.W = a.W;
    ta.part = a.part;
    ta.whole = whole;
    int rows = 0;
    for (int x = 0; x < a.nseq; ++x) rows = std::max(rows, st.e[x].nq * a.g);   // at most Hq * n
    const bool i8 = c->format == OTT_BYTE_INT;
    return c->d == 128 ? (i8 ? launch_t<128, OTT_BYTE_INT>(ta, st, rows, s) : launch_t<128, OTT_BYTE_FLOAT>(ta, st, rows, s))
                       : (i8 ? launch_t<64, OTT_BYTE_INT>(ta, st, rows, s) : launch_t<64, OTT_BYTE_FLOAT>(ta, st, rows, s));
}

}  // namespace ott
