// ott_chunk_tiles.cu -- attention of many query rows per kv head over the OTT
// stores (ott_chunk_attn with long chunks), on the tcgen05 tensor cores.
//
// Mathematics: as in ott_chunk.cu (exact key operand s * (code - 1), the
// rows' q . (z + s) apart; weights and values rounded to fp16). The offset
// q . z + q . s comes out of the same product: next to 112 tokens the key
// tile of a step holds, for each of its 7 groups of 16 tokens, the zeros and
// the scales of the group's block as rows 112 + 2w and 113 + 2w. One 128 x
// 128 product then gives the raw scores and the offsets; the softmax adds a
// group's offset to its 16 columns inside the multiply-add that it makes
// anyway. A group may come from any block or be 16 fp16 tokens (those two
// rows zero), so blocks of any size, lists of blocks, rings and pools pack
// into full steps.
//
// A CTA (512 threads, one per SM) serves up to 256 rows of one (sequence, kv
// head), as two tiles of 128 rows (row v = token * g + head) that share every
// dequantized step:
//   warps 0-3, 4-7  softmax of tile 0 and 1: a thread per row. S from TMEM,
//                   running maximum (the output is rescaled only when it has
//                   grown by 2^8), weights back into S's columns as fp16.
//   warps 8-14      producers: warp w dequantizes group w of each step from
//                   the packed words into the swizzled key tile and value
//                   tile (V transposed; both K-major). The words' order is that of mma
//                   fragments, (8 rows) x (16 bytes) per warp store, which
//                   the swizzle spreads over all banks.
//   warp 15         issues the products. Order on the tensor pipe:
//                   S0(j), O1(j-1), S1(j), O0(j): while one tile's weights are
//                   computed, the other tile's products run.
// TMEM: S0, S1 (fp32 128 columns, the weights overwrite the first 56), O0, O1.
// Work is cut into steps. Either every CTA gets an equal run of the steps of
// all tiles, so that long caches with few rows are split and there is no
// tail (a tile cut between CTAs leaves partials, merged by k_tiles_combine),
// or a tile of its own, whichever is estimated to end first (plan_tiles).
// After SUM_STEPS steps of a tile, whoever takes the next ones, its sums are
// carried over in fp32 (finish): the tensor cores truncate.
//
// What bounds it: 2,048 tokens over 32K (8 kv heads, 4 heads each, d = 128)
// take 840 us, 1.34 PFLOP/s of the sums that are asked for. An earlier build
// took 820; without the softmax 657 us, without unpacking 762, without either
// 644 (a step's products are 1,920 cycles, the key tile's 16 extra rows among
// them). So the softmax and the producers, who share the schedulers, hold the
// tensor cores up by a fifth; sums carried over add 1 to 4% to long caches.
// With short caches a tile's fixed cost joins them: finding it and its
// queries, the first copies, the output: 7 us. Not taken: dequantizing to
// fp16 in a pass of its own (six times the cache's bytes written, and read
// for every pair of tiles); three tiles of rows or a second softmax set (do
// not fit TMEM); exact values, their zeros and scales as further rows (a
// sixth fewer tokens per step, and sums that cancel, which lost accuracy over
// 131K tokens to the truncating accumulators); both score sets for alternate
// steps of a pair with one tile of rows (134 us for 128 rows of 256 heads
// over 4K, with or without: the producers are what it waits for).
#include <algorithm>
#include <climits>
#include <cmath>

#include "ott_chunk.cuh"
#include "ott_tcgen.cuh"

namespace ott {
namespace {

constexpr int GRPS = 7;              // groups of 16 tokens per step
constexpr int STEP_TOK = 16 * GRPS;
constexpr int ROWS = 128;            // rows of a tile
constexpr int THREADS = 512;
constexpr int PROD0 = 8, MMA_WARP = 15;
constexpr int META = 4;              // steps of group metadata in flight
constexpr int HIDDEN = 1, WIDE = 2;  // its flags: some row does not see some token; scores of halved scales
constexpr unsigned long long ANY_WIDE = 0x0002020202020202ull;
constexpr int SUM_STEPS = SUM_TOKENS / STEP_TOK;   // steps whose products stay one sum in TMEM
constexpr int MIN_STEPS = 2;         // steps per CTA at least
constexpr int FIXED = 4;             // a tile's fixed cost (find it, queries, fill the pipeline, output) in steps of 2 us

template <int D>
struct TCfg {
    static constexpr int ATOMS = D / 64;                   // 128-byte columns of a K-major tile
    static constexpr int QB = ROWS * D * 2, KB = ROWS * D * 2, VB = 2 * D * 128;
    static constexpr int OFF_Q = 0, OFF_K = 2 * QB, OFF_V = OFF_K + 2 * KB;
    static constexpr int OFF_POS = OFF_V + 2 * VB;          // int pos[META][STEP_TOK]
    static constexpr int OFF_FLAG = OFF_POS + META * STEP_TOK * 4;   // a byte of flag[META][8] per group
    // per producer: 16 fp16 rows, or the key scales and zeros of a block
    static constexpr int OFF_STG = (OFF_FLAG + META * 8 + 1023) / 1024 * 1024;
    static constexpr int OFF_BAR = OFF_STG + GRPS * 32 * D;    // barriers, tmem address, abort flag
    static constexpr int SMEM = OFF_BAR + 256 + 1024;       // + alignment to 1024
    static_assert(SMEM <= 227 * 1024, "shared memory");
    __host__ __device__ static constexpr uint32_t S(int t) { return 128u * t; }
    __host__ __device__ static constexpr uint32_t O(int t) { return 256u + (uint32_t)D * t; }
};

enum { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_SFULL = 8, B_PFULL = 10, B_OFULL = 12, B_COUNT = 13 };

struct TileArgs {
    ChunkArgs a;
    int CPT;          // groups of 16 slots per block
    int nC;           // CTAs
    long long W;      // places of all tiles: FIXED and its steps each
    float *part;      // [nC][2][D + 2][256]
    int whole;        // CTA i takes tile i whole, else an equal run of steps
};

// A tile pair of a (sequence, kv head): its rows, and the groups that they see.
struct Tile {
    int e, hkv, p;            // entry, kv head, pair
    int rows;                 // valid rows
    int jlo;                  // blocks [jlo, nf) and the listed ones before
    int nlo;                  // first group of new tokens that is seen
    int cps, gs;              // groups per listed block, of all listed blocks
    int gq, gf, gn;           // groups: quantized (the listed blocks' first), fp16 (ring, pool, cold pool), new
    int sq, steps;            // steps of quantized groups, then of the others; all steps
};

__host__ __device__ inline void tile_extent(const ChunkArgs &a, int cpt, const ChunkSeq &s, int p, Tile &t) {
    const int v0 = 256 * p, vend = s.nq * a.g;
    t.p = p;
    t.rows = vend - v0 < 256 ? vend - v0 : 256;
    const int first = v0 / a.g, last = (v0 + t.rows - 1) / a.g;   // tokens of the first and last row
    t.jlo = 0;
    t.nlo = 0;
    if (a.window > 0) {
        const int lo = s.pos0 + first - a.window + 1;   // the first row's window
        t.jlo = lo <= 0 ? 0 : (lo / a.G < s.nf ? lo / a.G : s.nf);
        // new tokens before the window (none of them a first token of the sequence)
        if (s.T >= a.sinks && lo > s.T) t.nlo = (lo - s.T) / 16;
    }
    // of a listed block, only the groups that can hold first tokens (they come first)
    t.cps = a.sinks / 16 < cpt ? (a.sinks + 15) / 16 : cpt;
    t.gs = t.jlo > 0 ? s.nsink * t.cps : 0;
    t.gq = t.gs + (s.nf - t.jlo) * cpt;
    t.gf = (s.ntail + s.npool + a.C + 15) / 16;
    t.gn = s.nnew > 0 ? last / 16 + 1 - t.nlo : 0;
    t.sq = (t.gq + GRPS - 1) / GRPS;
    t.steps = t.sq + (t.gf + t.gn + GRPS - 1) / GRPS;
}

// The tile that holds place x, and the place's number in it: a tile has FIXED
// places, so that CTAs with many short tiles get fewer steps, and then its
// steps. Warp-collective.
__device__ __forceinline__ Tile tile_at(const TileArgs &ta, const ChunkTable &st, long long x, int &step) {
    const ChunkArgs &a = ta.a;
    Tile t;
    t.e = ch_entry_of(st, a.nseq, x);
    const ChunkSeq &s = st.e[t.e];
    const unsigned rel = (unsigned)(x - s.base);
    t.hkv = (int)(rel / (unsigned)s.Iu);             // Iu: places of one kv head's tiles
    int left = (int)(rel % (unsigned)s.Iu);
    const int lane = threadIdx.x & 31;
    for (int p0 = 0;; p0 += 32) {                    // ends: s.S tiles hold Iu places
        int n = 0;
        if (p0 + lane < s.S) {
            Tile u;
            tile_extent(a, ta.CPT, s, p0 + lane, u);
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
            tile_extent(a, ta.CPT, s, min(p0 + l, s.S - 1), t);
            return t;
        }
        left -= __shfl_sync(0xffffffffu, inc, 31);
    }
}

// Tile number i of the launch where every CTA takes one: an entry's last rows
// (of all its heads) first, since they see the most.
__device__ __forceinline__ Tile tile_number(const TileArgs &ta, const ChunkTable &st, int i) {
    Tile t;
    int lo = 0, hi = ta.a.nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (st.e[mid].ubase <= i) lo = mid;
        else hi = mid;
    }
    const ChunkSeq &s = st.e[lo];
    t.e = lo;
    t.hkv = (i - s.ubase) % ta.a.Hkv;
    tile_extent(ta.a, ta.CPT, s, s.S - 1 - (i - s.ubase) / ta.a.Hkv, t);
    return t;
}

// The softmax warps and the product warp, each from its own place in the
// code: the tile's queries are in place, the last tile's output is read.
__device__ __forceinline__ void tile_sync() { asm volatile("barrier.sync 1, %0;" ::"n"(32 * (PROD0 + 1)) : "memory"); }

// ---------------------------------------------------------------- producers
// Orders within the tiles. Scores do not depend on the order of the channels
// as long as queries and keys share it, outputs not on that of a group's
// tokens, and the order of the output's channels is undone where it is read.
// So they are chosen for wide stores that meet no bank twice:
//   channels of a key row: the 8 fp16x2 that a lane unpacks from a word are
//     adjacent, 4 per 16-byte chunk (chan_at);
//   tokens of a group: 2i, 2i + 1, 2i + 8, 2i + 9 are adjacent (slot_of), in
//     the key rows (hence in the scores and weights) and in the value rows;
//   value rows (channels): the low three bits of the channel rotated (vrow),
//     so that 16 lanes of an 8-byte store meet all 8 chunks.
// Byte offset, before the swizzle, of channels c, c + 1 (c = 16 kt + 2 i + 8 o)
// in a key row, as (128-byte column, 16-byte chunk, word of it).
template <int D>
__device__ __forceinline__ uint32_t chan_at(int kt, int o, int i, int row) {
    const int q = o * (D / 16) + kt, p = q & 7;
    return (uint32_t)((q >> 3) * (ROWS * 128) + row * 128 + (((2 * i + (p >> 2)) ^ (row & 7)) << 4) + (p & 3) * 4);
}

// One 16-byte piece of an fp16 row (8 channels from 8 * ch on) into a tile of key rows.
template <int D>
__device__ __forceinline__ void put_row_piece(uint8_t *tile, int row, int ch, uint4 v) {
    const int kt = ch >> 1, o = ch & 1;
    *reinterpret_cast<uint32_t *>(tile + chan_at<D>(kt, o, 0, row)) = v.x;
    *reinterpret_cast<uint32_t *>(tile + chan_at<D>(kt, o, 1, row)) = v.y;
    *reinterpret_cast<uint32_t *>(tile + chan_at<D>(kt, o, 2, row)) = v.z;
    *reinterpret_cast<uint32_t *>(tile + chan_at<D>(kt, o, 3, row)) = v.w;
}

// Group x of the tile's quantized ones.
struct Group {
    const uint8_t *src;    // the block
    int j;                 // its number, -1: none
    int sub;               // group of the block
    int left;              // valid tokens of the block from the group's first on (<= 0: none)
    int per;               // groups of the block
};
__device__ __forceinline__ Group group_at(const ChunkArgs &a, const ChunkSeq &s, const Tile &t, int cpt, int u, int x) {
    Group g;
    if (x >= t.gq) {
        g.src = nullptr;
        g.j = -1;
        g.sub = g.left = 0;
        g.per = cpt;
        return g;
    }
    const bool listed = x < t.gs;
    const int per = listed ? t.cps : cpt, y = listed ? x : x - t.gs, jp = y / per;
    g.sub = y % per;
    g.per = per;
    g.left = 0;
    g.src = nullptr;
    g.j = t.jlo + jp;
    if (listed) {
        g.j = a.sel[(size_t)u * a.NB + jp];
        if (g.j >= t.jlo) g.j = -1;   // in the window's own range
    }
    if (g.j >= 0) {
        const int cnt = chunk_block_cnt(a, u, g.j);
        g.left = (listed ? min(cnt, a.sinks) : cnt) - 16 * g.sub;
        const size_t own = (size_t)u * a.NB + g.j;
        g.src = a.blk + (a.bt ? (size_t)a.bt[own] : own) * a.blk_bytes;
    }
    return g;
}

// A tile's quantized groups are made first, then the fp16 ones, each kind
// dealt to the 7 warps in runs: a warp walks through its blocks and meets a
// block's key scales once, and all warps are busy with the same kind (a step
// takes as long as its slowest group). In each of the two loops, round k
// makes a group while the next one's words are on their way; round -1 only
// starts the first loads (one copy of the code).
template <int D>
struct Producer {
    using C = TCfg<D>;
    static constexpr int NKT = D / 16, NW = D / 32;
    static constexpr int CPR = D / 8, RPI = 32 / CPR;   // 16-byte pieces of an fp16 row, rows per load of a warp
    const TileArgs &ta;
    const ChunkArgs &a;
    const ChunkSeq &s;
    const Tile &t;
    uint8_t *const sm;
    uint64_t *const bar;
    volatile int *const gave_up;
    const int w, lane, r, i, b, u;
    int pmin, lomax;       // smallest position, largest window start of the rows
    uint32_t it;

    __device__ Producer(const TileArgs &ta_, const ChunkSeq &s_, const Tile &t_, uint8_t *sm_, uint64_t *bar_,
                        volatile int *gave_up_, uint32_t it_)
        : ta(ta_), a(ta_.a), s(s_), t(t_), sm(sm_), bar(bar_), gave_up(gave_up_), w((threadIdx.x >> 5) - PROD0),
          lane(threadIdx.x & 31), r(lane >> 2), i(lane & 3), b(a.B0 + t.e), u(b * a.Hkv + t.hkv), it(it_) {
        pmin = s.pos0 + 256 * t.p / a.g;
        lomax = a.window > 0 ? s.pos0 + (256 * t.p + t.rows - 1) / a.g - a.window + 1 : 0;
    }
    __device__ void wait(int which) { bar_wait(&bar[which + (it & 1)], ((it >> 1) & 1u) ^ 1u, gave_up); }
    // The tile's part is written: pos (of lane < 16's token, INT_MAX: none)
    // decides whether some row does not see it, where `ask`; wide: its scores
    // count twice.
    __device__ void key_done(bool ask, int pos, bool wide) {
        bool hidden = false;
        if (ask) {
            hidden = __any_sync(0xffffffffu, lane < 16 && !(pos <= pmin && (pos >= lomax || pos < a.sinks)));
            if (lane < 16)
                reinterpret_cast<volatile int *>(sm + C::OFF_POS)[(it % META) * STEP_TOK + 16 * w + slot_of(lane)] = pos;
        }
        if (lane == 0) *reinterpret_cast<volatile uint8_t *>(sm + C::OFF_FLAG + (it % META) * 8 + w) = (hidden ? HIDDEN : 0) | (wide ? WIDE : 0);
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

    // Quantized groups x, x + 1 .. x + n - 1 (none from gq on).
    __device__ void quantized(int x, int n) {
        const int cpt = ta.CPT;
        uint32_t kr[NW], vr[NW], zr[2 * NKT], ks2[NKT][2];
        uint8_t *const stage = sm + C::OFF_STG + w * (32 * D);   // the block's key scales and zeros
        // (the next block's wait in registers: a copy into shared memory in
        // flight holds up every fence of the proxies behind it)
        const int row0 = slot_of(r), row1 = slot_of(r + 8);
        const uint32_t k0 = (16 * w + row0) * 128 + ((2 * i ^ (row0 & 7)) << 4), k1 = (16 * w + row1) * 128 + ((2 * i ^ (row1 & 7)) << 4);
        Group g, gn, gb;             // made, next, first of the next block
        uint4 hb = make_uint4(0, 0, 0, 0);   // gb's
        int xb = -1;                 // gb's number
        g.left = g.sub = g.per = 0;
        g.j = -1;
        g.src = nullptr;
        gn = gb = g;
        const Magic mg;
        int fresh = 0;               // steps for which the block's offset rows still have to be written
#pragma unroll 1
        for (int k = -1; k < n; ++k) {
            bool enter = false;
            if (g.left > 16 && g.sub + 1 < g.per) {
                gn.sub += 1;
                gn.left -= 16;
            } else if (k + 1 < n) {
                const int xn = x + k + 1;
                if (xn == xb) {
                    gn = gb;
                } else {   // the run's first group, or one behind a short block's tokens
                    gn = group_at(a, s, t, cpt, u, xn);
                    if (gn.left > 0 && lane < D / 4) hb = reinterpret_cast<const uint4 *>(gn.src)[lane];
                }
                enter = gn.left > 0;
            }
            if (k >= 0) {
                wait(B_KEMPTY);
                uint8_t *kb = key_tile();
                if (g.left > 0) {
                    uint32_t k8[NW];
#pragma unroll
                    for (int y = 0; y < NW; ++y) k8[y] = kr[y] >> 8;
                    uint8_t *const p[4] = {kb + k0, kb + (k0 ^ 16), kb + k1, kb + (k1 ^ 16)};
#pragma unroll
                    for (int th = 0; th < 2; ++th)
#pragma unroll
                        for (int q0 = 0; q0 < 2 * NKT; q0 += 4) {   // 4 fp16x2 of a word: a chunk
                            const int wi = 2 * (q0 >> 3) + th;
                            uint32_t f[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                f[y] = ch_key(mg, kr[wi], k8[wi], (q0 + y) & 7, ks2[(q0 + y) % NKT][(q0 + y) / NKT]);
                            // chunk 2i + 1 is chunk 2i with its lowest bit turned, whatever the swizzle
                            *reinterpret_cast<uint4 *>(p[2 * th + ((q0 >> 2) & 1)] + (q0 >> 3) * (ROWS * 128)) =
                                make_uint4(f[0], f[1], f[2], f[3]);
                        }
                    if (fresh > 0) {
                        // rows 112 + 2w, 113 + 2w: z and s; lane (r, i) copies the channels of k-tile r
                        --fresh;
                        if (r < NKT) {
#pragma unroll
                            for (int o = 0; o < 2; ++o) {
                                const uint2 z = *reinterpret_cast<const uint2 *>(stage + 4 * (16 * r + 2 * i + 8 * o));
                                *reinterpret_cast<uint32_t *>(kb + chan_at<D>(r, o, i, STEP_TOK + 2 * w)) = __byte_perm(z.x, z.y, 0x7632);
                                *reinterpret_cast<uint32_t *>(kb + chan_at<D>(r, o, i, STEP_TOK + 2 * w + 1)) = __byte_perm(z.x, z.y, 0x5410);
                            }
                        }
                    }
                } else {
                    zero_keys(kb);
                    fresh = 2;
                }
                const bool wide = *reinterpret_cast<volatile int *>(stage + 4 * D) != 0;   // (in a register, it would be spilled)
                const bool ask = g.left < 16 || a.window > 0 || wide;
                int pos = INT_MAX;
                if (ask && lane < 16 && lane < g.left)
                    pos = a.window > 0 ? a.bidx[((size_t)u * a.NB + g.j) * a.G + 16 * g.sub + lane] : 0;
                key_done(ask, pos, wide);
            }
            if (enter) {   // the block's scales, through shared memory; then the next block's are fetched
                __syncwarp();
                if (lane < D / 4) *reinterpret_cast<uint4 *>(stage + 16 * lane) = hb;
                const bool wide = __any_sync(0xffffffffu, lane < D / 4 && ch_wide(__vmaxu2(__vmaxu2(hb.x, hb.y), __vmaxu2(hb.z, hb.w))));
                *reinterpret_cast<volatile int *>(stage + 4 * D) = wide;   // the same by every lane
                const __half2 part = __float2half2_rn(wide ? 0.5f : 1.0f);
                __syncwarp();
#pragma unroll
                for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        const uint2 z = *reinterpret_cast<const uint2 *>(stage + 4 * (16 * kt + 2 * i + 8 * o));
                        ks2[kt][o] = ch_h2(__hmul2(ch_as_h2(__byte_perm(z.x, z.y, 0x5410)), part));
                    }
                fresh = 2;   // both slots
                xb = x + k + 1 - gn.sub + gn.per;
                if (xb < x + n) {
                    gb = group_at(a, s, t, cpt, u, xb);
                    if (gb.left > 0 && lane < D / 4) hb = reinterpret_cast<const uint4 *>(gb.src)[lane];
                }
            }
            const bool load = k + 1 < n && gn.left > 0;
            const uint8_t *tb = gn.src + ksz_bytes(D) + (size_t)gn.sub * tile_bytes(D);
            if (load) words(tb, kr);   // in flight under the value tile
            if (k >= 0) {
                wait(B_VEMPTY);
                uint8_t *vb = value_at();
                if (g.left > 0) {
                    uint32_t v8[NW];
#pragma unroll
                    for (int y = 0; y < NW; ++y) v8[y] = vr[y] >> 8;
#pragma unroll
                    for (int gm = 0; gm < NKT / 2; ++gm) {
                        const uint32_t *z = zr + 4 * gm;
                        const uint32_t s2[2] = {__byte_perm(z[0], z[1], 0x5410), __byte_perm(z[2], z[3], 0x5410)};
                        const uint32_t z2[2] = {__byte_perm(z[0], z[1], 0x7632), __byte_perm(z[2], z[3], 0x7632)};
#pragma unroll
                        for (int mm = 0; mm < 2; ++mm)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int mt = 2 * gm + mm, q = half * NKT + mt, wi = 2 * (q >> 3);
                                *reinterpret_cast<uint2 *>(vb + (16 * mt + 8 * half) * 128) =
                                    make_uint2(ch_val(mg, vr[wi], v8[wi], q & 7, s2[0], z2[0]),
                                               ch_val(mg, vr[wi + 1], v8[wi + 1], q & 7, s2[1], z2[1]));
                            }
                    }
                } else {
                    zero_values(vb);
                }
                value_done();
            }
            if (load) {
                words(tb + tile_v_off(D), vr);
#pragma unroll
                for (int gm = 0; gm < NKT / 2; ++gm) {
                    const uint4 z = reinterpret_cast<const uint4 *>(tb + tile_sz_off(D))[gm * 4 + i];
                    zr[4 * gm] = z.x; zr[4 * gm + 1] = z.y; zr[4 * gm + 2] = z.z; zr[4 * gm + 3] = z.w;
                }
            }
            g = gn;
        }
    }

    // n groups from the x-th of the fp16 ones on: ring, pool and cold pool in
    // whole groups, then the new tokens from group nlo on; past them, nothing.
    // A lane finds one row, the keys' or the values' (lane mod 16), and passes
    // its address round; keys come through registers, values through shared
    // memory, both under one wait. (Loads a group ahead would take registers
    // that the other loop, which has most of the work, would spill.)
    __device__ void plain(int x, int n) {
        const int ncold = a.C > 0 ? a.cmeta[2 * u] : 0, chead = a.C > 0 ? a.cmeta[2 * u + 1] : 0;
        const int nhot = s.ntail + s.npool + ncold;
        uint8_t *const stage = sm + C::OFF_STG + w * (32 * D);   // 16 rows, 16-byte chunks turned by the row
#pragma unroll 1
        for (int y = x; y < x + n; ++y) {
            int f = 0, left = 0;   // first token, tokens left
            if (y < t.gf) {
                f = 16 * y;
                left = nhot - f;
            } else if (y < t.gf + t.gn) {
                f = nhot + 16 * (y - t.gf + t.nlo);
                left = nhot + s.nnew - f;
            }
            unsigned long long at = 0;
            if ((lane & 15) < left)
                at = reinterpret_cast<unsigned long long>(
                    chunk_fp16_row(a, s, b, t.hkv, u, f + (lane & 15), ncold, chead, lane >= 16, D));
            uint4 kr[16 / RPI];
#pragma unroll
            for (int e = 0; e < 16 / RPI; ++e) {
                const unsigned long long p = __shfl_sync(0xffffffffu, at, RPI * e + lane / CPR);
                kr[e] = make_uint4(0, 0, 0, 0);
                if (p) kr[e] = reinterpret_cast<const uint4 *>(p)[lane % CPR];
            }
#pragma unroll
            for (int e = 0; e < 16 / RPI; ++e) {
                const int row = RPI * e + lane / CPR, ch = lane % CPR;
                const unsigned long long p = __shfl_sync(0xffffffffu, at, 16 + row);
                // no row: zeros (nothing is read)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ch_smem(stage + row * (2 * D) + ((ch ^ (row & 7)) << 4))),
                             "l"(p ? reinterpret_cast<const uint8_t *>(p) + 16 * ch : reinterpret_cast<const uint8_t *>(a.q)),
                             "r"(p ? 16 : 0)
                             : "memory");
            }
            const int pos = lane < 16 && lane < left ? chunk_fp16_pos(a, s, u, f + lane, ncold, chead) : INT_MAX;
            wait(B_KEMPTY);
            uint8_t *kb = key_tile();
#pragma unroll
            for (int e = 0; e < 16 / RPI; ++e)
                put_row_piece<D>(kb, 16 * w + slot_of(RPI * e + lane / CPR), lane % CPR, kr[e]);
            if (lane < 2 * CPR)
                *reinterpret_cast<uint4 *>(kb + (lane % CPR / 8) * (ROWS * 128) + (STEP_TOK + 2 * w + lane / CPR) * 128 +
                                           (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            key_done(true, pos, false);
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

    __device__ static void words(const uint8_t *p, uint32_t (&d)[NW]) {
        const int lane = threadIdx.x & 31;
        if constexpr (NW == 4) {
            const uint4 x = reinterpret_cast<const uint4 *>(p)[lane];
            d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
        } else {
            const uint2 x = reinterpret_cast<const uint2 *>(p)[lane];
            d[0] = x.x; d[1] = x.y;
        }
    }
    __device__ void zero_keys(uint8_t *kb) const {
#pragma unroll 1
        for (int e = lane; e < 18 * CPR; e += 32) {
            const int row = e / CPR < 16 ? 16 * w + e / CPR : STEP_TOK + 2 * w + e / CPR - 16, ch = e % CPR;
            *reinterpret_cast<uint4 *>(kb + (ch / 8) * (ROWS * 128) + row * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
    }
    __device__ static void zero_values(uint8_t *vb) {
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint2 *>(vb + 8 * c * 128) = make_uint2(0u, 0u);
    }
};

template <int D>
__device__ void produce(const TileArgs &ta, const ChunkSeq &s, const Tile &t, uint8_t *sm, uint64_t *bar,
                        volatile int *gave_up, int j0, int j1, uint32_t it) {
    Producer<D> p(ta, s, t, sm, bar, gave_up, it);
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
            mma_ss(tmem + C::S(t), dq + t * (C::QB / 16) + off, dk + slot * (C::KB / 16) + off, HI, instr_desc(128), k > 0);
        }
    };
    // groups whose keys are halves: their 16 columns once more
    auto scores_again = [&](int t, int slot, uint32_t it) {
        unsigned long long flags = *reinterpret_cast<const volatile unsigned long long *>(sm + C::OFF_FLAG + (it % META) * 8);
        if (!(flags & ANY_WIDE)) return;
#pragma unroll 1
        for (int w = 0; w < GRPS; ++w, flags >>= 8)
            if (flags & WIDE) {
#pragma unroll 1
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k / 4) * (ROWS * 128) + (k & 3) * 32) / 16;
                    mma_ss(tmem + C::S(t) + 16 * w, dq + t * (C::QB / 16) + off, dk + slot * (C::KB / 16) + off + w * (16 * 128 / 16),
                           desc_hi(1024, 2), instr_desc(16), true);
                }
            }
    };
    auto values = [&](int t, int slot, bool acc) {
#pragma unroll
        for (int k = 0; k < GRPS; ++k) {
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
            scores_again(0, slot, it);
            tc_commit(&bar[B_SFULL]);
        }
        __syncwarp();
        if (nt == 2) {
            if (j > 0) bar_wait(&bar[B_PFULL + 1], (c1 - 1) & 1u, gave_up);
            tc_after();
            if (elect_one()) {
                if (j > 0) {
                    values(1, prev, j > 1);
                    tc_commit(&bar[B_VEMPTY + prev]);
                }
                scores(1, slot);
                scores_again(1, slot, it);
                tc_commit(&bar[B_SFULL + 1]);
                tc_commit(&bar[B_KEMPTY + slot]);
            }
            ++c1;
        } else {
            if (elect_one()) tc_commit(&bar[B_KEMPTY + slot]);
        }
        __syncwarp();
        bar_wait(&bar[B_VFULL + slot], par, gave_up);
        bar_wait(&bar[B_PFULL], c0 & 1u, gave_up);
        ++c0;
        tc_after();
        if (elect_one()) {
            values(0, slot, j > 0);
            if (nt == 1) tc_commit(&bar[B_VEMPTY + slot]);
        }
        __syncwarp();
    }
    const int last = (it - 1) & 1;
    if (nt == 2) bar_wait(&bar[B_PFULL + 1], (c1 - 1) & 1u, gave_up);
    tc_after();
    if (elect_one()) {
        if (nt == 2) {
            values(1, last, steps > 1);
            tc_commit(&bar[B_VEMPTY + last]);
        }
        tc_commit(&bar[B_OFULL]);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- softmax
template <int D>
__device__ void softmax(const TileArgs &ta, const ChunkSeq &s, const Tile &t, uint8_t *sm, uint64_t *bar,
                        volatile int *gave_up, uint32_t tmem, int tile, int steps, uint32_t it, uint32_t cnt, float &m_ref,
                        float &l) {
    using C = TCfg<D>;
    const ChunkArgs &a = ta.a;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(32 * wq) << 16;
    const uint32_t ts = tmem + C::S(tile) + lanes, to = tmem + C::O(tile) + lanes;
    const int row = ROWS * tile + 32 * wq + lane;
    const int pos = s.pos0 + (256 * t.p + min(row, t.rows - 1)) / a.g, lo = a.window > 0 ? pos - a.window + 1 : 0;
    m_ref = -CUDART_INF_F;
    l = 0.0f;
    for (int j = 0; j < steps; ++j, ++it, ++cnt) {
        bar_wait(&bar[B_SFULL + tile], cnt & 1u, gave_up);
        tc_after();
        // groups with a token that some row does not see: -inf into its scores
        const int ms = it % META;
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
                        if (!chunk_sees(tp[16 * k + c], pos, lo, a.sinks)) f[c] = -CUDART_INF_F;
                    tm_st16(ts + 16 * k, f);
                }
            wait_st();
        }
        // The maximum: groups 4..6 first, then 0..3, which stay in registers
        // (64 of them; 4..6 are read again below, behind the weights of 0..3,
        // whose columns they do not share).
        float e[16], x[64];
        tm_ld16(ts + STEP_TOK, e);
#pragma unroll
        for (int k = 4; k < GRPS; ++k) tm_ld16(ts + 16 * k, x + 16 * (k - 4));
        wait_ld();
        tie16(e);
#pragma unroll
        for (int k = 0; k < 3; ++k) tie16(x + 16 * k);
        float mx = -CUDART_INF_F, off[GRPS];
#pragma unroll
        for (int k = 0; k < GRPS; ++k) off[k] = (e[2 * k] + e[2 * k + 1]) * a.sl2;
#pragma unroll
        for (int k = 4; k < GRPS; ++k) mx = fmaxf(mx, fmaf(max16(x + 16 * (k - 4)), a.sl2, off[k]));
#pragma unroll
        for (int k = 0; k < 4; ++k) tm_ld16(ts + 16 * k, x + 16 * k);
        wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) tie16(x + 16 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaf(max16(x + 16 * k), a.sl2, off[k]));
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
        float2 sum = make_float2(0.0f, 0.0f);
        auto weights = [&](int k, const float *y) {
            const float2 ad = make_float2(off[k] - mm, off[k] - mm), sc = make_float2(a.sl2, a.sl2);
            uint32_t p8[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float2 v = __ffma2_rn(make_float2(y[2 * c], y[2 * c + 1]), sc, ad);
                const float2 p = make_float2(ch_ex2(v.x), ch_ex2(v.y));
                sum = __fadd2_rn(sum, p);
                p8[c] = ch_h2(__floats2half2_rn(p.x, p.y));
            }
            tm_st8(ts + 8 * k, p8);
        };
        weights(0, x);
        weights(1, x + 16);
        weights(2, x + 32);
        tm_ld16(ts + 64, x);
        tm_ld16(ts + 80, x + 16);
        tm_ld16(ts + 96, x + 32);
        weights(3, x + 48);
        wait_ld();
        tie16(x);
        tie16(x + 16);
        tie16(x + 32);
        weights(4, x);
        weights(5, x + 16);
        weights(6, x + 32);
        l += sum.x + sum.y;
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
    const ChunkArgs &a = ta.a;
    const int wq = (threadIdx.x >> 5) & 3, row = ROWS * tile + 32 * wq + (threadIdx.x & 31), v = 256 * t.p + row;
    const uint32_t to = tmem + C::O(tile) + ((uint32_t)(32 * wq) << 16);
    float *pb = ta.part + ((size_t)blockIdx.x * 2 + slot) * (D + 2) * 256 + row;
    if (more) {
        const float mo = pb[0], M = fmaxf(mo, m), mr = M == -CUDART_INF_F ? 0.0f : M;
        const float sn = ch_ex2(m - mr), so = ch_ex2(mo - mr);
        l = fmaf(l, sn, pb[256] * so);
        const size_t at = (((size_t)(a.B0 + t.e) * a.Hq + t.hkv * a.g + v % a.g) * a.n + v / a.g) * D;
        const float inv = whole && row < t.rows ? chunk_norm(l, a.k == nullptr, a.q + at, D) : 0.0f;
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
        const float inv = row < t.rows ? chunk_norm(l, a.k == nullptr, a.q + at, D) : 0.0f;
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
template <int D, int ROLE>
__device__ void role_loop(const TileArgs &ta, const ChunkTable &st, uint8_t *sm, uint64_t *bar, volatile int *gave_up,
                          uint32_t tmem) {
    using C = TCfg<D>;
    const ChunkArgs &a = ta.a;
    // (places from the run's start on: fewer registers than the places)
    int done = 0;
    const long long x0 = ta.whole ? 0 : ch_range_start(ta.W, ta.nC, blockIdx.x);
    const int todo = ta.whole ? 1 : (int)(ch_range_start(ta.W, ta.nC, blockIdx.x + 1) - x0);
    uint32_t it = 0, ct[2] = {0, 0};   // steps done by the CTA, and by each tile
    for (uint32_t run = 0; done < todo;) {
        int at = 0;
        const Tile t = ta.whole ? tile_number(ta, st, blockIdx.x) : tile_at(ta, st, x0 + done, at);
        const ChunkSeq &s = st.e[t.e];
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
                    put_row_piece<D>(sm + C::OFF_Q + row / ROWS * C::QB, row % ROWS, ch, v[y]);
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
            produce<D>(ta, s, t, sm, bar, gave_up, j0, j1, it);
        }
        it += (uint32_t)n;
        ct[0] += (uint32_t)n;
        if (nt == 2) ct[1] += (uint32_t)n;
        ++run;
    }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    k_chunk_tiles(const __grid_constant__ TileArgs ta, const __grid_constant__ ChunkTable st) {
    using C = TCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (ch_smem(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    uint32_t *tm = reinterpret_cast<uint32_t *>(sm + C::OFF_BAR + 128);
    volatile int *gave_up = reinterpret_cast<volatile int *>(sm + C::OFF_BAR + 132);
    const ChunkArgs &a = ta.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int k = 0; k < 2; ++k) {
            bar_init(&bar[B_KFULL + k], GRPS);
            bar_init(&bar[B_VFULL + k], GRPS);
            bar_init(&bar[B_KEMPTY + k], 1);
            bar_init(&bar[B_VEMPTY + k], 1);
            bar_init(&bar[B_SFULL + k], 1);
            bar_init(&bar[B_PFULL + k], ROWS / 32);
        }
        bar_init(&bar[B_OFULL], 1);
        *gave_up = 0;
        for (int k = 0; k < META; ++k) *reinterpret_cast<unsigned long long *>(sm + C::OFF_FLAG + 8 * k) = 0;   // byte 7 stays
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // key rows that no group fills
    for (int x = threadIdx.x; x < 2 * C::ATOMS * 2 * 32; x += THREADS) {
        const int slot = x / (C::ATOMS * 64), at = x / 64 % C::ATOMS, rw = 126 + x / 32 % 2;
        *reinterpret_cast<uint32_t *>(sm + C::OFF_K + slot * C::KB + at * (ROWS * 128) + rw * 128 + (x % 32) * 4) = 0;
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
        role_loop<D, SOFTMAX>(ta, st, sm, bar, gave_up, tmem);
    } else {
        if (warp == MMA_WARP)
            role_loop<D, MULTIPLY>(ta, st, sm, bar, gave_up, tmem);
        else
            role_loop<D, PRODUCE>(ta, st, sm, bar, gave_up, tmem);
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
__global__ void __launch_bounds__(256) k_tiles_combine(const __grid_constant__ TileArgs ta, const __grid_constant__ ChunkTable st) {
    const ChunkArgs &a = ta.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the tile: x = (pair of the largest sequence, 32 rows), y = kv head, z = entry
    const ChunkSeq &s = st.e[blockIdx.z];
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
            tile_extent(a, ta.CPT, s, q, t);
            before += t.steps + FIXED;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        ts += before;
    }
    tile_extent(a, ta.CPT, s, p, t);
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
    const float inv = chunk_norm(L, a.k == nullptr, a.q + at, D);
    __half *o = a.out + at + CH * warp;
#pragma unroll
    for (int y = 0; y < CH; y += 8)
        *reinterpret_cast<uint4 *>(o + y) = make_uint4(
            ch_h2(__floats2half2_rn(acc[y] * inv, acc[y + 1] * inv)), ch_h2(__floats2half2_rn(acc[y + 2] * inv, acc[y + 3] * inv)),
            ch_h2(__floats2half2_rn(acc[y + 4] * inv, acc[y + 5] * inv)), ch_h2(__floats2half2_rn(acc[y + 6] * inv, acc[y + 7] * inv)));
}

template <int D>
cudaError_t launch_t(const TileArgs &ta, const ChunkTable &st, int rows, cudaStream_t s) {
    cudaError_t e = launch_pdl(k_chunk_tiles<D>, dim3((unsigned)ta.nC), THREADS, (size_t)TCfg<D>::SMEM, s, ta, st);
    if (e != cudaSuccess || ta.nC == 1 || ta.whole) return e;
    return launch_pdl(k_tiles_combine<D>, dim3((unsigned)((rows + 31LL) / 32), (unsigned)ta.a.Hkv, (unsigned)ta.a.nseq), 256, 0, s, ta, st);
}

}  // namespace

cudaError_t set_tiles_attributes(int d) {
    return d == 128 ? cudaFuncSetAttribute(k_chunk_tiles<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<128>::SMEM)
                    : cudaFuncSetAttribute(k_chunk_tiles<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<64>::SMEM);
}

// The launch's table in tiles: S pairs of tiles per kv head, Iu their steps.
// false: the sizes do not fit the kernel's 32-bit counters.
bool plan_tiles(const ott_cache *c, ChunkArgs &a, ChunkTable &st, int &nC, bool &whole, size_t &part_floats) {
    if (a.Hkv > 65535) return false;   // a grid dimension of the merge
    const int cpt = ntiles_of(c->G);
    long long base = 0, tiles = 0;
    int longest = 0;
    for (int x = 0; x < a.nseq; ++x) {
        ChunkSeq &s = st.e[x];
        s.base = base;
        s.ubase = (int)tiles;
        s.S = (int)(((long long)s.nq * a.g + 255) / 256);
        long long steps = 0;
        if (((long long)s.nf + s.nsink) * cpt + ((long long)s.ntail + s.npool + a.C + s.nq) / 16 + 4 > INT_MAX) return false;
        for (int p = 0; p < s.S; ++p) {
            Tile t;
            tile_extent(a, cpt, s, p, t);
            steps += t.steps + FIXED;
            longest = std::max(longest, t.steps);
            if (steps * a.Hkv > INT_MAX) return false;
        }
        s.Iu = (int)steps;
        base += steps * a.Hkv;
        tiles += (long long)s.S * a.Hkv;
        if (tiles > INT_MAX) return false;
    }
    st.e[a.nseq] = ChunkSeq{};
    st.e[a.nseq].base = a.W = base;
    st.e[a.nseq].ubase = (int)tiles;
    const double sms = c->sm_count, W = (double)base, nT = (double)tiles;
    // Equal runs of places, or a tile per CTA: by their estimated times. Cut
    // tiles and their merge cost 8 steps and 0.1 per part of a tile. 333 new
    // tokens of five short sequences (100 tiles): 41 us in runs, 17 with a
    // tile per CTA; 1,024 tokens (128 tiles) over 2,048: 70 and 66, over
    // 4,096: 91.3 and 90.4, over 7,168: 123 and 127. (Fitted to shapes of 8 kv
    // heads; elsewhere an estimate.)
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

cudaError_t launch_tiles(const ott_cache *c, const ChunkArgs &a, const ChunkTable &st, int nC, bool whole, cudaStream_t s) {
    TileArgs ta;
    ta.a = a;
    ta.CPT = ntiles_of(c->G);
    ta.nC = nC;
    ta.W = a.W;
    ta.part = a.part;
    ta.whole = whole;
    int rows = 0;
    for (int x = 0; x < a.nseq; ++x) rows = std::max(rows, st.e[x].nq * a.g);   // at most Hq * n
    return c->d == 128 ? launch_t<128>(ta, st, rows, s) : launch_t<64>(ta, st, rows, s);
}

}  // namespace ott
