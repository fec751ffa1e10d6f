// ott_chunk.cu -- attention of several query rows per kv head over the OTT
// stores: a chunk of new tokens (ott_chunk_attn) or one query with a window
// (ott_decode_attn_window). The plan of every such call, and the kernel for 5
// to 16 rows (up to four go to the decode kernel, ott_decode.cu, more than 16
// to ott_chunk_tiles.cu).
//
// Mathematics. A block's key channel is z + s * code. With code - 1 in
// {-1, 0, 1, 2}, s * (code - 1) is an exact fp16 number, and
//     q . k = sum_c q_c s_c (code_c - 1) + sum_c q_c (z_c + s_c),
// where the second sum is one number per (query row, block): the tensor
// cores get exact operands (q is fp16 as given), and the second sum is taken
// with z + s split into two fp16 numbers. So the logits keep fp32 accuracy;
// a key rounded to fp16 instead would move a channel of magnitude 40 by up
// to 2^-6 the same way for every token of the block that has that code. The
// softmax weights (relative 2^-11) and the values z + s * code are rounded to
// fp16: their errors differ from token to token and average out in the sum.
//
// Layout of the work. A unit is (sequence, kv head, slice of 8 or 16 query
// rows); row v = token * g + head, so that the g query heads that share a kv
// head share its blocks, too. Work items are what one copy brings: 8 fp16
// tokens (keys and values, 4 KB at d = 128) or a chunk of up to 64 slots of a
// block (5.1 KB, with the block's key scales where the warp has not met them).
// A grid of one CTA per SM (a multiple of that for very long runs) gives every
// warp an equal contiguous run of items; the copies run ahead of the products
// through a ring of stages that does not stop at the borders of units. A warp
// leaves one partial (max, sum, unnormalised output) per unit that it touches;
// k_chunk_combine merges them.
//
// What bounds it: the instructions that unpack codes into operands, of which
// 8 or 16 columns of products do not make enough use; the copies run ahead
// and HBM waits. Batch 32 x 4K, 32 heads of d = 128 (405 MB of cache): 188 us
// with 8 rows (NC = 1, 128 registers and 80 bytes spilled), 2.2 TB/s; 256 with
// 16 (NC = 2, 236 registers).
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "ott_chunk.cuh"

namespace ott {
namespace {

constexpr int FI = 8;                       // fp16 tokens per work item
constexpr int CT = CHUNK_TILES * TILE;      // block slots per work item
// Query rows per kv head up to which the decode kernel (its rows mode) and
// then this file's kernel serve a call; the tcgen05 tiles take the rest. Batch
// 32 x 4K, 32 heads: 4 rows 129 us in rows mode, 184 here (rows mode has one
// slice of up to 4 rows and would read the cache twice for 5); 16 rows 256 us
// here; 17 rows 441 us in tiles (64 rows 443), about 511 here in two slices.
constexpr int DEC_ROWS_MAX = 4, ROWS_MAX = 16;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(ch_smem(p)));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(ch_smem(p)));
}
__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(ch_smem(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(ch_smem(dst)),
        "l"(src), "r"(bytes), "r"(ch_smem(bar))
        : "memory");
}
// Bounded wait: gives up after a fixed number of polls instead of hanging.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity) {
    for (int it = 0; it < (1 << 22); ++it) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(ch_smem(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}
template <int NW>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[NW]) {
    if constexpr (NW == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x; w[1] = x.y;
    }
}

// NC groups of 8 query rows (the columns of an MMA). One group fits 16 warps
// of 128 registers; two need twice the accumulators, so 8 warps, each with
// twice the stages.
template <int D, int NC>
struct RowsCfg {
    static constexpr int NKT = D / 16, NW = D / 32;
    static constexpr int RB = 8 * NC;
    static constexpr int WARPS = NC == 1 ? 16 : 8, NST = NC == 1 ? 2 : 4;
    static constexpr int STAGE = stage_bytes(D);
    static constexpr int RS = D + 8;   // padded fp16 row (halves): conflict-free ldmatrix
    static constexpr int WARP_SMEM = NST * STAGE + 128;   // stages, barriers, what each stage holds
    static_assert(2 * FI * RS * 2 <= STAGE && STAGE % 128 == 0, "fp16 items fit a stage");
};

// A work item: its unit (entry, kv head, slice of rows), its number in the
// unit, and for one of a block the block's place and the chunk; all kept up
// by additions (a division per item costs as much as a tile of tokens).
struct Cursor {
    long long x;
    int e, hkv, sl, off, jp, k;
    int Sf, Iu;   // of the entry
    __device__ __forceinline__ void unit(const ChunkTable &st) {
        off = jp = k = 0;
        Sf = st.e[e].Sf;
        Iu = st.e[e].Iu;
    }
    // true: the next item is another unit's
    __device__ __forceinline__ bool next(const ChunkArgs &a, const ChunkTable &st) {
        ++x;
        if (off++ >= Sf && ++k == a.CPB) {
            k = 0;
            ++jp;
        }
        if (off < Iu) return false;
        if (++sl == st.e[e].S) {
            sl = 0;
            if (++hkv == a.Hkv) {
                hkv = 0;
                do ++e;
                while (e < a.nseq && st.e[e].S == 0);
            }
        }
        unit(st);
        return true;
    }
};

template <int D, int NC>
__global__ void __launch_bounds__(RowsCfg<D, NC>::WARPS * 32, 1)
    k_chunk_rows(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkTable st) {
    using C = RowsCfg<D, NC>;
    constexpr int NKT = C::NKT, NW = C::NW, NST = C::NST, RS = C::RS, KSZ = ksz_bytes(D), TB = tile_bytes(D);
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, i = lane & 3;
    uint8_t *stg = smem + (size_t)warp * C::WARP_SMEM;
    uint64_t *bars = reinterpret_cast<uint64_t *>(stg + NST * C::STAGE);
    int2 *meta = reinterpret_cast<int2 *>(stg + NST * C::STAGE + 64);   // (valid tokens, block) of each stage
    if (lane < NST) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(ch_smem(&bars[lane])) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int gw = warp * gridDim.x + blockIdx.x;   // warp indices dealt across the CTAs first
    if (gw >= a.NWp) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long x0 = ch_range_start(a.W, a.NWp, gw), x1 = ch_range_start(a.W, a.NWp, gw + 1);

    Cursor ic;
    ic.x = x0;
    ic.e = ch_entry_of(st, a.nseq, x0);
    {
        const ChunkSeq &s = st.e[ic.e];
        const unsigned rel = (unsigned)(x0 - s.base);   // a sequence's items fit 32 bits (checked on the host)
        const int h = (int)(rel / (unsigned)s.Iu), off = (int)(rel % (unsigned)s.Iu);
        ic.hkv = h / s.S;
        ic.sl = h % s.S;
        ic.unit(st);
        ic.off = off;
        if (off > s.Sf) {
            ic.jp = (off - s.Sf) / a.CPB;
            ic.k = (off - s.Sf) % a.CPB;
        }
    }
    Cursor cc = ic;

    auto cold_of = [&](int u, int &ncold, int &chead) {
        ncold = a.C > 0 ? __ldg(a.cmeta + 2 * u) : 0;
        chead = a.C > 0 ? __ldg(a.cmeta + 2 * u + 1) : 0;
    };
    auto issue = [&](const Cursor &c, int sg) {
        const ChunkSeq &s = st.e[c.e];
        const int hkv = c.hkv, b = a.B0 + c.e, u = b * a.Hkv + hkv;
        uint8_t *dst = stg + sg * C::STAGE;
        int2 m = make_int2(0, 0);
        if (c.off < c.Sf) {
            int ncold, chead;
            cold_of(u, ncold, chead);
            const int f0 = c.off * FI, cnt = min(FI, s.ntail + s.npool + ncold + s.nnew - f0);
            if (cnt > 0) {
                m.x = cnt;
                if (lane == 0) expect_tx(&bars[sg], 2 * FI * D * 2);
                __syncwarp();
                // rows past the end repeat the first (finite values under a zero weight)
                if (lane < 2 * FI) {
                    const int x = lane & (FI - 1);
                    bulk_copy(dst + (size_t)lane * RS * 2,
                              chunk_fp16_row(a, s, b, hkv, u, f0 + (x < cnt ? x : 0), ncold, chead, lane >= FI, D),
                              D * 2, &bars[sg]);
                }
            }
        } else {
            const int jp = c.jp, k = c.k;
            const int j = jp < s.nsink ? __ldg(a.sel + (size_t)u * a.NB + jp) : s.jlo + jp - s.nsink;
            // of a listed block, the first tokens: they come first
            const int rem = j < 0 ? 0 : min(CT, (jp < s.nsink ? min(a.sinks, chunk_block_cnt(a, u, j)) : chunk_block_cnt(a, u, j)) - CT * k);
            if (rem > 0) {
                m = make_int2(rem, j);
                if (lane == 0) {
                    const int nt = (rem + TILE - 1) / TILE;
                    const size_t own = (size_t)u * a.NB + j;
                    const uint8_t *src = a.blk + (a.bt ? (size_t)__ldg(a.bt + own) : own) * a.blk_bytes;
                    const bool hdr = k == 0 || c.x == x0;
                    expect_tx(&bars[sg], (uint32_t)((hdr ? KSZ : 0) + nt * TB));
                    if (hdr) bulk_copy(dst, src, KSZ, &bars[sg]);
                    bulk_copy(dst + KSZ, src + KSZ + (size_t)k * CHUNK_TILES * TB, (uint32_t)(nt * TB), &bars[sg]);
                }
            }
        }
        if (lane == 0) meta[sg] = m;
    };

    uint32_t Bq[NC][NKT][2];          // queries: B operand, column r of each group
    uint32_t ks2[NKT][2];             // the block's key scales, A operand order
    float off2[NC][2];                // q . (z + s) of columns 2i, 2i + 1, in log2 units
    bool wide = false;                // the block's key scales are halves
    float acc[NC][NKT][4], m_run[NC][2], l_run[NC][2];
    int pos[NC][2], lo[NC][2];        // the columns' positions and window starts
    int uo = 0, cnt_rows = 0;
    int ncold = 0, chead = 0, hkv = 0, b = 0, u = 0;

    auto begin_unit = [&](const Cursor &c) {
        const ChunkSeq &s = st.e[c.e];
        hkv = c.hkv;
        b = a.B0 + c.e;
        u = b * a.Hkv + hkv;
        cold_of(u, ncold, chead);
        const int v0 = c.sl * C::RB, vend = s.nq * a.g;
        cnt_rows = min(C::RB, vend - v0);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
            const int v = min(v0 + 8 * nc + r, vend - 1);   // rows past the last repeat it, unused
            const __half *qp = a.q + (((size_t)b * a.Hq + hkv * a.g + v % a.g) * a.n + v / a.g) * D;
#pragma unroll
            for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
                for (int o = 0; o < 2; ++o)
                    Bq[nc][kt][o] = __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * kt + 2 * i + 8 * o));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                pos[nc][x] = s.pos0 + min(v0 + 8 * nc + 2 * i + x, vend - 1) / a.g;
                lo[nc][x] = a.window > 0 ? pos[nc][x] - a.window + 1 : 0;
                m_run[nc][x] = -CUDART_INF_F;
                l_run[nc][x] = 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < NKT; ++mt) acc[nc][mt][0] = acc[nc][mt][1] = acc[nc][mt][2] = acc[nc][mt][3] = 0.0f;
        }
    };
    auto end_unit = [&]() {
        if (uo >= a.MAXU) {   // never with the host's bound; recorded instead of writing out of bounds
            if (lane == 0) atomicExch(&a.ctl[1], 1);
            return;
        }
        float *pb = a.part + ((size_t)gw * a.MAXU + uo) * a.RV * (D + 2);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float l = l_run[nc][x];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int col = 8 * nc + 2 * i + x;
                if (col < cnt_rows) {
                    float *p = pb + (size_t)col * (D + 2);
                    if (r == 0) *reinterpret_cast<float2 *>(p) = make_float2(m_run[nc][x], l);
#pragma unroll
                    for (int mt = 0; mt < NKT; ++mt) {
                        p[2 + 16 * mt + r] = acc[nc][mt][x];
                        p[2 + 16 * mt + r + 8] = acc[nc][mt][2 + x];
                    }
                }
            }
        ++uo;
    };
    // Scores whose largest (log2 units) are mx in this lane: the reference
    // that weights are taken against moves up, and the sums and outputs are
    // rescaled, only when one has grown by 2^GROW (the common case is one vote
    // and no exchange).
    auto rescale = [&](float (&mx)[NC][2]) {
        bool grew = false;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int x = 0; x < 2; ++x) grew |= mx[nc][x] > m_run[nc][x] + GROW;
        if (!__any_sync(0xffffffffu, grew)) return;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
            float al[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = fmaxf(mx[nc][x], m_run[nc][x]);
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                al[x] = v > m_run[nc][x] ? ch_ex2(m_run[nc][x] - v) : 1.0f;
                l_run[nc][x] *= al[x];
                m_run[nc][x] = v;
            }
#pragma unroll
            for (int mt = 0; mt < NKT; ++mt) {
                acc[nc][mt][0] *= al[0];
                acc[nc][mt][1] *= al[1];
                acc[nc][mt][2] *= al[0];
                acc[nc][mt][3] *= al[1];
            }
        }
    };

    // prime the ring
    int st_issue = 0;
    for (int k = 0; k < NST && ic.x < x1; ++k) {
        issue(ic, st_issue);
        ic.next(a, st);
        st_issue = st_issue + 1 == NST ? 0 : st_issue + 1;
    }
    begin_unit(cc);
    __syncwarp();

    uint32_t phase = 0;
    int sg = 0;
    const Magic mg;
    while (cc.x < x1) {
        const ChunkSeq &s = st.e[cc.e];
        const int2 mt_ = meta[sg];
        uint8_t *stage = stg + sg * C::STAGE;
        const bool fp = cc.off < cc.Sf;
        if (mt_.x > 0) {
            const bool wnd = a.window > 0;
            const int k = cc.k;
            const int32_t *bi = a.bidx + ((size_t)u * a.NB + mt_.y) * a.G + CT * k;   // the chunk's token indices
            if (!fp && wnd && lane < 8) asm volatile("prefetch.global.L1 [%0];" ::"l"(bi + min(8 * lane, mt_.x - 1)));
            if (!mbar_wait(&bars[sg], (phase >> sg) & 1u)) {
                if (lane == 0) atomicExch(&a.ctl[1], 1);
                // let the other copies in flight land before giving up the buffers
                for (int x = 0; x < NST; ++x)
                    if (x != sg) mbar_wait(&bars[x], (phase >> x) & 1u);
                return;
            }
            phase ^= 1u << sg;
            if (fp) {
                const __half *kr = reinterpret_cast<const __half *>(stage), *vr = kr + FI * RS;
                const int f = cc.off * FI + r;
                const bool have = r < mt_.x;
                const int t = have ? chunk_fp16_pos(a, s, u, f, ncold, chead) : INT_MAX;
                float d[NC][4], mx[NC][2];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) d[nc][0] = d[nc][1] = d[nc][2] = d[nc][3] = 0.0f;
#pragma unroll
                for (int kt = 0; kt < NKT; kt += 2) {
                    uint32_t f4[4];   // (kt, lo), (kt, hi), (kt + 1, lo), (kt + 1, hi); rows 8..15 are zero
                    ldsm_x4(f4, kr + (lane & 7) * RS + 16 * kt + 8 * (lane >> 3));
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) {
                        mma16816(d[nc], f4[0], 0u, f4[1], 0u, Bq[nc][kt][0], Bq[nc][kt][1]);
                        mma16816(d[nc], f4[2], 0u, f4[3], 0u, Bq[nc][kt + 1][0], Bq[nc][kt + 1][1]);
                    }
                }
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        mx[nc][x] = d[nc][x] =
                            chunk_sees(t, pos[nc][x], lo[nc][x], a.sinks) ? d[nc][x] * a.sl2 : -CUDART_INF_F;
                rescale(mx);
                uint32_t bp[NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    float p[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        p[x] = ch_ex2(d[nc][x] - (m_run[nc][x] == -CUDART_INF_F ? 0.0f : m_run[nc][x] - LIFT));
                        l_run[nc][x] += p[x];
                    }
                    bp[nc] = transpose8x8(ch_h2(__floats2half2_rn(p[0], p[1])));
                }
#pragma unroll
                for (int mt = 0; mt < NKT; mt += 2) {
                    uint32_t f4[4];
                    ldsm_x4_t(f4, vr + (lane & 7) * RS + 16 * mt + 8 * (lane >> 3));
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) {
                        mma1688(acc[nc][mt], f4[0], f4[1], bp[nc]);
                        mma1688(acc[nc][mt + 1], f4[2], f4[3], bp[nc]);
                    }
                }
            } else {
                if (k == 0 || cc.x == x0) {
                    // the block's key scales, and q . (z + s) by MMAs whose A
                    // rows all hold hi(z + s) (rows 0..7) or lo(z + s)
                    float d[NC][4];
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) d[nc][0] = d[nc][1] = d[nc][2] = d[nc][3] = 0.0f;
                    uint32_t top = 0;   // the largest scales
#pragma unroll
                    for (int kt = 0; kt < NKT; ++kt) {
                        uint32_t hi[2], lw[2];
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const uint2 sz = *reinterpret_cast<const uint2 *>(stage + 4 * (16 * kt + 2 * i + 8 * o));
                            const uint32_t s2 = __byte_perm(sz.x, sz.y, 0x5410);
                            top = __vmaxu2(top, s2);
                            ks2[kt][o] = s2;
                            ch_offset(s2, __byte_perm(sz.x, sz.y, 0x7632), hi[o], lw[o]);
                        }
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
                            mma16816(d[nc], hi[0], lw[0], hi[1], lw[1], Bq[nc][kt][0], Bq[nc][kt][1]);
                    }
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                        for (int x = 0; x < 2; ++x) off2[nc][x] = (d[nc][x] + d[nc][2 + x]) * a.sl2;
                    wide = __any_sync(0xffffffffu, ch_wide(top) || ch_wide(top >> 16));
                    if (wide) {
#pragma unroll
                        for (int kt = 0; kt < NKT; ++kt)
#pragma unroll
                            for (int o = 0; o < 2; ++o) ks2[kt][o] = ch_h2(__hmul2(ch_as_h2(ks2[kt][o]), __float2half2_rn(0.5f)));
                    }
                }
                // one tile of 16 slots at a time: a loop body that the
                // instruction cache holds (four tiles unrolled measured twice the time)
                const int nt = (mt_.x + TILE - 1) / TILE;
                // (twice: scores of halved scales, in a body of their own, so that the common one stays as it is)
                auto block_tiles = [&](auto twice) {
#pragma unroll 1
                    for (int tau = 0; tau < nt; ++tau) {
                        const uint8_t *tb = stage + KSZ + tau * TB;
                        float sc[NC][4], sd[NC][4], mx[NC][2];   // two chains of products, even and odd k-tiles
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                            for (int x = 0; x < 4; ++x) sc[nc][x] = sd[nc][x] = 0.0f;
                        {
                            uint32_t w[NW], w8[NW];
                            lds_words<NW>(tb + tile_k_off(D) + lane * NW * 4, w);
#pragma unroll
                            for (int x = 0; x < NW; ++x) w8[x] = w[x] >> 8;
#pragma unroll
                            for (int kt = 0; kt < NKT; ++kt) {
                                uint32_t f4[4];   // (token r + 8 th, channels 16 kt + 8 o): f4[th + 2 o]
#pragma unroll
                                for (int o = 0; o < 2; ++o)
#pragma unroll
                                    for (int th = 0; th < 2; ++th) {
                                        const int q = o * NKT + kt, wi = 2 * (q >> 3) + th;
                                        f4[th + 2 * o] = ch_key(mg, w[wi], w8[wi], q & 7, ks2[kt][o]);
                                    }
#pragma unroll
                                for (int nc = 0; nc < NC; ++nc)
                                    mma16816(kt & 1 ? sd[nc] : sc[nc], f4[0], f4[1], f4[2], f4[3], Bq[nc][kt][0], Bq[nc][kt][1]);
                            }
#pragma unroll
                            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                                for (int x = 0; x < 4; ++x) sc[nc][x] = decltype(twice)::value ? 2.0f * (sc[nc][x] + sd[nc][x]) : sc[nc][x] + sd[nc][x];
                        }
                        if (wnd || mt_.x < 16 * tau + 16) {   // a window, or the block's last tile
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int x = 16 * tau + r + 8 * h;
                                const int t = x >= mt_.x ? INT_MAX : (wnd ? __ldg(bi + x) : 0);
#pragma unroll
                                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                                    for (int y = 0; y < 2; ++y)
                                        if (!chunk_sees(t, pos[nc][y], lo[nc][y], a.sinks)) sc[nc][2 * h + y] = -CUDART_INF_F;
                            }
                        }
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                            for (int x = 0; x < 2; ++x) mx[nc][x] = fmaf(fmaxf(sc[nc][x], sc[nc][2 + x]), a.sl2, off2[nc][x]);
                        rescale(mx);
                        uint32_t bp[NC][2];   // weights, B operand: tokens 2i, 2i + 1 (+ 8) of column r
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc) {
                            float add[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                add[x] = off2[nc][x] - (m_run[nc][x] == -CUDART_INF_F ? 0.0f : m_run[nc][x] - LIFT);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float p[2];
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    p[x] = ch_ex2(fmaf(sc[nc][2 * h + x], a.sl2, add[x]));
                                    l_run[nc][x] += p[x];
                                }
                                bp[nc][h] = transpose8x8(ch_h2(__floats2half2_rn(p[0], p[1])));
                            }
                        }
                        uint32_t w[NW], w8[NW];
                        lds_words<NW>(tb + tile_v_off(D) + lane * NW * 4, w);
#pragma unroll
                        for (int x = 0; x < NW; ++x) w8[x] = w[x] >> 8;
#pragma unroll
                        for (int gm = 0; gm < NKT / 2; ++gm) {   // a value group: 32 channels, two m-tiles
                            const uint4 sz = *reinterpret_cast<const uint4 *>(tb + tile_sz_off(D) + (gm * 4 + i) * 16);
                            const uint32_t s2[2] = {__byte_perm(sz.x, sz.y, 0x5410), __byte_perm(sz.z, sz.w, 0x5410)};
                            const uint32_t z2[2] = {__byte_perm(sz.x, sz.y, 0x7632), __byte_perm(sz.z, sz.w, 0x7632)};
#pragma unroll
                            for (int mm = 0; mm < 2; ++mm) {
                                const int mt = 2 * gm + mm;
                                uint32_t f4[4];   // (channels r + 8 half, tokens 2i + 8 tp): f4[half + 2 tp]
#pragma unroll
                                for (int tp = 0; tp < 2; ++tp)
#pragma unroll
                                    for (int half = 0; half < 2; ++half) {
                                        const int q = half * NKT + mt, wi = 2 * (q >> 3) + tp;
                                        f4[half + 2 * tp] = ch_val(mg, w[wi], w8[wi], q & 7, s2[tp], z2[tp]);
                                    }
#pragma unroll
                                for (int nc = 0; nc < NC; ++nc)
                                    mma16816(acc[nc][mt], f4[0], f4[1], f4[2], f4[3], bp[nc][0], bp[nc][1]);
                            }
                        }
                    }
                };
                if (wide)
                    block_tiles(std::true_type{});
                else
                    block_tiles(std::false_type{});
            }
        }
        // refill the stage, move on
        __syncwarp();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (ic.x < x1) {
            issue(ic, sg);
            ic.next(a, st);
            __syncwarp();
        }
        const bool other = cc.next(a, st);
        sg = sg + 1 == NST ? 0 : sg + 1;
        if (other || cc.x >= x1) {
            end_unit();
            if (cc.x < x1) begin_unit(cc);
        }
    }
}

// Merge a row's partials: a CTA of cw warps per (sequence, query head,
// token), the warps' shares merged through shared memory.
constexpr int CMB_MAXW = 16;
template <int D>
__global__ void __launch_bounds__(CMB_MAXW * 32)
    k_chunk_combine(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkTable st, int RB) {
    constexpr int CPL = D / 32, GRP = 8;
    __shared__ float red[CMB_MAXW][D + 2];
    const int cw = blockDim.x >> 5, wi = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ChunkSeq &s = st.e[blockIdx.y];
    const int hq = blockIdx.x / a.n, tk = blockIdx.x % a.n;
    if (tk >= s.nq || s.S == 0) return;
    const int v = tk * a.g + hq % a.g, h = (hq / a.g) * s.S + v / RB, col = v % RB;
    const long long ub = s.base + (long long)h * s.Iu, ue = ub + s.Iu;
    const int wa = ch_warp_of(a.W, a.NWp, ub), wb = ch_warp_of(a.W, a.NWp, ue - 1);
    // the unit's place among those of warp wa
    const long long xa = ch_range_start(a.W, a.NWp, wa);
    const int ea = ch_entry_of(st, a.nseq, xa);
    const int uo_a = s.ubase + h - (st.e[ea].ubase + (int)((unsigned)(xa - st.e[ea].base) / (unsigned)st.e[ea].Iu));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float M = -CUDART_INF_F, L = 0.0f, acc[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) acc[c] = 0.0f;
    for (int k0 = wa + wi * GRP; k0 <= wb; k0 += cw * GRP) {
        float ms[GRP], ls[GRP], vs[GRP][CPL];
#pragma unroll
        for (int x = 0; x < GRP; ++x) {
            ms[x] = -CUDART_INF_F;
            ls[x] = 0.0f;
#pragma unroll
            for (int c = 0; c < CPL; ++c) vs[x][c] = 0.0f;
            const int w = k0 + x;
            if (w <= wb) {
                const float *p = a.part + (((size_t)w * a.MAXU + (w == wa ? uo_a : 0)) * a.RV + col) * (D + 2);
                ms[x] = p[0];
                ls[x] = p[1];
#pragma unroll
                for (int c = 0; c < CPL; c += 2) {
                    const float2 t = *reinterpret_cast<const float2 *>(p + 2 + lane * CPL + c);
                    vs[x][c] = t.x;
                    vs[x][c + 1] = t.y;
                }
            }
        }
        float mn = M;
#pragma unroll
        for (int x = 0; x < GRP; ++x) mn = fmaxf(mn, ms[x]);
        // (no maximum yet: nothing seen, or scores that are NaN, and then the sum, too, which stays)
        const float mr = mn == -CUDART_INF_F ? 0.0f : mn, so = ch_ex2(M - mr);
        L *= so;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc[c] *= so;
#pragma unroll
        for (int x = 0; x < GRP; ++x) {
            const float sn = ch_ex2(ms[x] - mr);   // 0 where nothing was seen
            L = fmaf(sn, ls[x], L);
#pragma unroll
            for (int c = 0; c < CPL; ++c) acc[c] = fmaf(sn, vs[x][c], acc[c]);
        }
        M = mn;
    }
    if (cw > 1) {
        if (lane == 0) {
            red[wi][0] = M;
            red[wi][1] = L;
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) red[wi][2 + lane * CPL + c] = acc[c];
        __syncthreads();
        if (wi != 0) return;
        M = -CUDART_INF_F;
        for (int x = 0; x < cw; ++x) M = fmaxf(M, red[x][0]);
        L = 0.0f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc[c] = 0.0f;
        for (int x = 0; x < cw; ++x) {
            const float sx = red[x][0] == -CUDART_INF_F ? 0.0f : ch_ex2(red[x][0] - M);
            L = fmaf(sx, red[x][1], L);
#pragma unroll
            for (int c = 0; c < CPL; ++c) acc[c] = fmaf(sx, red[x][2 + lane * CPL + c], acc[c]);
        }
    }
    const size_t at = (((size_t)(a.B0 + blockIdx.y) * a.Hq + hq) * a.n + tk) * D;
    const float inv = chunk_norm(L, a.k == nullptr, a.q + at, D);
    __half *o = a.out + at + lane * CPL;
    uint32_t w[CPL / 2];
#pragma unroll
    for (int c = 0; c < CPL; c += 2) w[c / 2] = ch_h2(__floats2half2_rn(acc[c] * inv, acc[c + 1] * inv));
    if constexpr (CPL == 4)
        *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(o) = w[0];
}

// The blocks j < jlo of each unit that hold one of the sequence's first
// `sinks` tokens, ascending, into sel[u][0 .. nsink), -1 behind them. A
// block's indices ascend, so its first one decides; a token lies in one
// block at most, so there are at most `sinks` such blocks.
constexpr int SINK_THREADS = 256, SINK_PER = 4;   // blocks per thread and round, their loads in flight together
// (The decode kernel's warps looking for the blocks themselves, up to 32 of
// them, spared a windowed step of batch 32 this launch, 56 -> 54 us, and cost
// every call of rows mode registers: verification of four tokens 129 -> 133.)
__global__ void __launch_bounds__(SINK_THREADS)
    k_window_sinks(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkTable st, int32_t *sel) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int e = blockIdx.x / a.Hkv, u = a.B0 * a.Hkv + blockIdx.x;
    const int jlo = st.e[e].jlo, nsink = st.e[e].nsink;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nsink == 0) return;
    constexpr int NWARP = SINK_THREADS / 32;
    __shared__ int wcnt[SINK_PER][NWARP];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int32_t *out = sel + (size_t)u * a.NB;
    int found = 0;
    for (int j0 = 0; j0 < jlo; j0 += SINK_THREADS * SINK_PER) {
        int first[SINK_PER];
#pragma unroll
        for (int y = 0; y < SINK_PER; ++y) {
            const int j = j0 + y * SINK_THREADS + threadIdx.x;
            first[y] = j < jlo && chunk_block_cnt(a, u, j) > 0 ? __ldg(a.bidx + ((size_t)u * a.NB + j) * a.G) : INT_MAX;
        }
        unsigned bal[SINK_PER];
#pragma unroll
        for (int y = 0; y < SINK_PER; ++y) {
            bal[y] = __ballot_sync(0xffffffffu, first[y] < a.sinks);
            if (lane == 0) wcnt[y][wid] = __popc(bal[y]);
        }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < SINK_PER; ++y) {
            int before = found;
            for (int x = 0; x < NWARP; ++x) {
                before += x < wid ? wcnt[y][x] : 0;
                found += wcnt[y][x];
            }
            const int at = before + __popc(bal[y] & ((1u << lane) - 1u));
            if (first[y] < a.sinks && at < nsink) out[at] = j0 + y * SINK_THREADS + threadIdx.x;
        }
        __syncthreads();
    }
    for (int x = found + threadIdx.x; x < nsink; x += SINK_THREADS) out[x] = -1;
}

template <int D, int NC>
cudaError_t launch_rows(const ChunkArgs &a, const ChunkTable &st, cudaStream_t s) {
    using C = RowsCfg<D, NC>;
    // CTAs only as wide as the active warps need
    const int wpc = (a.NWp + a.ctas - 1) / a.ctas;
    return launch_pdl(k_chunk_rows<D, NC>, dim3((unsigned)a.ctas), wpc * 32, (size_t)C::WARP_SMEM * wpc, s, a, st);
}

template <int D, int NC>
cudaError_t rows_attribute() {
    using C = RowsCfg<D, NC>;
    static_assert(C::WARP_SMEM * C::WARPS <= 227 * 1024, "shared memory");
    return cudaFuncSetAttribute(k_chunk_rows<D, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::WARP_SMEM * C::WARPS);
}

// One launch's worth of sequences: B0 .. B0 + nseq - 1.
struct Plan {
    ChunkArgs a;
    ChunkTable st;
    int NC;       // this file's kernel: groups of 8 rows; 0: another's
    int gs;       // the decode kernel in rows mode: rows per slice; 0: tiles (ott_chunk_tiles.cu)
    int ipb;      // work items per block
    int nC;       // tiles: CTAs
    bool whole;   // ... each with a tile of its own
    bool sinks, any;
    size_t part_floats;
};

// false: the sizes do not fit the kernels' 32-bit counters
bool make_plan(const ott_cache *c, const ChunkCall &call, int B0, Plan &p) {
    ChunkArgs &a = p.a;
    a.blk = c->blk;
    a.blk_bytes = c->blk_bytes;
    a.bidx = c->bidx;
    a.bcnt = c->bcnt;
    a.bt = c->paged ? c->bt : nullptr;
    a.sel = c->sel;
    a.pidx = c->pidx;
    a.cidx = c->cidx;
    a.cmeta = c->cmeta;
    a.rk = c->rk;
    a.rv = c->rv;
    a.pk = c->pk;
    a.pv = c->pv;
    a.ck = c->ck;
    a.cv = c->cv;
    a.q = call.q;
    a.k = call.k;
    a.v = call.v;
    a.out = call.out;
    a.part = nullptr;
    a.ctl = c->ctl;
    a.n = call.n;
    a.B0 = B0;
    a.nseq = std::min(c->B - B0, CHUNK_SEQS);
    a.Hq = c->Hq;
    a.Hkv = c->Hkv;
    a.g = c->gq;
    a.NB = c->NB;
    a.G = c->G;
    a.P = c->P;
    a.C = c->cold > 0 ? c->cold : 0;
    a.ring = c->ring;
    a.jfull = (c->P + c->G - 1) / c->G;   // from this block on, the pool is full
    a.CPB = chunks_per_block(c->G);
    a.window = call.window;
    a.sinks = call.window > 0 ? call.sinks : 0;
    a.sl2 = (float)(1.4426950408889634 / std::sqrt((double)c->d));
    // 8 rows per pass where they suffice: half the accumulators, twice the warps
    const bool decode = call.k == nullptr;
    int nq_max = 0;
    for (int x = 0; x < a.nseq; ++x) nq_max = std::max(nq_max, call.lens ? call.lens[B0 + x] : call.n);
    const long long rows = (long long)nq_max * c->gq;
    p.gs = rows <= DEC_ROWS_MAX ? slice_heads((int)rows) : 0;
    p.NC = p.gs ? 0 : (rows <= 8 ? 1 : (rows <= ROWS_MAX ? 2 : 0));
    const bool tiles = p.gs == 0 && p.NC == 0;
    const int RB = tiles ? 256 : (p.gs ? p.gs : 8 * p.NC);
    a.RV = p.gs ? p.gs : (int)std::min<long long>(RB, (long long)nq_max * c->gq);
    // decode kernel: whole blocks as items where there are fewer of them than
    // warps (each item's fixed cost is then paid once per block)
    long long blocks = 0;
    for (int x = 0; p.gs && x < a.nseq; ++x) {
        const int b = B0 + x, nq = call.lens ? call.lens[b] : call.n;
        const long long T = c->ragged ? c->Tb[b] : c->T, seen = call.window > 0 ? std::min<long long>(T, (long long)call.window + nq) : T;
        blocks += (seen / c->G + 1) * c->Hkv * ((nq * (long long)c->gq + RB - 1) / RB);
    }
    const bool few = p.gs && blocks < (long long)c->sm_count * DEC_WARPS;
    p.ipb = few ? 1 : a.CPB;
    // Most slots of the list are empty (the first tokens share their first
    // block, but any of them may have passed through the pool into a later
    // one). With an item each, empty slots are warps' shares that others
    // could have worked on: batch 32 x 4K, window 1,024, four first tokens,
    // 61 us, and 56 with 8 slots an item. With warps to spare, a warp would
    // read 8 blocks one behind the other: one sequence of 131K, window 4,096,
    // 16 first tokens, 27 us, and 17 with an item each.
    a.spi = few ? 1 : 8;
    const int fi = p.gs ? FP16_CHUNK : FI;
    long long base = 0, units = 0;
    int min_iu = INT_MAX;
    p.sinks = false;
    for (int x = 0; x < a.nseq; ++x) {
        const int b = B0 + x;
        ChunkSeq &s = p.st.e[x];
        s = ChunkSeq{};
        s.base = base;
        s.ubase = (int)units;
        s.T = (int)(c->ragged ? c->Tb[b] : c->T);
        s.nf = c->ragged ? c->nfb[b] : c->nf;
        s.nq = call.lens ? call.lens[b] : call.n;
        s.nnew = decode ? 0 : s.nq;
        s.pos0 = decode ? s.T - 1 : s.T;
        const long long tail = (long long)s.nf * c->G;
        s.ntail = (int)(s.T - tail);
        s.ring_start = (int)(tail % c->ring);
        s.npool = pool_after(c->P, c->G, s.nf, c->pct);
        // the windows of all its queries start here or later; of tiles, each
        // has a range of its own, and the list covers the last one's
        const int lo = s.pos0 + (tiles ? std::max(0, s.nq - 1) : 0) - a.window + 1;
        if (a.window > 0 && lo > 0) {
            s.jlo = std::min(s.nf, lo / c->G);
            s.nsink = std::min(a.sinks, s.jlo);
        }
        s.Sf = (int)(((long long)s.ntail + s.npool + a.C + s.nnew + fi - 1) / fi);
        const long long iu = s.Sf + (p.gs ? (s.nsink + a.spi - 1) / a.spi : (long long)s.nsink * p.ipb) + (long long)(s.nf - s.jlo) * p.ipb;
        s.S = (int)(((long long)s.nq * c->gq + RB - 1) / RB);
        if (s.S == 0) continue;
        p.sinks |= s.nsink > 0;
        if (tiles) continue;
        s.Iu = (int)iu;
        min_iu = (int)std::min<long long>(min_iu, iu);
        if (iu > INT_MAX || iu * c->Hkv * s.S > INT_MAX) return false;
        base += iu * c->Hkv * s.S;
        units += (long long)c->Hkv * s.S;
        if (units > INT_MAX) return false;
    }
    if (tiles) {
        if (!plan_tiles(c, a, p.st, p.nC, p.whole, p.part_floats)) return false;
        p.any = a.W > 0;
        return true;
    }
    p.st.e[a.nseq] = ChunkSeq{};
    p.st.e[a.nseq].base = base;
    p.st.e[a.nseq].ubase = (int)units;
    a.W = base;
    p.any = base > 0;
    if (!p.any) {
        p.part_floats = 0;
        return true;
    }
    // a warp's run is one sum per unit: where it would be longer than
    // SUM_TOKENS, more CTAs than SMs
    const long long slots = (long long)c->sm_count * (p.gs ? DEC_WARPS : p.NC == 1 ? 16 : 8), most = slots * (SUM_TOKENS / CT);
    const long long waves = std::max(1LL, (a.W + most - 1) / most);
    a.ctas = (int)(c->sm_count * waves);
    a.NWp = (int)std::min<long long>(a.W, slots * waves);
    const long long L = (a.W + a.NWp - 1) / a.NWp;   // items of a warp's range, at most
    a.MAXU = (int)std::min<long long>(L, (L - 1) / min_iu + 2);
    p.part_floats = (size_t)a.NWp * a.MAXU * a.RV * (c->d + 2) * (p.gs ? 2 : 1);
    return true;
}

template <int D>
cudaError_t launch_plan(const ott_cache *c, const Plan &p, cudaStream_t s) {
    const ChunkArgs &a = p.a;
    cudaError_t e = cudaSuccess;
    if (p.sinks)
        e = launch_pdl(k_window_sinks, dim3((unsigned)(a.nseq * a.Hkv)), SINK_THREADS, 0, s, a, p.st, c->sel);
    if (e == cudaSuccess && p.gs > 0) return launch_decode_rows(c, a, p.st, p.gs, p.ipb, s);
    if (e == cudaSuccess && p.NC == 0) return launch_tiles(c, a, p.st, p.nC, p.whole, s);
    if (e == cudaSuccess)
        e = p.NC == 1 ? launch_rows<D, 1>(a, p.st, s) : launch_rows<D, 2>(a, p.st, s);
    if (e != cudaSuccess) return e;
    // about two rounds of 8 partials per combine warp
    const long long per_unit = (long long)a.NWp / std::max(1, p.st.e[a.nseq].ubase) + 2;
    const int cw = (int)std::max<long long>(1, std::min<long long>(CMB_MAXW, (per_unit + 15) / 16));
    return launch_pdl(k_chunk_combine<D>, dim3((unsigned)((long long)a.Hq * a.n), (unsigned)a.nseq), 32 * cw, 0, s, a,
                      p.st, 8 * p.NC);
}

}  // namespace

cudaError_t set_chunk_attributes(int d, int smem_max) {
    cudaError_t e = set_decode_rows_attributes(d, smem_max);
    if (e != cudaSuccess) return e;
    e = d == 128 ? rows_attribute<128, 1>() : rows_attribute<64, 1>();
    if (e != cudaSuccess) return e;
    const cudaError_t e2 = d == 128 ? rows_attribute<128, 2>() : rows_attribute<64, 2>();
    return e2 == cudaSuccess ? set_tiles_attributes(d) : e2;
}

int run_chunk(const ott_cache *c, const ChunkCall &call, cudaStream_t s, cudaError_t &err) {
    err = cudaSuccess;
    if ((long long)c->Hq * call.n > INT_MAX) return OTT_ERR_INVALID;
    Plan p;
    size_t need = 0;
    for (int B0 = 0; B0 < c->B; B0 += CHUNK_SEQS) {
        if (!make_plan(c, call, B0, p)) return OTT_ERR_INVALID;
        need = std::max(need, p.part_floats);
    }
    if (need == 0) return OTT_OK;
    Scratch scr(c, need, s);
    if (!scr.ptr) return OTT_ERR_OOM;
    for (int B0 = 0; B0 < c->B && err == cudaSuccess; B0 += CHUNK_SEQS) {
        make_plan(c, call, B0, p);
        if (!p.any) continue;
        p.a.part = static_cast<float *>(scr.ptr);
        err = c->d == 128 ? launch_plan<128>(c, p, s) : launch_plan<64>(c, p, s);
    }
    const cudaError_t e2 = scr.release();
    if (err == cudaSuccess) err = e2;
    return err == cudaSuccess ? OTT_OK : OTT_ERR_CUDA;
}

}  // namespace ott
