// ott_byte_rows.cu -- attention of few query rows per kv head over the cache
// held in 8 bits, over all its blocks or over those that a bound selects; the
// plan of every such call (more than 16 rows go to ott_byte_tiles.cu).
//
// Mathematics. A code is an exact fp16 number, so the tensor cores get the
// codes themselves: scores are (q . code) * ks, one multiplication in fp32. The
// values' scale goes into the weight: with lv = log2(vs),
//     z = (q . code) ks log2(e) / sqrt(d) + lv,   w = 2^(z - m),
//     out = sum w code / sum (w / vs),
// where m runs with the largest z (not the largest score). So a block costs
// no operation per element for its scales, and a weight is rounded once, to
// fp16, where its product with the codes counts most; what falls below fp16's
// range is small beside the row's largest w * code, whatever its scale.
//
// Layout of the work, as ott_chunk.cu's: a unit is a (sequence, kv head, slice
// of 8 or 16 query rows), row v = token * g + head; with selected blocks, a
// slice of one token's heads. Work items are what a copy brings: 16 fp16
// tokens, or 32 tokens of a block (64 d bytes, contiguous, as the lanes'
// fragments: 16-byte loads from shared memory, no transposition; and the
// block's record). Every warp gets an equal contiguous run of the items of all
// units, with a ring of stages of its own that its copies fill ahead. It leaves
// one partial per unit that it touches, in a place that goes by the run;
// k_byte_combine merges the partials of a row. A CTA whose warps all work for
// one unit merges their results first (131K tokens of 8 kv heads: 33 partials a
// row instead of 152, the merge 8 -> 5 us).
// SMs do not get equal shares of HBM: with equal runs alone, the warps of batch
// 32 x 4K, 32 heads, ended between 133 and 168 us. So in long calls only the
// first seven eighths of a unit's items (its A items) are cut into equal runs,
// one per warp; the rest (B items) are cut into short runs, about three per
// warp, which warps claim from a counter when they have nothing else to copy.
// Who took a run does not show in the result.
// Short calls, no more units than SMs, give every unit a CTA or a cluster of
// them, which reads one another's shared memory and writes the unit's rows: no
// second kernel. One sequence of 1,024 tokens, 8 kv heads (clusters of two): 6.8
// us, with a merge kernel 8.2; 4 x 2,048: 7.7 and 8.6; five drafts with 40
// blocks each (a CTA per unit) 26.6 and 29.1; one of 4,096 7.4 and 7.6.
//
// What bounds it: HBM. Batch 32 x 4K, 32 heads of d = 128 (1.07 GB of cache)
// takes 161 us, 6.7 TB/s; with four queries each, 165. Calls of a few ten us
// add the start of the copies and the merge: 131K tokens, 8 kv heads (269 MB),
// 47 us, 5.7 TB/s; 32 sequences of 1K to 7K from a paged pool (272 MB) 51. 12
// warps with two stages each instead of 8 with three: 161 and 50.5 us became
// 160 and 53.
#include <algorithm>
#include <climits>
#include <cmath>

#include "ott_byte.cuh"
#include "ott_select.cuh"

namespace ott {
namespace {

constexpr int ROWS_MAX = 16;   // rows per kv head up to which this file's kernel serves a call
constexpr int QT = 32, FT = 16;   // tokens of a work item: of a block, fp16
// Items of a unit per CTA of its own: clusters grow while a CTA has more than
// SPREAD_ITEMS (32: 4 x 2,048 tokens 7.7 -> 9.5 us) and SMs are left; beyond
// DIRECT_ITEMS a call is cut into equal runs (8 units of 513 items in clusters
// of eight, which leave 88 SMs idle: 25.2 us, in runs 19.5; 43 items, above).
constexpr int DIRECT_ITEMS = 48, SPREAD_ITEMS = 16;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

// The place of own shared memory in the CTA of that rank of the cluster.
__device__ __forceinline__ float *of_rank(float *own, int rank) {
    uint64_t at;
    asm("mapa.u64 %0, %1, %2;" : "=l"(at) : "l"(own), "r"(rank));
    return reinterpret_cast<float *>(at);
}
// Every thread of the cluster's CTAs that still run comes by; what they wrote before is visible behind it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// NC groups of 8 query rows (the columns of an MMA).
template <int D, int NC>
struct RowsCfg {
    static constexpr int NKS = D / 16, PP = D / 64;
    static constexpr int WARPS = 8, NST = 3;
    static constexpr int ITEM = QT * 2 * D;                // bytes of a block's item
    static constexpr int STAGE = ITEM + 128;               // with its record; 16 fp16 tokens fit, too
    static_assert(2 * FT * D * 2 <= ITEM, "fp16 items");
    static constexpr int WARP_SMEM = NST * STAGE + 256;    // stages, barriers, what each stage holds
    static_assert(STAGE % 128 == 0 && NST * 8 <= 64, "stages");
    static_assert(WARP_SMEM * WARPS <= 227 * 1024, "shared memory");
};

// The entry that holds work item x: the last one whose base (of A or B items) is <= x.
template <bool B>
__device__ __forceinline__ int entry_of(const ByteTable &st, int nseq, long long x) {
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((B ? st.e[mid].base2 : st.e[mid].base) <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A work item: its unit (entry, kv head, slice of rows), its number in the
// unit, and for one of a block the block's place and the part.
struct Cursor {
    int e, hkv, sl, off, jp, k;
    int lo, hi, Sf;   // of the entry: the unit's items of this kind, its fp16 items
    bool b;           // B items
    __device__ __forceinline__ void unit(const ByteArgs &a, const ByteTable &st, int skip) {
        const ByteSeq &s = st.e[e];
        lo = b ? s.Ia : 0;
        hi = b ? s.Iu : s.Ia;
        Sf = s.Sf;
        off = lo + skip;
        const int x = max(0, off - Sf);
        jp = x / a.IPB;
        k = x % a.IPB;
    }
    __device__ __forceinline__ void seek(const ByteArgs &a, const ByteTable &st, bool b_, long long x) {
        b = b_;
        e = b ? entry_of<true>(st, a.nseq, x) : entry_of<false>(st, a.nseq, x);
        const ByteSeq &s = st.e[e];
        const unsigned rel = (unsigned)(x - (b ? s.base2 : s.base)), len = (unsigned)(b ? s.Iu - s.Ia : s.Ia);   // (32 bits: checked on the host)
        const int h = (int)(rel / len);
        hkv = h / s.S;
        sl = h % s.S;
        unit(a, st, (int)(rel % len));
    }
    // true: the next item is another unit's
    __device__ __forceinline__ bool next(const ByteArgs &a, const ByteTable &st) {
        if (off++ >= Sf && ++k == a.IPB) {
            k = 0;
            ++jp;
        }
        if (off < hi) return false;
        if (++sl == st.e[e].S) {
            sl = 0;
            if (++hkv == a.Hkv) {
                hkv = 0;
                do ++e;
                while (e < a.nseq && (st.e[e].S == 0 || (b && st.e[e].Iu == st.e[e].Ia)));
            }
        }
        if (e < a.nseq) unit(a, st, 0);
        return true;
    }
};

// What a stage holds: valid tokens (0: none, nothing to wait for; -1: no more
// items), the unit, first fp16 token (of the new ones: + FRESH; -1: a block's
// item), whether it is the first of its unit in the run, and if it is the last
// the partial's place, else -1.
struct Desc {
    int valid, e, hkv, sl, f0, first, part, pad;
};
constexpr int FRESH = 1 << 30;

// A items x0 .. x1 - 1 (x0 < x1) are of one unit.
__device__ __forceinline__ bool one_unit(const ByteArgs &a, const ByteTable &st, long long x0, long long x1) {
    const int e = entry_of<false>(st, a.nseq, x0);
    const unsigned Ia = (unsigned)st.e[e].Ia, rel = (unsigned)(x0 - st.e[e].base);
    return x1 <= st.e[e].base + (long long)(rel / Ia + 1) * Ia;
}

// Rows of slice sl of an entry: first row, number of rows (a row is token * g + head).
__device__ __forceinline__ void slice_rows(const ByteArgs &a, const ByteSeq &s, int sl, int &v0, int &cnt) {
    if (a.sel) {
        const int h0 = sl % a.SG * a.RB;
        v0 = sl / a.SG * a.g + h0;
        cnt = min(a.RB, a.g - h0);
    } else {
        v0 = sl * a.RB;
        cnt = min(a.RB, s.nq * a.g - v0);
    }
}

template <int D, int NC, int FMT>
__global__ void __launch_bounds__(RowsCfg<D, NC>::WARPS * 32, 1)
    k_byte_rows(const __grid_constant__ ByteArgs a, const __grid_constant__ ByteTable st) {
    using C = RowsCfg<D, NC>;
    constexpr int NKS = C::NKS, PP = C::PP, NST = C::NST;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, i = lane & 3;
    const int rot = D == 128 ? 8 * (i >> 1) : 0;
    uint8_t *stg = smem + (size_t)warp * C::WARP_SMEM;
    uint64_t *bars = reinterpret_cast<uint64_t *>(stg + NST * C::STAGE);
    Desc *desc = reinterpret_cast<Desc *>(stg + NST * C::STAGE + 64);
    if (lane < NST) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(ch_smem(&bars[lane])) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int wpc = blockDim.x >> 5, gw = blockIdx.x * wpc + warp;
    // A CTA whose warps all work for one unit merges their results.
    bool merge = a.direct;
    if (!a.direct && wpc > 1 && a.Wb == 0) {
        const int g1 = min(a.NWp, (int)(blockIdx.x + 1) * wpc);
        merge = g1 > (int)blockIdx.x * wpc && one_unit(a, st, ch_range_start(a.W, a.NWp, blockIdx.x * wpc), ch_range_start(a.W, a.NWp, g1));
    }
    if (!a.direct && gw >= a.NWp) {   // the last CTA may have warps to spare
        if (merge) __syncthreads();
        return;
    }   // (the others wait for the kernel before this one below, and so does the grid)
    // the run at hand: the next item, how many are left, the places of its partials
    Cursor ic;
    int left;
    const int rank = a.direct ? (int)blockIdx.x % a.cluster : 0;
    if (a.direct) {   // this CTA's unit, this warp's share of it (there may be none)
        const int unit = (int)blockIdx.x / a.cluster, part = rank * wpc + warp, parts = a.cluster * wpc;
        int e = 0;
        for (int hi = a.nseq; hi - e > 1;) {
            const int mid = (e + hi) >> 1;
            if (st.e[mid].ubase <= unit) e = mid;
            else hi = mid;
        }
        const int h = unit - st.e[e].ubase, from = (int)((long long)st.e[e].Iu * part / parts);
        ic.b = false;
        ic.e = e;
        ic.hkv = h / st.e[e].S;
        ic.sl = h % st.e[e].S;
        ic.unit(a, st, from);
        left = (int)((long long)st.e[e].Iu * (part + 1) / parts) - from;
    } else {
        const long long x0 = ch_range_start(a.W, a.NWp, gw);
        left = (int)(ch_range_start(a.W, a.NWp, gw + 1) - x0);
        ic.seek(a, st, false, x0);
    }
    size_t place = (size_t)gw * a.MAXU;
    int room = a.MAXU;
    bool first = true, more = a.Wb > 0;
    int claimed = 0;        // lane 0: the run claimed last
    constexpr int CLAIM = 2;   // items before the end of a run when the next one is claimed
    auto claim = [&]() {
        if (more && lane == 0) claimed = atomicAdd(&a.ctl[2], 1);
    };

    // Slots of the next 32 blocks of the issuing cursor's unit, a lane each.
    int slots = -1, slots_from = INT_MIN;
    auto issue = [&](const Cursor &c, int sg, int &f0) {
        const ByteSeq &s = st.e[c.e];
        const int b = a.B0 + c.e, u = b * a.Hkv + c.hkv;
        uint8_t *dst = stg + sg * C::STAGE;
        int m;
        if (c.off < c.Sf) {
            const bool fresh = c.off >= s.Ft;
            f0 = (fresh ? c.off - s.Ft : c.off) * FT;
            m = min(FT, (fresh ? s.nq : s.T % a.G) - f0);
            // Two copies; the rows past the end keep what the stage held, and are masked where they are read. (A copy per
            // row, to padded rows, spared bank conflicts and cost a warp about 5,000 cycles an item.)
            if (lane == 0) {
                const size_t at = (fresh ? (size_t)u * a.n + f0 : (size_t)u * a.G + f0) * D;
                expect_tx(&bars[sg], (uint32_t)m * (2 * D * 2));
                bulk_copy(dst, (fresh ? a.k : a.tk) + at, (uint32_t)m * (D * 2), &bars[sg]);
                bulk_copy(dst + FT * D * 2, (fresh ? a.v : a.tv) + at, (uint32_t)m * (D * 2), &bars[sg]);
            }
            if (fresh) f0 += FRESH;
        } else {
            f0 = -1;
            if (c.jp < slots_from || c.jp >= slots_from + 32) {
                slots_from = c.jp;
                const int jp = c.jp + lane;
                slots = -1;
                if (jp < s.nb) {
                    int j = jp;
                    if (a.sel) j = a.sel[(((size_t)b * a.n + c.sl / a.SG) * a.Hkv + c.hkv) * a.Kc + jp];
                    const size_t own = (size_t)u * a.NB + j;
                    if (j >= 0) slots = a.bt ? a.bt[own] : (int)own;
                }
            }
            const int slot = __shfl_sync(0xffffffffu, slots, c.jp - slots_from);
            m = slot < 0 ? 0 : QT;
            if (slot >= 0 && lane == 0) {
                expect_tx(&bars[sg], C::ITEM + 16);
                bulk_copy(dst, a.blk + (size_t)slot * a.blk_bytes + (size_t)c.k * C::ITEM, C::ITEM, &bars[sg]);
                bulk_copy(dst + C::ITEM, a.rec + slot, 16, &bars[sg]);
            }
        }
        return m;
    };
    // The next item into stage sg (whose reads are done).
    auto feed = [&](int sg) {
        if (left == 0) {
            int q = 0;
            if (more) {
                q = __shfl_sync(0xffffffffu, claimed, 0);
                more = q < a.NQ;
            }
            if (!more) {
                if (lane == 0) desc[sg].valid = -1;
                return;
            }
            const long long x = ch_range_start(a.Wb, a.NQ, q);
            left = (int)(ch_range_start(a.Wb, a.NQ, q + 1) - x);
            ic.seek(a, st, true, x);
            slots_from = INT_MIN;
            place = (size_t)a.NWp * a.MAXU + (size_t)q * a.MAXU2;
            room = a.MAXU2;
            first = true;
            if (left <= CLAIM) claim();
        }
        Desc d;
        d.e = ic.e;
        d.hkv = ic.hkv;
        d.sl = ic.sl;
        d.valid = issue(ic, sg, d.f0);
        d.first = first;
        const bool other = ic.next(a, st);
        --left;
        first = other || left == 0;
        d.part = -1;
        if (other) slots_from = INT_MIN;
        if (first && !merge) {
            d.part = (int)place++;
            if (--room < 0) {   // never with the host's bound; recorded instead of writing out of bounds
                if (lane == 0) atomicExch(&a.ctl[1], 1);
                d.part = -1;
            }
        }
        if (lane == 0) desc[sg] = d;
        if (left == CLAIM) claim();
    };

    uint32_t Bq[NC][NKS][2];          // queries: B operand, column r of each group
    float acc[NC][NKS][4], m_run[NC][2], l_run[NC][2];
    int tok[NC][2];                   // the columns' tokens (of the chunk)
    int cnt_rows = 0;

    auto begin_unit = [&](const Desc &c) {
        const ByteSeq &s = st.e[c.e];
        const int b = a.B0 + c.e;
        int v0;
        slice_rows(a, s, c.sl, v0, cnt_rows);
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
            const int v = v0 + min(8 * nc + r, cnt_rows - 1);   // rows past the last repeat it, unused
            const __half *qp = a.q + (((size_t)b * a.Hq + c.hkv * a.g + v % a.g) * a.n + v / a.g) * D + (D / 4) * i;
#pragma unroll
            for (int ks = 0; ks < NKS; ++ks) {
                const uint2 w = *reinterpret_cast<const uint2 *>(qp + 16 * (ks >> 2) + ((4 * (ks & 3)) ^ rot));
                Bq[nc][ks][0] = w.x;
                Bq[nc][ks][1] = w.y;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                tok[nc][x] = (v0 + min(8 * nc + 2 * i + x, cnt_rows - 1)) / a.g;
                m_run[nc][x] = -CUDART_INF_F;
                l_run[nc][x] = 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < NKS; ++mt) acc[nc][mt][0] = acc[nc][mt][1] = acc[nc][mt][2] = acc[nc][mt][3] = 0.0f;
        }
    };
    auto end_unit = [&](int part) {
        float *pb = a.part + (size_t)part * a.RV * (D + 2);
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
                    for (int mt = 0; mt < NKS; ++mt) {
                        p[2 + 16 * mt + r] = acc[nc][mt][x];
                        p[2 + 16 * mt + r + 8] = acc[nc][mt][2 + x];
                    }
                }
            }
    };
    // z values whose largest is mx in this lane: the reference moves up, and
    // sums and outputs are rescaled, only when one has grown by 2^GROW.
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
            for (int mt = 0; mt < NKS; ++mt) {
                acc[nc][mt][0] *= al[0];
                acc[nc][mt][1] *= al[1];
                acc[nc][mt][2] *= al[0];
                acc[nc][mt][3] *= al[1];
            }
        }
    };
    // Weights of 16 tokens from their z (d[nc]: tokens r, r + 8, columns 2i,
    // 2i + 1): sums, and the B operand of the values' product.
    auto weights = [&](const float (&d)[4], int nc, float iv, uint32_t &b0, uint32_t &b1) {
        float p[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const float m = m_run[nc][y & 1];
            p[y] = ch_ex2(d[y] - (m == -CUDART_INF_F ? 0.0f : m - LIFT));
        }
        l_run[nc][0] = fmaf(p[0] + p[2], iv, l_run[nc][0]);
        l_run[nc][1] = fmaf(p[1] + p[3], iv, l_run[nc][1]);
        b0 = transpose8x8(ch_h2(__floats2half2_rn(p[0], p[1])));
        b1 = transpose8x8(ch_h2(__floats2half2_rn(p[2], p[3])));
    };

    asm volatile("griddepcontrol.wait;" ::: "memory");   // (the place in the plan is found while the kernel before runs)
    if (left <= CLAIM) claim();
    const Cursor start = ic;
    for (int k = 0; k < NST; ++k) feed(k);
    if (a.direct) {   // the rows of a warp without items, too
        Desc d;
        d.e = start.e;
        d.hkv = start.hkv;
        d.sl = start.sl;
        begin_unit(d);
    }
    __syncwarp();

    uint32_t phase = 0;
    int sg = 0;
    for (;;) {
        const Desc dc = desc[sg];
        const int valid = dc.valid;
        if (valid < 0) break;
        if (dc.first && !a.direct) begin_unit(dc);
        uint8_t *stage = stg + sg * C::STAGE;
        if (valid > 0) {
            if (!mbar_wait(&bars[sg], (phase >> sg) & 1u)) {
                if (lane == 0) atomicExch(&a.ctl[1], 1);
                // let the other copies in flight land before giving up the buffers
                for (int x = 0; x < NST; ++x)
                    if (x != sg) mbar_wait(&bars[x], (phase >> x) & 1u);
                if (merge) __syncthreads();   // the others' barriers
                if (a.direct && a.cluster > 1) {
                    cluster_sync();
                    cluster_sync();
                }
                return;
            }
            phase ^= 1u << sg;
            if (dc.f0 >= 0) {
                // 16 fp16 tokens: of the open block, or new ones (causal)
                const bool fresh = dc.f0 >= FRESH;
                const int f0 = fresh ? dc.f0 - FRESH : dc.f0;
                const __half *kr = reinterpret_cast<const __half *>(stage), *vr = kr + FT * D;
                float d[NC][4], mx[NC][2];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) d[nc][0] = d[nc][1] = d[nc][2] = d[nc][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < NKS; ks += 2) {
                    const int ch = (D / 4) * i + 16 * (ks >> 2) + ((4 * (ks & 3)) ^ rot);
                    const uint4 x = *reinterpret_cast<const uint4 *>(kr + r * D + ch);
                    const uint4 y = *reinterpret_cast<const uint4 *>(kr + (r + 8) * D + ch);
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) {
                        mma16816(d[nc], x.x, y.x, x.y, y.y, Bq[nc][ks][0], Bq[nc][ks][1]);
                        mma16816(d[nc], x.z, y.z, x.w, y.w, Bq[nc][ks + 1][0], Bq[nc][ks + 1][1]);
                    }
                }
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int t = r + 8 * (y >> 1);
                        const bool see = t < valid && (!fresh || f0 + t <= tok[nc][y & 1]);
                        d[nc][y] = see ? d[nc][y] * a.sl2 : -CUDART_INF_F;
                    }
                    mx[nc][0] = fmaxf(d[nc][0], d[nc][2]);
                    mx[nc][1] = fmaxf(d[nc][1], d[nc][3]);
                }
                rescale(mx);
                uint32_t bp[NC][2];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) weights(d[nc], nc, 1.0f, bp[nc][0], bp[nc][1]);
                // values of tokens 2i, 2i + 1 (+ 8) that there are
                auto halves = [&](int t) { return (t < valid ? 0xffffu : 0u) | (t + 1 < valid ? 0xffff0000u : 0u); };
                const uint32_t keep0 = halves(2 * i), keep1 = halves(2 * i + 8);
#pragma unroll
                for (int mt = 0; mt < NKS; ++mt) {
                    uint32_t f[4];   // (channels, tokens): (0..7, 0..7), (8..15, 0..7), (0..7, 8..15), (8..15, 8..15)
                    ldsm_x4_t(f, vr + ((lane & 7) + 8 * (lane >> 4)) * D + 16 * mt + 8 * (lane >> 3 & 1));
                    f[0] &= keep0;
                    f[1] &= keep0;
                    f[2] &= keep1;
                    f[3] &= keep1;
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) mma16816(acc[nc][mt], f[0], f[1], f[2], f[3], bp[nc][0], bp[nc][1]);
                }
            } else {
                const float4 rec = *reinterpret_cast<const float4 *>(stage + C::ITEM);   // ks, vs, lv, iv
                const float sc = rec.x * a.sl2;
                float d[2][NC][4], mx[NC][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint4 *kp = reinterpret_cast<const uint4 *>(stage + t * (C::ITEM / 2)) + lane;
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) d[t][nc][0] = d[t][nc][1] = d[t][nc][2] = d[t][nc][3] = 0.0f;
#pragma unroll
                    for (int pp = 0; pp < PP; ++pp) {
                        const uint4 x = kp[pp * 32], y = kp[(pp + PP) * 32];
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            uint32_t a0, a1, a2, a3;
                            byte_unpack<FMT>(xw[w], a0, a2);
                            byte_unpack<FMT>(yw[w], a1, a3);
#pragma unroll
                            for (int nc = 0; nc < NC; ++nc)
                                mma16816(d[t][nc], a0, a1, a2, a3, Bq[nc][4 * pp + w][0], Bq[nc][4 * pp + w][1]);
                        }
                    }
                }
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int y = 0; y < 4; ++y) d[t][nc][y] = fmaf(d[t][nc][y], sc, rec.z);
                    mx[nc][0] = fmaxf(fmaxf(d[0][nc][0], d[0][nc][2]), fmaxf(d[1][nc][0], d[1][nc][2]));
                    mx[nc][1] = fmaxf(fmaxf(d[0][nc][1], d[0][nc][3]), fmaxf(d[1][nc][1], d[1][nc][3]));
                }
                rescale(mx);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t bp[NC][2];
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) weights(d[t][nc], nc, rec.w, bp[nc][0], bp[nc][1]);
                    const uint4 *vp = reinterpret_cast<const uint4 *>(stage + t * (C::ITEM / 2) + C::ITEM / 4) + lane;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        const uint4 x = vp[c * 32];
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t a0, a1, a2, a3;
                            byte_unpack<FMT>(xw[2 * h], a0, a2);
                            byte_unpack<FMT>(xw[2 * h + 1], a1, a3);
#pragma unroll
                            for (int nc = 0; nc < NC; ++nc)
                                mma16816(acc[nc][2 * c + h], a0, a1, a2, a3, bp[nc][0], bp[nc][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        // the stage's reads (generic proxy) come before the copy that refills it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        feed(sg);
        __syncwarp();
        if (dc.part >= 0) end_unit(dc.part);
        sg = sg + 1 == NST ? 0 : sg + 1;
    }
    if (!merge) return;
    // Every warp's largest z and sum, then its output at the common reference,
    // in its first stage (its copies have all been read).
    float *const own = reinterpret_cast<float *>(stg);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float l = l_run[nc][x];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int col = 8 * nc + 2 * i + x;
            if (r == 0) *reinterpret_cast<float2 *>(own + col * (D + 2)) = make_float2(m_run[nc][x], l);
#pragma unroll
            for (int mt = 0; mt < NKS; ++mt) {
                own[col * (D + 2) + 2 + 16 * mt + r] = acc[nc][mt][x];
                own[col * (D + 2) + 2 + 16 * mt + r + 8] = acc[nc][mt][2 + x];
            }
        }
    __syncthreads();
    const int nw = a.direct ? wpc : min(wpc, a.NWp - (int)blockIdx.x * wpc);
    int v0, rows;
    slice_rows(a, st.e[start.e], start.sl, v0, rows);
    // a CTA's results go to its place among the partials; to the second stage of its first warp, for the cluster
    float *const pb = a.direct ? reinterpret_cast<float *>(smem + C::STAGE) : a.part + (size_t)(blockIdx.x * wpc) * a.MAXU * a.RV * (D + 2);
    auto write = [&](int col, float L, const float (&o)[D / 32]) {
        // a row sees a token at least, so that L = 0 means scores of -inf or NaN alone: NaN
        const int v = v0 + col;
        const float inv = 1.0f / L;
        __half *out = a.out + (((size_t)(a.B0 + start.e) * a.Hq + start.hkv * a.g + v % a.g) * a.n + v / a.g) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) out[32 * c + lane] = __float2half_rn(o[c] * inv);
    };
    for (int col = warp; col < cnt_rows; col += nw) {
        float M = -CUDART_INF_F, L = 0.0f, o[D / 32];
        for (int w = 0; w < nw; ++w) M = fmaxf(M, reinterpret_cast<const float *>(smem + (size_t)w * C::WARP_SMEM)[col * (D + 2)]);
        const float mr = M == -CUDART_INF_F ? 0.0f : M;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[c] = 0.0f;
        for (int w = 0; w < nw; ++w) {
            const float *p = reinterpret_cast<const float *>(smem + (size_t)w * C::WARP_SMEM) + col * (D + 2);
            const float sw = ch_ex2(p[0] - mr);   // 0 where nothing was seen
            L = fmaf(sw, p[1], L);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] = fmaf(sw, p[2 + 32 * c + lane], o[c]);
        }
        if (a.direct && a.cluster == 1) {
            write(col, L, o);
            continue;
        }
        float *p = pb + (size_t)col * (D + 2);
        if (lane == 0) *reinterpret_cast<float2 *>(p) = make_float2(M, L);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) p[2 + 32 * c + lane] = o[c];
    }
    if (!a.direct || a.cluster == 1) return;
    cluster_sync();
    for (int col = rank + a.cluster * warp; col < cnt_rows; col += a.cluster * wpc) {
        float *const at = pb + col * (D + 2);
        float m = -CUDART_INF_F;
        if (lane < a.cluster) m = *of_rank(at, lane);
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float mr = M == -CUDART_INF_F ? 0.0f : M;
        float L = 0.0f, o[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[c] = 0.0f;
#pragma unroll 4
        for (int x = 0; x < a.cluster; ++x) {
            const float *p = of_rank(at, x);
            const float sw = ch_ex2(__shfl_sync(0xffffffffu, m, x) - mr);   // 0 where nothing was seen
            L = fmaf(sw, p[1], L);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] = fmaf(sw, p[2 + 32 * c + lane], o[c]);
        }
        write(col, L, o);
    }
    cluster_sync();   // no CTA ends while its results are read
}

// Merge a row's partials: a CTA of cw warps per (sequence, query head, token),
// the warps' shares merged through shared memory.
constexpr int CMB_MAXW = 8;   // (small enough to wait beside the rows kernel's CTAs)
template <int D>
__global__ void __launch_bounds__(CMB_MAXW * 32)
    k_byte_combine(const __grid_constant__ ByteArgs a, const __grid_constant__ ByteTable st) {
    constexpr int CPL = D / 32, GRP = 8;
    __shared__ float red[CMB_MAXW][D + 2];
    const int cw = blockDim.x >> 5, wi = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane * CPL;
    const ByteSeq &s = st.e[blockIdx.y];
    const int hq = blockIdx.x / a.n, tk = blockIdx.x % a.n;
    const bool row = tk < s.nq;
    int wa = 0, uo_a = 0, col = 0, n0 = 0, n01 = 0, na = 0, parts = 0;
    int first = 0, inner = 0, last = 0;   // A: where the parts of the unit's first CTA, of the inner ones, and of the last begin
    size_t qa = 0;                        // B: the first part's place
    int uo_b = 0;
    if (row) {   // the plan, while the rows kernel still runs
        const int hd = hq % a.g, v = a.sel ? hd : tk * a.g + hd;
        const int sl = a.sel ? tk * a.SG + hd / a.RB : v / a.RB, h = hq / a.g * s.S + sl;
        col = v % a.RB;
        const long long ub = s.base + (long long)h * s.Ia, ue = ub + s.Ia;
        wa = ch_warp_of(a.W, a.NWp, ub);
        const int wb = ch_warp_of(a.W, a.NWp, ue - 1);
        // the unit's place among those of warp wa
        const long long xa = ch_range_start(a.W, a.NWp, wa);
        const int ea = entry_of<false>(st, a.nseq, xa);
        uo_a = s.ubase + h - (st.e[ea].ubase + (int)((unsigned)(xa - st.e[ea].base) / (unsigned)st.e[ea].Ia));
        // The unit's parts: one of each CTA that merged its warps (all of whose items are the unit's), else one of each warp.
        const int ca = wa / a.wpc, cb = wb / a.wpc;
        auto merged = [&](int c) {
            return a.wpc > 1 && a.Wb == 0 && ch_range_start(a.W, a.NWp, (long long)c * a.wpc) >= ub &&
                   ch_range_start(a.W, a.NWp, min(a.NWp, (c + 1) * a.wpc)) <= ue;
        };
        if (a.Wb == 0) {
            const bool ma = merged(ca), mb = ca == cb ? ma : merged(cb);
            first = ma ? ca * a.wpc : wa;
            inner = (ca + 1) * a.wpc;
            last = cb * a.wpc;
            if (ma) uo_a = 0;
            n0 = ma ? 1 : min(wb + 1, inner) - wa;
            n01 = n0 + max(0, cb - ca - 1);
            na = n01 + (ca == cb ? 0 : mb ? 1 : wb - last + 1);
        } else {
            first = wa;
            n0 = n01 = na = wb - wa + 1;
        }
        parts = na;
        if (s.Iu > s.Ia) {
            const int Ib = s.Iu - s.Ia;
            const long long b0 = s.base2 + (long long)h * Ib;
            const int r0 = ch_warp_of(a.Wb, a.NQ, b0), r1 = ch_warp_of(a.Wb, a.NQ, b0 + Ib - 1);
            const long long xb = ch_range_start(a.Wb, a.NQ, r0);
            // the unit's place among those of run r0 (entries may have no B items: counted by walking)
            int e = entry_of<true>(st, a.nseq, xb);
            int u0 = (int)((unsigned)(xb - st.e[e].base2) / (unsigned)(st.e[e].Iu - st.e[e].Ia));
            for (uo_b = -u0; e < (int)blockIdx.y; ++e)
                if (st.e[e].Iu > st.e[e].Ia) uo_b += st.e[e].S * a.Hkv;
            uo_b += h;
            qa = (size_t)a.NWp * a.MAXU + (size_t)r0 * a.MAXU2;
            parts = na + r1 - r0 + 1;
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the next call's runs are claimed from the start
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.ctl[2] = 0;
    if (!row) return;
    float M = -CUDART_INF_F, L = 0.0f, acc[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) acc[c] = 0.0f;
    for (int k0 = wi * GRP; k0 < parts; k0 += cw * GRP) {
        float ms[GRP], ls[GRP], vs[GRP][CPL];
#pragma unroll
        for (int x = 0; x < GRP; ++x) {
            ms[x] = -CUDART_INF_F;
            ls[x] = 0.0f;
#pragma unroll
            for (int c = 0; c < CPL; ++c) vs[x][c] = 0.0f;
            const int k = k0 + x;
            if (k < parts) {
                size_t at;
                if (k < na) {
                    const int w = k < n0 ? first + k : k < n01 ? inner + (k - n0) * a.wpc : last + (k - n01);
                    at = (size_t)w * a.MAXU + (k == 0 ? uo_a : 0);
                } else {
                    at = qa + (size_t)(k - na) * a.MAXU2 + (k == na ? uo_b : 0);
                }
                const float *p = a.part + (at * a.RV + col) * (D + 2);
                ms[x] = p[0];
                ls[x] = p[1];
#pragma unroll
                for (int c = 0; c < CPL; c += 2) {
                    const float2 t = *reinterpret_cast<const float2 *>(p + 2 + ch + c);
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
        const float mr = M == -CUDART_INF_F ? 0.0f : M;
        L = 0.0f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc[c] = 0.0f;
        for (int x = 0; x < cw; ++x) {
            const float sx = ch_ex2(red[x][0] - mr);
            L = fmaf(sx, red[x][1], L);
#pragma unroll
            for (int c = 0; c < CPL; ++c) acc[c] = fmaf(sx, red[x][2 + lane * CPL + c], acc[c]);
        }
    }
    // a row sees a token at least, so that L = 0 means scores of -inf or NaN alone: NaN
    const float inv = 1.0f / L;
    __half *o = a.out + (((size_t)(a.B0 + blockIdx.y) * a.Hq + hq) * a.n + tk) * D + ch;
#pragma unroll
    for (int c = 0; c < CPL; c += 2) *reinterpret_cast<__half2 *>(o + c) = __floats2half2_rn(acc[c] * inv, acc[c + 1] * inv);
}

// ---------------------------------------------------------------- selection
// A cluster of up to 16 CTAs per (sequence, kv head) takes the bounds of its
// blocks for every token of the sequence, and then, one token per CTA, the
// selection.
// A slab is 32 BPL blocks' channel ranges in shared memory (16-byte pieces
// turned by the block, so that 8 lanes that read one piece of their own blocks
// meet all banks). A warp takes a (slab, token, four of its heads): BPL blocks
// per lane. max(q lo, q hi) is q hi for positive q, else q lo. Products of two
// fp16 numbers are exact, so a multiply-add of fp16 factors into an fp32 sum
// rounds once, as the sum does: two of them, of (q or 0) lo and (0 or q) hi, and
// the ranges need no conversion. (Conversions, a selection and an fp32
// multiply-add: 131K tokens 22.4 -> 23.6 us in all, drafts of five tokens over
// 512 blocks, seven heads, 30.2 -> 33.5; the half selected by its byte, then
// one multiply-add: 22.6, 31.5.) Where a CTA has no more tasks than warps, a
// warp alone on its scheduler, some 30 cycles per channel, decides; elsewhere
// two blocks per lane share the queries' loads.
constexpr int SEL_THREADS = 512, SEL_BLOCKS = 256, SEL_CLUSTER = 16;   // blocks in shared memory at a time
// Bounds go to the shared memory of the CTA that selects by them where they
// take no more than this (131K tokens 19.5 us in all, by way of L2 20.0; not
// more than the slabs and heads before them: the selection's keys lie there).
constexpr size_t KEPT_BYTES = 16384;

struct SelectArgs {
    const __half2 *dig;
    const int32_t *bt;
    const __half *q;
    float *bound;       // [nseq][n][Hkv][groups][stride]: by four heads; null: the token's CTA has them, behind its heads
    int32_t *sel;       // [B][n][Hkv][Kc]
    int n, B0, Hq, Hkv, g, NB, K, Kc, stride;
    int groups, cluster, slabs;   // (of 32 blocks, even where BPL is 2) groups of four heads per kv head; CTAs per (sequence, kv head), slabs in shared memory at a time
};
struct SelectTable {
    int nb[CHUNK_SEQS], nq[CHUNK_SEQS];
};
template <int D>
__host__ __device__ constexpr int heads_bytes() { return D * 16; }   // four heads per channel
static_assert(KEPT_BYTES <= SEL_THREADS / 32 * heads_bytes<64>(), "keys end before the bounds");

// (q, 0) of a q that is not positive, (0, q) of one that is
__device__ __forceinline__ uint32_t by_sign(__half q) {
    const uint32_t x = __half_as_ushort(q);
    return __hgt(q, __ushort_as_half(0)) ? x << 16 : x;
}
// sum + q.x lo + q.y hi, of which one is 0
__device__ __forceinline__ void add_bound(float &sum, uint32_t q, uint32_t range) {
    asm("{\n .reg .b16 l, h, n, p;\n mov.b32 {l, h}, %1;\n mov.b32 {n, p}, %2;\n fma.rn.f32.f16 %0, n, l, %0;\n"
        " fma.rn.f32.f16 %0, p, h, %0;\n}"
        : "+f"(sum)
        : "r"(range), "r"(q));
}

template <int D, int BPL>
__global__ void __launch_bounds__(SEL_THREADS, 2)
    k_byte_select(const __grid_constant__ SelectArgs a, const __grid_constant__ SelectTable t) {
    constexpr int V4 = D / 4, WARPS = SEL_THREADS / 32, SLAB = 32 * BPL;
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int rank = blockIdx.x % a.cluster, unit = blockIdx.x / a.cluster, e = unit / a.Hkv, hkv = unit % a.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int u = (a.B0 + e) * a.Hkv + hkv, nb = t.nb[e], nq = t.nq[e];
    const int all = (nb + SLAB - 1) / SLAB, per = (all + a.cluster - 1) / a.cluster, s0 = min(all, rank * per),
              s1 = nq > 0 ? min(all, s0 + per) : s0;
    uint4 *const heads = reinterpret_cast<uint4 *>(smem + a.slabs * (32 * D * 4) + warp * heads_bytes<D>());
    float *const kept = reinterpret_cast<float *>(smem + a.slabs * (32 * D * 4) + WARPS * heads_bytes<D>());
    // (the cluster's CTAs run once this barrier is through: bounds may be stored into their shared memory)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool running = false;
    for (int sb = s0; sb < s1; sb += a.slabs / BPL) {
        const int ns = min(a.slabs / BPL, s1 - sb);
        if (sb > s0) __syncthreads();   // the slabs before are read
        for (int z = threadIdx.x; z < ns * SLAB * V4; z += SEL_THREADS) {
            const int x = z / V4, v = z % V4, j = sb * SLAB + x;
            if (j < nb) {
                const size_t own = (size_t)u * a.NB + j, slot = a.bt ? (size_t)a.bt[own] : own;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ch_smem(smem + x * (D * 4) + ((v ^ (x & 7)) << 4))),
                             "l"(a.dig + slot * D + 4 * v)
                             : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (!running) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        running = true;
        for (int task = warp; task < ns * nq * a.groups; task += WARPS) {
            const int x = task % ns, tk = task / ns / a.groups, grp = task / ns % a.groups, j = (sb + x) * SLAB + lane;
            const uint4 *row = reinterpret_cast<const uint4 *>(smem + (x * SLAB + lane) * (D * 4));
            const __half *q = a.q + (((size_t)(a.B0 + e) * a.Hq + hkv * a.g) * a.n + tk) * D;
            __half qv[4][D / 32];   // a short last group repeats its last head
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int y = 0; y < D / 32; ++y) qv[p][y] = q[(size_t)min(4 * grp + p, a.g - 1) * a.n * D + 32 * y + lane];
            __syncwarp();
#pragma unroll
            for (int y = 0; y < D / 32; ++y)
                heads[32 * y + lane] = make_uint4(by_sign(qv[0][y]), by_sign(qv[1][y]), by_sign(qv[2][y]), by_sign(qv[3][y]));
            __syncwarp();
            float sum[BPL][4] = {};
#pragma unroll(4 / BPL)
            for (int c4 = 0; c4 < V4; ++c4) {
                uint32_t w[BPL][4];
#pragma unroll
                for (int o = 0; o < BPL; ++o) {
                    const uint4 d = row[o * (32 * V4) + (c4 ^ (lane & 7))];
                    w[o][0] = d.x; w[o][1] = d.y; w[o][2] = d.z; w[o][3] = d.w;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint4 q4 = heads[4 * c4 + y];
                    const uint32_t qs[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int o = 0; o < BPL; ++o)
#pragma unroll
                        for (int p = 0; p < 4; ++p) add_bound(sum[o][p], qs[p], w[o][y]);
                }
            }
            float *to;
            if (a.bound) to = a.bound + ((((size_t)e * a.n + tk) * a.Hkv + hkv) * a.groups + grp) * a.stride;
            else to = of_rank(kept + (tk / a.cluster * a.groups + grp) * a.stride, tk % a.cluster);
#pragma unroll
            for (int o = 0; o < BPL; ++o) {
                float best = -CUDART_INF_F;
#pragma unroll
                for (int p = 0; p < 4; ++p) best = sum[o][p] > best ? sum[o][p] : best;
                if (j + 32 * o < nb) to[j + 32 * o] = best;
            }
        }
    }
    if (!running) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // every CTA of the cluster comes by here; the bounds are visible to all of them behind it
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int tk = rank; tk < nq; tk += a.cluster) {
        const size_t at = ((size_t)e * a.n + tk) * a.Hkv + hkv;
        pick_blocks(a.bound ? a.bound + at * a.groups * a.stride : kept + tk / a.cluster * a.groups * a.stride, a.groups, a.stride, nb, a.K, a.Kc, a.sel + ((size_t)a.B0 * a.n * a.Hkv + at) * a.Kc,
                    reinterpret_cast<uint32_t *>(smem));
        __syncthreads();
    }
}

// ---------------------------------------------------------------- plans
struct Plan {
    ByteArgs a;
    ByteTable st;
    SelectArgs ba;
    SelectTable bt;
    bool any, pick;
    bool two;      // bounds: two blocks per lane
    int NC;        // groups of 8 rows; 0: tiles
    int ctas;
    int nC;        // tiles: CTAs
    bool whole;    // ... each with a tile of its own
    size_t part_floats, bound_floats;
    int cw, nbmax;
    size_t kept;   // bytes of bounds that a CTA which selects keeps
};

// Kc: slots of a list of selected blocks. false: sizes beyond the kernels' 32-bit counters.
bool make_plan(const ott_byte_cache *c, const ByteCall &call, int B0, int Kc, Plan &p) {
    ByteArgs &a = p.a;
    a.blk = c->blk;
    a.rec = c->rec;
    a.bt = c->paged ? c->bt : nullptr;
    a.tk = c->tk;
    a.tv = c->tv;
    a.q = call.q;
    a.k = call.k;
    a.v = call.v;
    a.out = call.out;
    a.ctl = c->ctl;
    a.sel = nullptr;
    a.blk_bytes = c->blk_bytes;
    a.n = call.n;
    a.B0 = B0;
    a.nseq = std::min(c->B - B0, CHUNK_SEQS);
    a.Hq = c->Hq;
    a.Hkv = c->Hkv;
    a.g = c->g;
    a.NB = c->NB;
    a.G = c->G;
    a.Kc = Kc;
    a.IPB = c->G / QT;
    a.sl2 = (float)(1.4426950408889634 / std::sqrt((double)c->d));
    int nq_max = 0;
    p.nbmax = 0;
    for (int x = 0; x < a.nseq; ++x) {
        ByteSeq &s = p.st.e[x];
        const int T = c->T[B0 + x], nq = call.lens ? call.lens[B0 + x] : call.n;
        s.T = T;
        s.nq = nq;
        s.nb = call.topk > 0 ? std::min(call.topk, T / c->G) : T / c->G;
        s.Ft = (T % c->G + FT - 1) / FT;
        s.Sf = s.Ft + (call.k ? (nq + FT - 1) / FT : 0);
        nq_max = std::max(nq_max, nq);
        if (nq > 0) p.nbmax = std::max(p.nbmax, T / c->G);
        p.bt.nb[x] = T / c->G;
        p.bt.nq[x] = nq;
    }
    p.any = nq_max > 0;
    p.pick = call.topk > 0;
    p.part_floats = p.bound_floats = 0;
    p.NC = 0;
    if (!p.any) return true;
    const bool pick = p.pick;
    const long long rows = pick ? c->g : (long long)nq_max * c->g;
    if (!pick && rows > ROWS_MAX) return plan_byte_tiles(c, a, p.st, p.nC, p.whole, p.part_floats);
    p.NC = rows <= 8 ? 1 : 2;
    a.RB = 8 * p.NC;
    a.SG = pick ? (c->g + a.RB - 1) / a.RB : 1;
    a.RV = (int)std::min<long long>(rows, a.RB);
    constexpr int WARPS = 8;
    long long W = 0, units = 0, longest = 0;
    for (int x = 0; x < a.nseq; ++x) {
        ByteSeq &s = p.st.e[x];
        s.ubase = (int)units;
        const long long S = s.nq == 0 ? 0 : pick ? (long long)s.nq * a.SG : ((long long)s.nq * c->g + a.RB - 1) / a.RB;
        const long long Iu = s.Sf + (long long)s.nb * a.IPB;
        if (S * c->Hkv * Iu > INT_MAX || units + S * c->Hkv > INT_MAX) return false;
        s.S = (int)S;
        s.Iu = s.Ia = (int)Iu;
        if (S > 0) longest = std::max(longest, Iu);
        W += S * c->Hkv * Iu;
        units += S * c->Hkv;
    }
    // A items in equal runs, at least two items each, sums ending after SUM_TOKENS tokens. An eighth of the units
    // as B items where a warp has 64 items or more and a unit 16 runs at most; elsewhere their partials cost more
    // than they even out. Without and with them: batch 32 x 4K, 32 heads (108 items a warp, 1.2 runs a unit) 166
    // and 161 us, four queries each 182 and 165; batch 16 x 32K, 8 kv heads (9.5 runs) 164 and 162; 4 x 131K (38
    // runs) 161 and 163; 600K tokens, 8 kv heads (152 runs) 183 and 193; 131K (27 items a warp) 46 and 51 to 60.
    int ctas = c->sm_count;
    while (ctas < (1 << 20) && W / ((long long)ctas * WARPS) >= SUM_TOKENS / QT) ctas += c->sm_count;
    a.NWp = (int)std::max<long long>(1, std::min<long long>((long long)ctas * WARPS, W / 2));
    const bool claims = W / a.NWp >= 64 && longest * a.NWp / W <= 16;
    long long base = 0, base2 = 0, ia_min = LLONG_MAX, ib_min = LLONG_MAX;
    for (int x = 0; x < a.nseq; ++x) {
        ByteSeq &s = p.st.e[x];
        if (claims) s.Ia = s.Iu - s.Iu / 8;
        s.base = base;
        s.base2 = base2;
        base += (long long)s.S * c->Hkv * s.Ia;
        base2 += (long long)s.S * c->Hkv * (s.Iu - s.Ia);
        if (s.S == 0) continue;
        ia_min = std::min<long long>(ia_min, s.Ia);
        if (s.Iu > s.Ia) ib_min = std::min<long long>(ib_min, s.Iu - s.Ia);
    }
    p.st.e[a.nseq] = ByteSeq{};
    p.st.e[a.nseq].base = a.W = base;
    p.st.e[a.nseq].base2 = a.Wb = base2;
    p.st.e[a.nseq].ubase = (int)units;
    p.ctas = (int)std::min<long long>(ctas, a.NWp);
    a.wpc = (a.NWp + p.ctas - 1) / p.ctas;
    p.ctas = (a.NWp + a.wpc - 1) / a.wpc;
    a.direct = false;
    a.cluster = 1;
    int fits = 0;
    while (fits < 4 && longest > (long long)SPREAD_ITEMS * a.cluster && units <= c->rows_clusters[fits]) {
        a.cluster *= 2;
        ++fits;
    }
    if (units <= c->sm_count && longest <= (long long)DIRECT_ITEMS * a.cluster) {
        a.direct = true;
        a.wpc = (int)std::min<long long>(WARPS, (longest + a.cluster - 1) / a.cluster);
        p.ctas = (int)units * a.cluster;
        a.NWp = p.ctas * a.wpc;
    }
    const long long run = (base + a.NWp - 1) / a.NWp;
    a.MAXU = (int)std::min<long long>((run - 1) / ia_min + 2, run);
    a.NQ = 0;
    a.MAXU2 = 0;
    if (base2 > 0) {
        a.NQ = (int)std::max<long long>(1, std::min<long long>(base2 / 4, 3LL * a.NWp));
        const long long run2 = (base2 + a.NQ - 1) / a.NQ;
        a.MAXU2 = (int)std::min<long long>((run2 - 1) / ib_min + 2, run2);
    }
    const long long places = a.direct ? 0 : (long long)a.NWp * a.MAXU + (long long)a.NQ * a.MAXU2;
    if (places > INT_MAX) return false;
    p.part_floats = (size_t)places * a.RV * (c->d + 2);
    // merge: warps per row by the partials of a unit
    const long long all = W, parts = (base2 > 0 ? longest * a.NWp / all + longest * a.NQ / all : longest * a.NWp / all / a.wpc + 2 * a.wpc) + 2;
    p.cw = (int)std::min<long long>(CMB_MAXW, (parts + 7) / 8);
    if (pick) {
        // CTAs per (sequence, kv head): as many as give every SM one, but a slab each (two each: five drafts 38 -> 43 us)
        const int slabs = std::max(1, (p.nbmax + 31) / 32);
        int cluster = 1;
        while (cluster < c->max_cluster && 2 * cluster <= slabs && (long long)a.nseq * c->Hkv * cluster < c->sm_count)
            cluster *= 2;
        const int groups = (c->g + 3) / 4, own = (slabs + cluster - 1) / cluster;   // slabs of a CTA
        p.two = (long long)own * nq_max * groups > SEL_THREADS / 32;
        p.ba = {c->dig, a.bt, call.q, nullptr, nullptr, call.n, B0, c->Hq, c->Hkv, c->g, c->NB, call.topk, Kc, p.nbmax,
                groups, cluster, std::min(SEL_BLOCKS / 32, p.two ? (own + 1) / 2 * 2 : own)};
        p.kept = (size_t)((nq_max + cluster - 1) / cluster) * groups * p.nbmax * 4;
        if (p.kept > KEPT_BYTES) {
            p.kept = 0;
            p.bound_floats = (size_t)a.nseq * call.n * c->Hkv * groups * p.nbmax;
        }
    }
    return true;
}

template <int D, int NC, int FMT>
cudaError_t launch_rows(const Plan &p, cudaStream_t s) {
    using C = RowsCfg<D, NC>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3((unsigned)p.a.wpc * 32);
    cfg.dynamicSmemBytes = (size_t)C::WARP_SMEM * p.a.wpc;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.a.direct && p.a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_byte_rows<D, NC, FMT>, p.a, p.st);
}

template <int D>
int select_smem(int slabs, int nb, int kept) {
    return std::max(slabs * (32 * D * 4) + SEL_THREADS / 32 * heads_bytes<D>() + kept, (nb + 3) / 4 * 16);
}

template <int D>
cudaError_t launch_select(const ott_byte_cache *c, const Plan &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.a.nseq * c->Hkv * p.ba.cluster));
    cfg.blockDim = dim3(SEL_THREADS);
    cfg.dynamicSmemBytes = (size_t)select_smem<D>(p.ba.slabs, p.nbmax, (int)p.kept);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.ba.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, p.two ? k_byte_select<D, 2> : k_byte_select<D, 1>, p.ba, p.bt);
}

template <int D>
cudaError_t launch_plan(const ott_byte_cache *c, const Plan &p, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (p.NC == 0) return launch_byte_tiles(c, p.a, p.st, p.nC, p.whole, s);
    if (p.pick) e = launch_select<D>(c, p, s);
    const bool i8 = c->format == OTT_BYTE_INT;
    if (e == cudaSuccess)
        e = p.NC == 1 ? (i8 ? launch_rows<D, 1, OTT_BYTE_INT>(p, s) : launch_rows<D, 1, OTT_BYTE_FLOAT>(p, s))
                      : (i8 ? launch_rows<D, 2, OTT_BYTE_INT>(p, s) : launch_rows<D, 2, OTT_BYTE_FLOAT>(p, s));
    if (e == cudaSuccess && !p.a.direct)
        e = launch_pdl(k_byte_combine<D>, dim3((unsigned)(c->Hq * p.a.n), (unsigned)p.a.nseq), 32 * p.cw, 0, s, p.a, p.st);
    return e;
}

// clusters: how many of 2, 4, 8 and 16 CTAs run at a time (the least of the instances asked so far)
template <int D, int NC, int FMT>
cudaError_t rows_attribute(int (&clusters)[4]) {
    using C = RowsCfg<D, NC>;
    auto *kern = k_byte_rows<D, NC, FMT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::WARP_SMEM * C::WARPS);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int x = 0; x < 4 && e == cudaSuccess; ++x) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2u << x);
        cfg.blockDim = dim3(C::WARPS * 32);
        cfg.dynamicSmemBytes = (size_t)C::WARP_SMEM * C::WARPS;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2u << x;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            fit = 0;
        }
        clusters[x] = std::min(clusters[x], fit);
    }
    return e;
}
template <int D>
cudaError_t set_attributes(ott_byte_cache *c) {
    for (int &x : c->rows_clusters) x = INT_MAX;
    const bool i8 = c->format == OTT_BYTE_INT;
    const cudaError_t e = i8 ? rows_attribute<D, 1, OTT_BYTE_INT>(c->rows_clusters) : rows_attribute<D, 1, OTT_BYTE_FLOAT>(c->rows_clusters);
    if (e != cudaSuccess) return e;
    return i8 ? rows_attribute<D, 2, OTT_BYTE_INT>(c->rows_clusters) : rows_attribute<D, 2, OTT_BYTE_FLOAT>(c->rows_clusters);
}

// shared memory of the selection that a launch may ask for
int pick_smem(const ott_byte_cache *c) { return c->smem_optin - 2048; }

}  // namespace

cudaError_t set_byte_attributes(ott_byte_cache *c) {
    cudaError_t e = c->d == 128 ? set_attributes<128>(c) : set_attributes<64>(c);
    // clusters of 16 CTAs where this GPU has room for them, else of 8
    c->max_cluster = SEL_CLUSTER;
    for (int two = 0; two < 2 && e == cudaSuccess; ++two) {
        auto *select = c->d == 128 ? (two ? k_byte_select<128, 2> : k_byte_select<128, 1>)
                                   : (two ? k_byte_select<64, 2> : k_byte_select<64, 1>);
        e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, pick_smem(c));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(SEL_CLUSTER);
        cfg.blockDim = dim3(SEL_THREADS);
        cfg.dynamicSmemBytes = (size_t)pick_smem(c);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = SEL_CLUSTER;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (cudaOccupancyMaxActiveClusters(&fit, select, &cfg) != cudaSuccess || fit < 1) {
            cudaGetLastError();
            c->max_cluster = 8;
        }
    }
    return e == cudaSuccess ? set_byte_tiles_attributes(c->d, c->format) : e;
}

// err: the CUDA error behind OTT_ERR_CUDA.
int run_byte_attn(const ott_byte_cache *c, const ByteCall &call, cudaStream_t s, cudaError_t &err) {
    err = cudaSuccess;
    int nb_all = 0;   // the most blocks of any sequence: the width of the lists that a caller gets
    for (int b = 0; b < c->B; ++b) nb_all = std::max(nb_all, c->T[b] / c->G);
    const int Kc = std::min(call.topk, nb_all);
    if (Kc > 0 && ((long long)nb_all + 3) / 4 * 16 > pick_smem(c)) return OTT_ERR_INVALID;
    // With nothing to select, the call is the one over every block.
    ByteCall cl = call;
    if (Kc == 0) cl.topk = 0;
    if ((long long)c->Hq * cl.n > INT_MAX || (cl.topk > 0 && (long long)CHUNK_SEQS * c->Hkv * SEL_CLUSTER > INT_MAX))
        return OTT_ERR_INVALID;
    const int passes = (c->B + CHUNK_SEQS - 1) / CHUNK_SEQS;
    size_t floats = 0, parts = 0, bounds = 0;
    auto plan = [&](int x, Plan &p) { return make_plan(c, cl, x * CHUNK_SEQS, Kc, p); };
    Plan p;
    for (int x = 0; x < passes; ++x) {   // every pass is checked before the first is queued
        if (!plan(x, p)) return OTT_ERR_INVALID;
        parts = std::max(parts, p.part_floats);
        bounds = std::max(bounds, p.bound_floats);
    }
    const size_t lists = cl.topk > 0 && !cl.sel ? (size_t)c->U * cl.n * Kc : 0;
    parts = (parts + 63) / 64 * 64;
    bounds = (bounds + 63) / 64 * 64;
    floats = parts + bounds + lists;
    Scratch scratch(c->part, c->part_floats, c->device, floats, s);
    if (!scratch.ptr) return OTT_ERR_OOM;
    float *base = static_cast<float *>(scratch.ptr);
    for (int x = 0; x < passes && err == cudaSuccess; ++x) {
        if (passes > 1) plan(x, p);
        if (!p.any) continue;
        p.a.part = base;
        if (cl.topk > 0) {
            p.ba.bound = p.bound_floats ? base + parts : nullptr;
            p.ba.sel = cl.sel ? cl.sel : reinterpret_cast<int32_t *>(base + parts + bounds);
            p.a.sel = p.ba.sel;
        }
        err = c->d == 128 ? launch_plan<128>(c, p, s) : launch_plan<64>(c, p, s);
    }
    const cudaError_t e2 = scratch.release();
    if (err == cudaSuccess) err = e2;
    return err == cudaSuccess ? OTT_OK : OTT_ERR_CUDA;
}

}  // namespace ott
