// ott_byte.cuh -- the cache held in 8 bits (ott_byte_*): device layout, and the
// interface of its translation units (ott_byte.cu: the calls, writing and
// reading back; ott_byte_rows.cu: attention of few rows, selection of blocks;
// ott_byte_tiles.cu: attention of many rows).
//
// One unit = one (sequence, kv head). Block j of a unit holds tokens j G ..
// j G + G - 1, in slot u * NB + j of the pool, or in slot bt[u][j] of a paged one:
//
//   blk + slot * 2 G d: G / 16 groups of 16 tokens, 32 d bytes each
//     [0, 16 d)     keys' codes:   pieces of 16 bytes at (p * 32 + lane) * 16
//     [16 d, 32 d)  values' codes: the same
//   rec[slot]: what a block's codes mean (ByteRec)
//   dig[slot][d]: smallest and largest key of each channel, fp16, as written
//
// A code is one byte: int8 biased by 128 (so that OR-ing it into the mantissa
// of fp16 1024 and subtracting 1152 gives the number), or e4m3. Both are exact
// in fp16. Pieces are what a lane = 4 r + i of an mma.sync m16n8k16 fragment takes:
//
//   keys, piece p = pp + (d/64) * th: token r + 8 th, byte y: channel
//     (d/4) i + 16 pp + (y ^ rot), rot = 8 for lanes i >= 2 of d = 128, else 0
//     (so that 16-byte stores of the dequantized halves meet all banks);
//   values, piece c: byte 4 w + y: channel 32 c + r + 8 w, token 2 i + {0, 1, 8, 9}[y].
//
// The open block: tk, tv [U][G][d] fp16, token t at row t mod G.
//
// Every kernel starts while the one before it on the stream may still write
// what it will read (programmatic dependent launches): codes, records, block
// table, selections, queries that are another call's output. All of that is
// read by plain loads behind griddepcontrol.wait; a load by way of the
// read-only path (__ldg) is defined only for data that nobody writes while the
// kernel runs, and does not have to stay behind the wait.
#pragma once

#include "ott_chunk.cuh"

// Scales of a block's keys and values (fp32, code * scale), log2 and
// reciprocal of the values' (0 where all values are 0: then 2^-40 and 2^40,
// which multiply codes that are 0).
struct alignas(16) ByteRec {
    float ks, vs, lv, iv;
};

struct ott_byte_cache {
    int B, Hq, Hkv, d, G, format, max_tokens;
    int U, g, NB;
    long long blk_bytes;
    int poisoned, device, sm_count, smem_optin;
    int max_cluster;    // CTAs of a cluster that selects blocks
    int rows_clusters[4];   // clusters of 2, 4, 8, 16 CTAs of the rows kernel that run at a time
    void *mem;
    size_t mem_bytes;
    uint8_t *blk;
    ByteRec *rec;
    __half2 *dig;
    __half *tk, *tv;
    int paged;
    long long pool_blocks, free_blocks;
    int32_t *bt;        // [U][NB]
    int32_t *fstack;    // [pool_blocks] free slots, free_blocks of them (the host counts)
    float *part;        // partial results, bounds and selections of a call
    size_t part_floats;
    int *ctl;           // [1]: a bounded wait gave up; [2]: runs of B items claimed (0 between calls)
    std::vector<int> T;
};

namespace ott {

constexpr int BYTE_MAX_SEQS = RAGGED_MAX;

// Attention call: k null: one query per sequence at its last token.
struct ByteCall {
    const __half *q, *k, *v;
    __half *out;
    int n;             // rows of room per sequence
    const int *lens;   // null: n each
    int topk;          // 0: every block
    int32_t *sel;      // [B][n][Hkv][Kc] or null
};
int run_byte_attn(const ott_byte_cache *c, const ByteCall &call, cudaStream_t s, cudaError_t &err);
cudaError_t set_byte_attributes(ott_byte_cache *c);

// One sequence of an attention launch.
struct ByteSeq {
    long long base, base2;   // first work item (A, B); entry [nseq] holds the totals
    int ubase;         // first work unit
    int S;             // slices of query rows per kv head, or pairs of tiles (0: no queries)
    int T, nq;         // tokens in the cache, query tokens
    int nb;            // blocks that a query attends
    int Ft, Sf;        // work items of the open block; and with the new tokens'
    int Iu, Ia;        // work items of a unit, the A items among them
};
struct ByteTable {
    ByteSeq e[CHUNK_SEQS + 1];
};
struct ByteArgs {
    const uint8_t *blk;
    const ByteRec *rec;
    const int32_t *bt;         // null: slot u * NB + j
    const __half *tk, *tv;
    const __half *q, *k, *v;   // [B][Hq][n][d], [B][Hkv][n][d]
    __half *out;
    float *part;
    int *ctl;
    const int32_t *sel;        // [B][n][Hkv][Kc]; null: every block
    long long blk_bytes;
    int n, B0, nseq, Hq, Hkv, g, NB, G, Kc;
    int IPB;                   // work items per block
    int SG;                    // selected blocks: slices of heads per token
    int RB;                    // rows per slice
    long long W, Wb;           // work items: A, B
    int NWp, wpc, MAXU, RV;    // active warps, warps per CTA, units that a warp's run of A items can touch, rows of a partial
    int NQ, MAXU2;             // runs of B items, units that one can touch
    bool direct;               // a CTA or a cluster of them per unit, which writes its rows
    int cluster;               // ... its CTAs
    float sl2;                 // log2(e) / sqrt(d)
};

// ott_byte_tiles.cu
bool plan_byte_tiles(const ott_byte_cache *c, ByteArgs &a, ByteTable &st, int &nC, bool &whole, size_t &part_floats);
cudaError_t launch_byte_tiles(const ott_byte_cache *c, const ByteArgs &a, const ByteTable &st, int nC, bool whole,
                              cudaStream_t s);
cudaError_t set_byte_tiles_attributes(int d, int format);

// Two or four codes -> fp16x2, exactly.
template <int FMT>
__device__ __forceinline__ void byte_unpack(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == OTT_BYTE_INT) {
        const __half2 off = __float2half2_rn(-1152.0f);
        lo = ch_h2(__hadd2(ch_as_h2(__byte_perm(w, 0x64646464u, 0x4140)), off));
        hi = ch_h2(__hadd2(ch_as_h2(__byte_perm(w, 0x64646464u, 0x4342)), off));
    } else {
        asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

}  // namespace ott
