// Decode attention over the quantised paged cache (layout: quant_format.h), one kernel per call.
//
// With K[j] = kmin_j + ks_j * a_j and V[j] = vmin_j + vs_j * c_j (codes a, c; parameters per row and
// group of elements), the scores and the output of one query row are
//     x_j = scale * sum_groups ( ks_j (q . a_j) + kmin_j * sum(q) )
//     out = ( sum_j (p_j vs_j) c_j + sum_j p_j vmin_j ) / sum_j p_j,      p_j = exp(x_j - max x)
// so the matrix products run on the codes themselves and every parameter is applied to a score or
// a weight in fp32: nothing is dequantised.  A code becomes an fp16 operand by masking alone: the
// bits of code c in the low bits of an fp16 are the subnormal c * 2^-24 (bits 4..7: c * 2^-20), and
// the tensor core multiplies subnormals exactly; the powers of two are divided out in fp32.
// Q is brought to fp16 exactly by a power of two per query row (bf16 has 8 significant bits, fp16
// 11; what lies 2^-24 or more below the row's largest element loses bits).
//
// The weights p_j vs_j are rounded to fp16 (2^-11 relative) for the product with the V codes.  They
// are kept near 1 by a reference of their own: m is the reference of the softmax, M that of
// x_j + log2 vs_j, and f = 2^(m - M).  Both are raised only when a weight passes 2^8, so the usual
// tile has no cross-lane maximum at all; sums stay in fp32 and are exact in the reference.
//
// Work.  A unit is one sequence and kh adjacent KV heads; a stage is kTileRows-row tiles of every
// one of those heads.  The stages of all units are laid end to end and CTA c of a persistent grid
// (one per SM) takes an equal contiguous range; its piece of a unit is a segment.  A page of kh
// heads is contiguous (codes and parameters), so a stage is a few bulk copies.  One warp copies
// into a ring of stages, the others each take 16-row tiles of one KV head: S^T = K Q^T and
// O^T += V^T P^T on mma.m16n8k16 with the keys (then the elements of V) on M and the query columns
// on N, and own running state per warp, merged once per segment.
//
// A segment that covers its unit writes the output; any other writes its normalised partial rows
// and log2-sum-exps, and the CTA that completes the unit (an acquire-release counter) merges them
// in segment order, so the result depends on no timing.  Every wait is bounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "launch.h"
#include "ptx.cuh"
#include "quant_format.h"

namespace da {

struct QuantParams {
    const __nv_bfloat16* q;      // [B, Hq, sq, D]
    __nv_bfloat16* out;
    const unsigned char* pool;   // [num_pages, Hkv, page_size * row bytes]
    const int* block_table;
    const unsigned* kv_lens;
    int kv_stride, max_pages, page_size, num_pages;
    int B, Hq, Hkv;
    int cols;                    // query columns of one KV head: Hq / Hkv * sq
    int sq, causal;
    int kh;                      // KV heads per unit, a power of two
    int slices_shift;            // log2 of the warps that split a head's columns
    float scale_log2;
    unsigned* counters;          // one per unit, zero between calls
    float* part_lse;             // [segments, kh * cols]
    float* part_o;               // [segments, kh * cols, D]
    unsigned* err;
};

template <int D_, int BITS_, int NG_, int NC_>
struct QuantGeometry {
    static constexpr int D = D_, BITS = BITS_, NG = NG_, NC = NC_;
    static constexpr int RB = kQuantRowCodes(D, BITS);
    static constexpr int PB = kQuantRowParams(D, D / NG);
    static constexpr int ROW = 2 * RB + PB;
    static constexpr int NT = NC / 8;                      // 8-column n-tiles of a warp
    static constexpr int W = 8;                             // consumer warps
    static constexpr int kConsumers = 32 * W;
    static constexpr int kThreads = kConsumers + 32;       // and one copying warp
    static constexpr int kTiles = (D == 128 && BITS == 8) ? 8 : 16;   // 16-row tiles of a stage
    static constexpr int kStageRows = kTiles * 16;
    static constexpr int kStageBytes = kStageRows * ROW;
    static constexpr int kMergeStride = D + 4;             // floats of a merge row
    static constexpr int kMergeFloats = 8 * 8 * kMergeStride + 2 * 8 * 8;
    static constexpr int kMiscBytes = 512;
    static constexpr int kSchedBytes = (2 * kMaxPagedBatch + 2) * 4;
    static constexpr int kFixedBytes = kMergeFloats * 4 + kMiscBytes + kSchedBytes;
    static constexpr int kStagesFit = (kSmemBudget - 128 - kFixedBytes) / kStageBytes;
    static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
    static constexpr int kSmemBytes = 128 + kStages * kStageBytes + kFixedBytes;
    static_assert(kStages >= 2 && kStageBytes % 128 == 0 && kTiles >= W, "ring");
};

struct QuantSmem {
    unsigned char* stages;
    float* merge_o;      // [8 warps][8 columns][kMergeStride]
    float* merge_m;      // [8][8]
    float* merge_l;      // [8][8]
    uint64_t* full;
    uint64_t* empty;
    uint64_t* group;
    unsigned* stage_len;     // rows per head of the stage that lie inside the sequence
    unsigned* stage_pages;   // bit i: page i of the stage was copied
    volatile int* abort;
    int* last_flag;
    int* seq_prefix;     // [B + 1] exclusive prefix of the sequences' stages
    int* seq_len;        // [B]
};

template <class Gm>
__device__ __forceinline__ QuantSmem quant_carve(unsigned char* raw) {
    QuantSmem s;
    unsigned char* base = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    s.stages = base;
    unsigned char* p = base + Gm::kStages * Gm::kStageBytes;
    s.full = reinterpret_cast<uint64_t*>(p);
    s.empty = s.full + 8;
    s.group = s.empty + 8;
    s.stage_len = reinterpret_cast<unsigned*>(s.group + 1);
    s.stage_pages = s.stage_len + 8;
    s.abort = reinterpret_cast<volatile int*>(s.stage_pages + 8);
    s.last_flag = const_cast<int*>(s.abort) + 1;
    p += Gm::kMiscBytes;
    s.merge_o = reinterpret_cast<float*>(p);
    s.merge_m = s.merge_o + 8 * 8 * Gm::kMergeStride;
    s.merge_l = s.merge_m + 64;
    s.seq_prefix = reinterpret_cast<int*>(s.merge_l + 64);
    s.seq_len = s.seq_prefix + kMaxPagedBatch + 1;
    return s;
}

struct QuantUnit {
    int b, g, u;     // sequence, group of kh KV heads, unit index
    int len, nt;     // live rows, stages
    int base;        // global index of the first stage
};

__device__ __forceinline__ QuantUnit quant_locate(const QuantParams& p, const QuantSmem& sm, int t) {
    const int upb = p.Hkv / p.kh;
    int lo = 0, hi = p.B - 1;            // largest b with seq_prefix[b] * upb <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm.seq_prefix[mid] * upb <= t) lo = mid; else hi = mid - 1;
    }
    QuantUnit U;
    U.b = lo;
    U.nt = sm.seq_prefix[lo + 1] - sm.seq_prefix[lo];
    const int r = t - sm.seq_prefix[lo] * upb;
    U.g = r / U.nt;
    U.u = lo * upb + U.g;
    U.len = sm.seq_len[lo];
    U.base = sm.seq_prefix[lo] * upb + U.g * U.nt;
    return U;
}

__device__ __forceinline__ bool quant_sync(const QuantSmem& sm, uint32_t& phase, unsigned* err) {
    mbar_arrive(sm.group);
    const bool ok = mbar_wait_warp(sm.group, phase, sm.abort);
    phase ^= 1u;
    if (!ok) {
        *sm.abort = 1;
        record_error(err, kErrWaitGroup);
    }
    return ok;
}

// D(16x8, f32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// N consecutive words of shared memory at `addr` (aligned to their size, at most 16 bytes a load)
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&r)[N]) {
    if constexpr (N == 1) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
                         : "r"(addr + 4 * i));
    }
}

// Row of a 16-row tile (0..7; +8 for the second half) that stands at fragment row i: neighbouring
// fragment rows lie in rows of unlike parity (the K loads of a quarter warp then cover all banks at
// 64 bytes a row) and the rows 2 t, t = 0..3, are the first four (two of each parity for the V loads).
__device__ __forceinline__ int quant_tile_row(int i) { return ((i >> 1) ^ (i & 1)) | ((i & 1) << 2); }

constexpr float kQuantUnset = -3.402823466e38f;   // reference of a column that has seen no row

template <class Gm>
struct QuantWarp {
    static constexpr int D = Gm::D, BITS = Gm::BITS, NG = Gm::NG, NT = Gm::NT;
    static constexpr int S = D / 16;             // 16-element slices: MMA k-steps of a K row, m-tiles of V
    static constexpr int KW = Gm::RB / 16;       // words of a K row per lane
    static constexpr int VW = Gm::RB / 32;       // words of a V row per lane
    static constexpr int PW = 2 * NG;            // parameter words of a row
    // powers of two of the code operands: 2^-24, and 2^-20 for the upper codes of the 4-bit pairs
    static constexpr float kUnit = 16777216.f;
    static constexpr float kUnitHi = BITS == 4 ? 1048576.f : 16777216.f;

    int lane, gq, qd;                // fragment row, quad lane
    int head, col0;                  // KV head of the unit, first query column
    uint32_t qf[S][NT][2];           // Q^T fragments (fp16, scaled by a power of two per column)
    float qsum[NG][NT][2];           // sum of a column's scaled elements per group, in code units
    float cf[NT][2];                 // score units -> log2 domain
    float o[S][NT][4];               // O^T: rows gq (element 16 m + 2 gq) and gq + 8 (element + 1)
    float z[NG][NT][2];              // this lane's share of sum p * vmin
    float l[NT][2];                  // this lane's share of sum p
    float m[NT][2], M[NT][2], f[NT][2];
    int tok[NT][2];                  // query token of the column (causal)
    uint32_t koff[2], voff[4], poff[2];   // lane offsets inside a tile: K rows, V rows, parameters

    __device__ __forceinline__ void init(int lane_, int head_, int col0_, int sq, int half_k,
                                         int half_p) {
        lane = lane_;
        gq = lane >> 2;
        qd = lane & 3;
        head = head_;
        col0 = col0_;
        const int r = quant_tile_row(gq);
        const int ra = quant_tile_row(2 * qd), rb = quant_tile_row(2 * qd + 1);
        koff[0] = r * Gm::RB + qd * (4 * KW);
        koff[1] = koff[0] + half_k;
        voff[0] = ra * Gm::RB + gq * (4 * VW);
        voff[1] = rb * Gm::RB + gq * (4 * VW);
        voff[2] = voff[0] + half_k;
        voff[3] = voff[1] + half_k;
        poff[0] = r * Gm::PB;
        poff[1] = poff[0] + half_p;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) tok[nt][e] = (col0 + nt * 8 + 2 * qd + e) % sq;
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nt][e] = 0.f;
                m[nt][e] = M[nt][e] = kQuantUnset;
                f[nt][e] = 1.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) z[g][nt][e] = 0.f;
            }
    }

    // Query rows row0 .. row0 + cols - 1 (columns at or past cols are zero)
    __device__ __forceinline__ void load_q(const QuantParams& p, size_t row0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = col0 + nt * 8 + gq;
            const bool ok = c < p.cols;
            const uint2* row = reinterpret_cast<const uint2*>(p.q + (row0 + (ok ? c : 0)) * D);
            uint2 raw[S];                 // elements 16 s + 4 qd .. + 3
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                raw[s] = ok ? __ldg(row + 4 * s + qd) : make_uint2(0u, 0u);
                top = max(top, max((raw[s].x << 16) & 0x7fffffffu, raw[s].x & 0x7fff0000u));
                top = max(top, max((raw[s].y << 16) & 0x7fffffffu, raw[s].y & 0x7fff0000u));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest element goes to [2^14, 2^15)
            const int ex = min(max(static_cast<int>(top >> 23), 27), 254);
            const float up = __int_as_float((268 - ex) << 23);
            const float down = __int_as_float((ex - 14) << 23);
            float gs[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) gs[g] = 0.f;
            float v[S][4];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                v[s][0] = bf16_lo_to_f32(raw[s].x) * up;
                v[s][1] = bf16_hi_to_f32(raw[s].x) * up;
                v[s][2] = bf16_lo_to_f32(raw[s].y) * up;
                v[s][3] = bf16_hi_to_f32(raw[s].y) * up;
                gs[s * NG / S] += (v[s][0] + v[s][1]) + (v[s][2] + v[s][3]);
            }
            if (BITS == 8) {
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    qf[s][nt][0] = pack_f16x2(v[s][0], v[s][1]);
                    qf[s][nt][1] = pack_f16x2(v[s][2], v[s][3]);
                }
            } else {
                // a word holds two slices; its masked pairs are codes i and i + 4, at 2^-24 for
                // i = 0, 2 and at 2^-20 for i = 1, 3
#pragma unroll
                for (int w = 0; w < S / 2; ++w) {
                    qf[2 * w][nt][0] = pack_f16x2(v[2 * w][0], v[2 * w + 1][0]);
                    qf[2 * w][nt][1] = pack_f16x2(v[2 * w][2], v[2 * w + 1][2]);
                    qf[2 * w + 1][nt][0] = pack_f16x2(v[2 * w][1] * 0.0625f, v[2 * w + 1][1] * 0.0625f);
                    qf[2 * w + 1][nt][1] = pack_f16x2(v[2 * w][3] * 0.0625f, v[2 * w + 1][3] * 0.0625f);
                }
            }
            // to the score fragment's columns 2 qd, 2 qd + 1 (held here by the quads of those rows)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float x = gs[g];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x *= 1.f / kUnit;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qsum[g][nt][e] = __shfl_sync(0xffffffffu, x, (2 * qd + e) * 4);
            }
            const float c2 = p.scale_log2 * down * kUnit;
#pragma unroll
            for (int e = 0; e < 2; ++e) cf[nt][e] = __shfl_sync(0xffffffffu, c2, (2 * qd + e) * 4);
        }
    }

    // Raises the references to the maxima of this tile (and of all tiles before).
    __device__ __forceinline__ void raise(const float (&x)[NT][4], const float (&ls)[2]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a = fmaxf(x[nt][e], x[nt][e + 2]);
                float b = fmaxf(x[nt][e] + ls[0], x[nt][e + 2] + ls[1]);
#pragma unroll
                for (int off = 4; off < 32; off *= 2) {
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
                }
                a = fmaxf(a, m[nt][e]);
                b = fmaxf(b, M[nt][e]);
                const float al = fast_exp2(m[nt][e] - a), ao = fast_exp2(M[nt][e] - b);
                m[nt][e] = a;
                M[nt][e] = b;
                f[nt][e] = fast_exp2(a - b);
                l[nt][e] *= al;
#pragma unroll
                for (int g = 0; g < NG; ++g) z[g][nt][e] *= al;
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    o[i][nt][e] *= ao;
                    o[i][nt][e + 2] *= ao;
                }
            }
    }

    // One 16-row tile at shared-memory addresses k, v, par (row 0 of the tile's first half).
    // MASKED: bit r of rows = row r of the tile counts, and column c sees keys up to last + tok[c].
    template <bool MASKED>
    __device__ __forceinline__ void tile(uint32_t k, uint32_t v, uint32_t par, uint32_t rows,
                                         int key0, int last) {
        uint32_t ka[KW], kb[KW], pa[PW], pb_[PW];
        lds<KW>(k + koff[0], ka);
        lds<KW>(k + koff[1], kb);
        lds<PW>(par + poff[0], pa);
        lds<PW>(par + poff[1], pb_);
        float x[NT][4];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
            for (int w = g * KW / NG; w < (g + 1) * KW / NG; ++w) {
                if constexpr (BITS == 4) {
                    const uint32_t a8 = ka[w] >> 8, b8 = kb[w] >> 8;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t mask = h ? 0x00f000f0u : 0x000f000fu;
                        const uint32_t a0 = ka[w] & mask, a1 = kb[w] & mask, a2 = a8 & mask,
                                       a3 = b8 & mask;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(acc[nt], a0, a1, a2, a3, qf[2 * w + h][nt][0],
                                          qf[2 * w + h][nt][1]);
                    }
                } else {
                    const uint32_t a0 = __byte_perm(ka[w], 0u, 0x4140), a1 = __byte_perm(kb[w], 0u, 0x4140),
                                   a2 = __byte_perm(ka[w], 0u, 0x4342), a3 = __byte_perm(kb[w], 0u, 0x4342);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(acc[nt], a0, a1, a2, a3, qf[w][nt][0], qf[w][nt][1]);
                }
            }
            const float sa = bf16_lo_to_f32(pa[2 * g]), na = bf16_hi_to_f32(pa[2 * g]);
            const float sb = bf16_lo_to_f32(pb_[2 * g]), nb = bf16_hi_to_f32(pb_[2 * g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = (e < 2 ? na : nb) * qsum[g][nt][e & 1];
                    const float base = g == 0 ? y : y + x[nt][e];
                    x[nt][e] = __fmaf_rn(e < 2 ? sa : sb, acc[nt][e], base);
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] *= cf[nt][e & 1];

        float vsa[NG], vsb[NG], vna[NG], vnb[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            vsa[g] = bf16_lo_to_f32(pa[2 * g + 1]);
            vna[g] = bf16_hi_to_f32(pa[2 * g + 1]);
            vsb[g] = bf16_lo_to_f32(pb_[2 * g + 1]);
            vnb[g] = bf16_hi_to_f32(pb_[2 * g + 1]);
        }
        if constexpr (MASKED) {
            // rows that do not count may hold anything, NaN parameters too
            const int r = quant_tile_row(gq);
            const bool oka = (rows >> r) & 1u, okb = (rows >> (r + 8)) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + r + (e < 2 ? 0 : 8);
                    if (!(e < 2 ? oka : okb) || key - tok[nt][e & 1] > last) x[nt][e] = -CUDART_INF_F;
                }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (!oka) vsa[g] = vna[g] = 0.f;
                if (!okb) vsb[g] = vnb[g] = 0.f;
            }
        }

        // weights: p for the sums, p * f * vs for the product
        float pe[NT][4], wt[NG][NT][4], top;
        auto weights = [&]() {
            top = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pe[nt][e] = fast_exp2(x[nt][e] - m[nt][e & 1]);
                    top = fmaxf(top, pe[nt][e]);
                    const float pf = pe[nt][e] * f[nt][e & 1];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        wt[g][nt][e] = pf * (e < 2 ? vsa[g] : vsb[g]);
                        // a key that the column does not see adds nothing, whatever its row holds
                        if (MASKED && x[nt][e] == -CUDART_INF_F) wt[g][nt][e] = 0.f;
                        top = fmaxf(top, wt[g][nt][e]);
                    }
                }
        };
        weights();
        if (__any_sync(0xffffffffu, top > 256.f)) {
            float sa = vsa[0], sb = vsb[0];
#pragma unroll
            for (int g = 1; g < NG; ++g) {
                sa = fmaxf(sa, vsa[g]);
                sb = fmaxf(sb, vsb[g]);
            }
            // a scale's exponent within [-64, 120]: 0 has none, and 2^(m - M) stays a normal number
            const float ls[2] = {fminf(fmaxf(fast_log2(sa), -64.f), 120.f),
                                 fminf(fmaxf(fast_log2(sb), -64.f), 120.f)};
            raise(x, ls);
            weights();
        }
        uint32_t pb[NG][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] += pe[nt][0] + pe[nt][2];
            l[nt][1] += pe[nt][1] + pe[nt][3];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float za = pe[nt][e] * vna[g], zb = pe[nt][e + 2] * vnb[g];
                    if (MASKED && x[nt][e] == -CUDART_INF_F) za = 0.f;
                    if (MASKED && x[nt][e + 2] == -CUDART_INF_F) zb = 0.f;
                    z[g][nt][e] += za + zb;
                }
                pb[g][nt][0] = movmatrix_trans(pack_f16x2(wt[g][nt][0], wt[g][nt][1]));
                pb[g][nt][1] = movmatrix_trans(pack_f16x2(wt[g][nt][2], wt[g][nt][3]));
            }
        }

        // O^T += V^T P^T: pairs of keys for one element from the words of two rows
        uint32_t va[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) lds<VW>(v + voff[i], va[i]);
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7632u : 0x5410u;
                const uint32_t lo = __byte_perm(va[0][w], va[1][w], sel);
                const uint32_t hi = __byte_perm(va[2][w], va[3][w], sel);
                if constexpr (BITS == 4) {
                    const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
                    const int t = 4 * w + 2 * h;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16_16816(o[t][nt], lo & 0x000f000fu, lo & 0x00f000f0u, hi & 0x000f000fu,
                                      hi & 0x00f000f0u, pb[t * NG / S][nt][0], pb[t * NG / S][nt][1]);
                        mma_f16_16816(o[t + 1][nt], lo8 & 0x000f000fu, lo8 & 0x00f000f0u,
                                      hi8 & 0x000f000fu, hi8 & 0x00f000f0u,
                                      pb[(t + 1) * NG / S][nt][0], pb[(t + 1) * NG / S][nt][1]);
                    }
                } else {
                    const int t = 2 * w + h;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(o[t][nt], lo & 0x00ff00ffu, (lo >> 8) & 0x00ff00ffu,
                                      hi & 0x00ff00ffu, (hi >> 8) & 0x00ff00ffu,
                                      pb[t * NG / S][nt][0], pb[t * NG / S][nt][1]);
                }
            }
    }

    // Ends a segment: sums over the lanes, and o becomes sum p V relative to m (its final value but
    // for the division by l), so that m, l and o merge like any softmax state.
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
                const float back = fast_exp2(M[nt][e] - m[nt][e]);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
#pragma unroll
                    for (int off = 4; off < 32; off *= 2)
                        z[g][nt][e] += __shfl_xor_sync(0xffffffffu, z[g][nt][e], off);
#pragma unroll
                    for (int i = g * S / NG; i < (g + 1) * S / NG; ++i) {
                        o[i][nt][e] = __fmaf_rn(o[i][nt][e] * kUnit, back, z[g][nt][e]);
                        o[i][nt][e + 2] = __fmaf_rn(o[i][nt][e + 2] * kUnitHi, back, z[g][nt][e]);
                    }
                }
            }
    }

    // The columns of n-tile nt in merge slot `slot`.
    __device__ __forceinline__ void stash(const QuantSmem& sm, int slot, int nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = slot * 8 + 2 * qd + e;
            if (gq == 0) {
                sm.merge_m[c] = m[nt][e];
                sm.merge_l[c] = l[nt][e];
            }
            float* row = sm.merge_o + c * Gm::kMergeStride + 2 * gq;
#pragma unroll
            for (int i = 0; i < S; ++i)
                *reinterpret_cast<float2*>(row + 16 * i) = make_float2(o[i][nt][e], o[i][nt][e + 2]);
        }
    }

    // Merges merge slot `slot` into the columns of n-tile nt.
    __device__ __forceinline__ void fold(const QuantSmem& sm, int slot, int nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = slot * 8 + 2 * qd + e;
            const float m2 = sm.merge_m[c], top = fmaxf(m[nt][e], m2);
            const float a = fast_exp2(m[nt][e] - top), b = fast_exp2(m2 - top);
            m[nt][e] = top;
            l[nt][e] = l[nt][e] * a + sm.merge_l[c] * b;
            const float* row = sm.merge_o + c * Gm::kMergeStride + 2 * gq;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const float2 y = *reinterpret_cast<const float2*>(row + 16 * i);
                o[i][nt][e] = o[i][nt][e] * a + y.x * b;
                o[i][nt][e + 2] = o[i][nt][e + 2] * a + y.y * b;
            }
        }
    }
};

__device__ __forceinline__ void store_row4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Merges the nseg partial rows of a unit by log-sum-exp in segment order and stores its output.
template <class Gm>
__device__ __forceinline__ void quant_merge_unit(const QuantParams& p, size_t row0, int first_seg,
                                                 int nseg) {
    constexpr int D4 = Gm::D / 4;
    const int SH = p.kh * p.cols;
    const float* lse = p.part_lse + static_cast<size_t>(first_seg) * SH;
    const float4* o = reinterpret_cast<const float4*>(p.part_o + static_cast<size_t>(first_seg) * SH * Gm::D);
    for (int i = threadIdx.x; i < SH * D4; i += Gm::kConsumers) {
        const int r = i / D4;
        float top = -CUDART_INF_F;
#pragma unroll 4
        for (int k = 0; k < nseg; ++k) top = fmaxf(top, __ldcg(lse + static_cast<size_t>(k) * SH + r));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int k = 0; k < nseg; ++k) {
            const float e = __ldcg(lse + static_cast<size_t>(k) * SH + r);
            const float4 y = __ldcg(o + static_cast<size_t>(k) * SH * D4 + i);
            const float w = e == -CUDART_INF_F ? 0.f : fast_exp2(e - top);   // an empty piece: zeros
            sum += w;
            acc = fma4(w, y, acc);
        }
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        store_row4(p.out + row0 * Gm::D + static_cast<size_t>(i) * 4,
                   make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
}

template <int D, int BITS, int NG, int NC>
__global__ void __launch_bounds__(QuantGeometry<D, BITS, NG, NC>::kThreads, 1)
quant_attn_kernel(const QuantParams p) {
    using Gm = QuantGeometry<D, BITS, NG, NC>;
    extern __shared__ unsigned char smem_raw[];
    const QuantSmem sm = quant_carve<Gm>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Gm::kStages; ++s) {
            mbar_init(sm.full + s, 1u);
            mbar_init(sm.empty + s, Gm::W);
        }
        mbar_init(sm.group, Gm::kConsumers);
        *sm.abort = 0;
        *sm.last_flag = 0;
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    allow_dependent_launch();

    // ---- schedule
    const int kh = p.kh, P = p.page_size;
    const int tok = Gm::kStageRows / kh;         // rows of one KV head in a stage
    {
        const int cap = p.max_pages * P;
        for (int b = threadIdx.x; b < p.B; b += Gm::kThreads) {
            const unsigned raw = __ldg(p.kv_lens + static_cast<size_t>(b) * p.kv_stride);
            const int len = raw > static_cast<unsigned>(cap) ? cap : static_cast<int>(raw);
            sm.seq_len[b] = len;
            sm.seq_prefix[b + 1] = (len + tok - 1) / tok;
        }
        __syncthreads();
        if (warp == 0) {
            int carry = 0;
            for (int base = 0; base < p.B; base += 32) {
                const int b = base + lane;
                int v = b < p.B ? sm.seq_prefix[b + 1] : 0;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, v, off);
                    if (lane >= off) v += y;
                }
                if (b < p.B) sm.seq_prefix[b + 1] = v + carry;
                carry += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) sm.seq_prefix[0] = 0;
        }
    }
    __syncthreads();
    const int N = sm.seq_prefix[p.B] * (p.Hkv / kh);
    const int C = min(static_cast<int>(gridDim.x), N);
    int t0 = 0, t1 = 0;
    if (static_cast<int>(blockIdx.x) < C) {
        t0 = static_cast<int>(static_cast<long long>(blockIdx.x) * N / C);
        t1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * N / C);
    }
    const int pe = min(P, tok);                  // rows of one page in a stage
    const int page_shift = 31 - __clz(P), pe_shift = 31 - __clz(pe);
    const int block = pe * Gm::ROW;              // bytes of one (page, head) in a stage

    if (warp == Gm::W) {
        // ================================================================ copying warp
        const int npg = tok >> pe_shift;         // pages of a stage (<= 32)
        bool ok = true;
        int it = 0;
        QuantUnit U{};
        U.nt = 0;
        int nxt = -1;                            // this lane's page of the stage to come
        auto fetch = [&](int t) {
            if (t >= t1) return;
            if (t >= U.base + U.nt || U.nt == 0) U = quant_locate(p, sm, t);
            const int slot = ((t - U.base) * tok >> page_shift) + lane;
            const bool in = lane < npg && slot < ((U.len + P - 1) >> page_shift);
            nxt = in ? __ldg(p.block_table + static_cast<size_t>(U.b) * p.max_pages + slot) : -1;
        };
        fetch(t0);
        for (int t = t0; t < t1; ++t, ++it) {
            const int s = it % Gm::kStages;
            const uint32_t ph = (it / Gm::kStages) & 1;
            const int page = nxt, g = U.g, len = U.len, key0 = (t - U.base) * tok;
            fetch(t + 1);                        // its latency passes while this stage's slot frees
            if (!mbar_wait_warp(sm.empty + s, ph ^ 1u, sm.abort)) { ok = false; break; }
            const bool good = page >= 0 && page < p.num_pages;
            const unsigned pages = __ballot_sync(0xffffffffu, good);
            unsigned char* dst = sm.stages + s * Gm::kStageBytes;
            if (lane == 0) {
                sm.stage_len[s] = min(tok, len - key0);
                sm.stage_pages[s] = pages;
                mbar_arrive_expect_tx(sm.full + s, __popc(pages) * kh * block);
            }
            __syncwarp();
            const size_t page_bytes = static_cast<size_t>(P) * Gm::ROW;
            if (P <= tok) {
                // the kh heads of a page are contiguous
                if (good)
                    bulk_load(dst + lane * kh * block,
                              p.pool + (static_cast<size_t>(page) * p.Hkv + g * kh) * page_bytes,
                              kh * block, sm.full + s);
            } else if (pages) {
                // tok rows of one page: K codes, V codes and parameters of each head
                const int pg = __shfl_sync(0xffffffffu, page, 0), r0 = key0 & (P - 1);
                const int h = lane / 3, part = lane - 3 * h;
                if (h < kh) {
                    const unsigned char* src =
                        p.pool + (static_cast<size_t>(pg) * p.Hkv + g * kh + h) * page_bytes;
                    unsigned char* to = dst + h * block;
                    if (part < 2)
                        bulk_load(to + part * pe * Gm::RB, src + (part * P + r0) * Gm::RB, pe * Gm::RB,
                                  sm.full + s);
                    else
                        bulk_load(to + 2 * pe * Gm::RB, src + 2 * P * Gm::RB + r0 * Gm::PB, pe * Gm::PB,
                                  sm.full + s);
                }
            }
            __syncwarp();
        }
        if (!ok) {
            *sm.abort = 1;
            record_error(p.err, kErrWaitEmpty);
            if (lane == 0) {
                // let every copy this warp issued land before the CTA can exit
                for (int k = it - 1; k >= 0 && k >= it - Gm::kStages; --k)
                    if (!mbar_wait(sm.full + (k % Gm::kStages), (k / Gm::kStages) & 1, nullptr, kWaitLimitNs)) {
                        record_error(p.err, kErrDrain);
                        break;
                    }
            }
        }
        return;
    }

    // ==================================================================== consumer warps
    // Warp w: column slice w % CS, then KV head, then its share of that head's tiles.
    const int cs = warp & ((1 << p.slices_shift) - 1);
    const int wt = warp >> p.slices_shift, WT = Gm::W >> p.slices_shift;
    const int head = wt & (kh - 1);
    const int kh_shift = 31 - __clz(kh);
    QuantWarp<Gm> cw;
    // the second eight rows of a tile: next in the page, or on the next page (8-row pages)
    cw.init(lane, head, cs * NC, p.sq, pe >= 16 ? 8 * Gm::RB : kh * block,
            pe >= 16 ? 8 * Gm::PB : kh * block);
    uint32_t gphase = 0;

    // sequences without rows: zero output rows
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (sm.seq_len[b] != 0) continue;
        const size_t n = static_cast<size_t>(p.Hq) * p.sq * D;
        for (size_t i = threadIdx.x; i < n; i += Gm::kConsumers)
            p.out[b * n + i] = __float2bfloat16_rn(0.f);
    }

    auto unit_row0 = [&](const QuantUnit& U) -> size_t {   // first q / out row of the unit
        return (static_cast<size_t>(U.b) * p.Hkv + U.g * kh) * p.cols;
    };
    QuantUnit U{};
    if (t0 < t1) {
        U = quant_locate(p, sm, t0);
        cw.load_q(p, unit_row0(U) + head * p.cols);
    }
    int it = 0;
    for (int t = t0; t < t1;) {
        const int tend = min(t1, U.base + U.nt);
        const bool whole = t == U.base && tend == U.base + U.nt;
        // rows a causal column may see: keys up to last + its token; without masking, every row
        const int last = p.causal ? U.len - p.sq : 0x7fffffff;
        cw.reset();
        for (; t < tend; ++t, ++it) {
            const int s = it % Gm::kStages;
            const uint32_t ph = (it / Gm::kStages) & 1;
            if (!mbar_wait_warp(sm.full + s, ph, sm.abort)) {
                *sm.abort = 1;
                record_error(p.err, kErrWaitFull);
                return;
            }
            const int nvalid = static_cast<int>(sm.stage_len[s]);
            const unsigned pages = sm.stage_pages[s];
            const uint32_t base = smem_u32(sm.stages + s * Gm::kStageBytes);
            const int key0 = (t - U.base) * tok;
            for (int i = wt; i < Gm::kTiles; i += WT) {
                const int r0 = (i >> kh_shift) * 16;       // first row of the tile
                const int pg = r0 >> pe_shift;
                const uint32_t blk = base + (pg * kh + head) * block;
                const int rr = r0 & (pe - 1);
                const uint32_t k = blk + rr * Gm::RB, v = k + pe * Gm::RB,
                               par = blk + 2 * pe * Gm::RB + rr * Gm::PB;
                const int n = nvalid - r0;
                uint32_t rows = n >= 16 ? 0xffffu : n > 0 ? (1u << n) - 1u : 0u;
                if (!((pages >> pg) & 1u)) rows &= pe >= 16 ? 0u : 0xff00u;
                if (pe < 16 && !((pages >> (pg + 1)) & 1u)) rows &= 0x00ffu;
                if (rows == 0u) continue;
                if (rows == 0xffffu && key0 + r0 + 15 <= last)
                    cw.template tile<false>(k, v, par, rows, 0, 0);
                else
                    cw.template tile<true>(k, v, par, rows, key0 + r0, last);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.empty + s);
        }

        // ---- end of the segment
        cw.settle();
        const int first_seg = tile_owner(U.base, N, C) + U.u;
        const int nseg = tile_owner(U.base + U.nt - 1, N, C) + U.u - first_seg + 1;
        const int seg = static_cast<int>(blockIdx.x) + U.u;
        const int SH = kh * p.cols;
        const size_t row0 = unit_row0(U);
#pragma unroll
        for (int nt = 0; nt < Gm::NT; ++nt) {
            // warps past the eighth (same head and columns as warp - 8) are folded into those first
            if (Gm::W == 16) {
                if (warp >= 8) cw.stash(sm, warp - 8, nt);
                if (!quant_sync(sm, gphase, p.err)) return;
                if (warp < 8) cw.fold(sm, warp, nt);
                __syncwarp();
            }
            if (warp < 8) cw.stash(sm, warp, nt);
            if (!quant_sync(sm, gphase, p.err)) return;
            // rows of this round: (head, slice, column); their pieces lie in the slots of KS warps
            constexpr int D4 = D / 4;
            const int pieces_shift = p.slices_shift + kh_shift;
            const int KS = 8 >> pieces_shift;
            for (int i = threadIdx.x; i < (8 << pieces_shift) * D4; i += Gm::kConsumers) {
                const int d4 = i % D4, r = i / D4;
                const int c = r & 7, vw = r >> 3;             // vw: head << slices_shift | slice
                const int col = (vw & ((1 << p.slices_shift) - 1)) * NC + nt * 8 + c;
                if (col >= p.cols) continue;
                float top = kQuantUnset;
                for (int k = 0; k < KS; ++k)
                    top = fmaxf(top, sm.merge_m[((k << pieces_shift) + vw) * 8 + c]);
                float sum = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < KS; ++k) {
                    const int slot = ((k << pieces_shift) + vw) * 8 + c;
                    const float w = fast_exp2(sm.merge_m[slot] - top);
                    sum += w * sm.merge_l[slot];
                    acc = fma4(w, *reinterpret_cast<const float4*>(
                                      sm.merge_o + slot * Gm::kMergeStride + 4 * d4), acc);
                }
                const float inv = sum == 0.f ? 0.f : 1.0f / sum;   // no row at all: zeros
                const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                const int ur = (vw >> p.slices_shift) * p.cols + col;
                if (whole) {
                    store_row4(p.out + (row0 + ur) * D + 4 * d4, v);
                } else {
                    const size_t pr = static_cast<size_t>(seg) * SH + ur;
                    *reinterpret_cast<float4*>(p.part_o + pr * D + 4 * d4) = v;
                    if (d4 == 0) p.part_lse[pr] = sum == 0.f ? -CUDART_INF_F : top + fast_log2(sum);
                }
            }
            if (!quant_sync(sm, gphase, p.err)) return;
        }
        const QuantUnit done = U;
        if (t < t1) {
            U = quant_locate(p, sm, t);
            cw.load_q(p, unit_row0(U) + head * p.cols);
        }
        if (!whole) {
            // the barrier above orders every partial store before thread 0's release
            if (threadIdx.x == 0) {
                const unsigned prev = atomic_add_acq_rel_gpu(p.counters + done.u);
                *sm.last_flag = prev == static_cast<unsigned>(nseg - 1) ? 1 : 0;
            }
            if (!quant_sync(sm, gphase, p.err)) return;
            if (*sm.last_flag) {
                quant_merge_unit<Gm>(p, row0, first_seg, nseg);
                if (threadIdx.x == 0) p.counters[done.u] = 0u;
            }
            if (!quant_sync(sm, gphase, p.err)) return;
        }
    }
}

// Launches the instantiation for head dim D and BITS-bit codes: groups = D / group, narrow: at
// most 8 query columns per KV head.
template <int D, int BITS>
cudaError_t launch_quant(int groups, bool narrow, const QuantParams& p, int grid, cudaStream_t st);

template <int D, int BITS, int NG, int NC>
cudaError_t launch_quant_as(const QuantParams& p, int grid, cudaStream_t st) {
    using Gm = QuantGeometry<D, BITS, NG, NC>;
    void* args[] = {const_cast<QuantParams*>(&p)};
    return launch_configured(reinterpret_cast<const void*>(&quant_attn_kernel<D, BITS, NG, NC>),
                             Gm::kSmemBytes, grid, Gm::kThreads, st, args);
}

template <int D, int BITS>
cudaError_t launch_quant_any(int groups, bool narrow, const QuantParams& p, int grid, cudaStream_t st) {
    switch (groups) {
        case 1: return narrow ? launch_quant_as<D, BITS, 1, 8>(p, grid, st)
                              : launch_quant_as<D, BITS, 1, 16>(p, grid, st);
        case 2: return narrow ? launch_quant_as<D, BITS, 2, 8>(p, grid, st)
                              : launch_quant_as<D, BITS, 2, 16>(p, grid, st);
        case 4:
            if constexpr (D == 128)
                return narrow ? launch_quant_as<D, BITS, 4, 8>(p, grid, st)
                              : launch_quant_as<D, BITS, 4, 16>(p, grid, st);
            break;
    }
    return cudaErrorInvalidValue;
}

}  // namespace da
