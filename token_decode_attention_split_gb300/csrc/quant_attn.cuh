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
// tile has no cross-lane maximum at all.  The result is the same for any reference; sums stay in fp32.
//
// V's codes are taken about their middle code: sum w c = sum w (c - mid) + mid sum w, the second sum
// in fp32 (it joins vmin) and the first as the product minus mid times the sum of the rounded weights
// (one more MMA per tile, whose A operand is mid everywhere), so a weight's rounding error meets
// centred codes.  At 131071 keys the output's error falls from 0.0030 to 0.0018 of its norm (its own
// bf16 rounding is 0.0017).
//
// Work.  A unit is one sequence and kh adjacent KV heads; a stage is 128 or 256 rows, split evenly
// over those heads.  The stages of all units are laid end to end, each unit followed by unit_pad empty
// places for the time that its end takes, and CTA c of a persistent grid (one per SM) takes an equal
// contiguous range of places; its piece of a unit is a segment.  A page of kh
// heads is contiguous (codes and parameters), so a stage is a few bulk copies.  The warps of a copying
// warpgroup fill a ring of stages; consumer warps each take 16-row tiles of one KV head: S^T = K Q^T
// and O^T += V^T P^T on mma.m16n8k16 with the keys (then the elements of V) on M and the query columns
// on N, each with a running state of its own, merged once per segment.
//
// What bounds it.  8-bit codes: HBM.  4-bit codes halve the bytes and leave 48 ns of HBM time per
// 16-row tile and SM (D = 128, 136 bytes a row) for about 225 warp instructions, 104 of them the masks,
// shifts and byte permutes that make fp16 operands (two cycles each on their pipe): the kernel is issue
// bound at about 53 ns a tile (measured with the cache in L2), so everything around the tiles is kept
// off the schedulers.  Twelve consumer warps of 160 registers in three groups, each on every third
// stage, and three copying warps: 64 ns a tile (66 with eight consumer warps in one group, 71 with
// sixteen of 112 registers; 74 with one copying warp, whose lookup, wait and copy take longer than a
// stage); fp32 arithmetic on register pairs (f32x2) and waits that nap instead of polling: 62 ns; warp
// indices broadcast, so that no warp-wide instruction needs a convergence check: 56 ns; cheaper ends: 53 ns.
//
// A segment that covers its unit writes the output; any other writes its normalised partial rows
// and log2-sum-exps, and the CTA that completes the unit (an acquire-release counter) merges them
// in segment order, so the result depends on no timing.  Every wait is bounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "f32x2.cuh"
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
    int kh_shift, upb;           // log2 of the KV heads per unit, units per sequence: Hkv >> kh_shift
    int unit_pad;                // empty places after a unit's stages
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
    // Consumer warps work in groups, each group on its own stage in turn.
    static constexpr bool kNarrow4 = NC == 8 && BITS == 4;
    static constexpr int kGroups = kNarrow4 ? 3 : 1;
    static constexpr int WG = kNarrow4 ? 4 : 8;            // warps of a group
    static constexpr int W = kGroups * WG;
    static constexpr int kConsumers = 32 * W;
    // Copying warps (of one more warpgroup), each on every kCopyWarps-th stage.  The ring has a multiple
    // of kGroups and of kCopyWarps slots, so a slot is always filled by the same warp and emptied by
    // the same group: nobody can wait for a phase two rounds away, which a parity could not tell from
    // the one before.
    static constexpr int kCopyWarps = kGroups;
    static constexpr int kThreads = kConsumers + 128;
    // Registers per thread: the launch gives every thread the same share of 65536; the copying
    // warpgroup hands most of its own to the consumers.
    static constexpr int kLaunchRegs = kNarrow4 ? 128 : 168;
    static constexpr int kCopyRegs = kNarrow4 ? 32 : 40;
    static constexpr int kConsumerRegs = kNarrow4 ? 160 : 232;
    static_assert(kConsumers * kConsumerRegs + 128 * kCopyRegs <= kThreads * kLaunchRegs, "registers");
    static constexpr int kTiles = kNarrow4 || (D == 128 && BITS == 8) ? 8 : 16;   // 16-row tiles of a stage
    static constexpr int UT = NC == 8 && NG < 4 ? kTiles / WG : 1;   // tiles that a warp takes together
    static constexpr int TPW = NC == 8 ? kTiles / WG / UT : 1;   // sets of them whose places are kept
    static constexpr int kStageRows = kTiles * 16;
    static constexpr int kStageBytes = kStageRows * ROW;
    static constexpr int kMergeStride = D + 4;             // floats of a merge row
    static constexpr int kMergeFloats = W * NC * (kMergeStride + 2);   // [warp][column]
    static constexpr int kMaxStages = kGroups == 3 ? 9 : 8;
    static constexpr int kMiscBytes = 512;
    static constexpr int kSchedBytes = (2 * kMaxPagedBatch + 2) * 4;
    static constexpr int kFixedBytes = kMergeFloats * 4 + kMiscBytes + kSchedBytes;
    static constexpr int kStagesFit = (kSmemBudget - 128 - kFixedBytes) / kStageBytes;
    static constexpr int kStages =
        (kStagesFit > kMaxStages ? kMaxStages : kStagesFit) / kCopyWarps * kCopyWarps;
    static constexpr int kSmemBytes = 128 + kStages * kStageBytes + kFixedBytes;
    static_assert(kCopyWarps <= 3 && kStages >= 2 && kStages >= kCopyWarps && kStages % kCopyWarps == 0 &&
                  kStages % kGroups == 0 && kStageBytes % 128 == 0 && kTiles >= WG, "ring");
};

struct QuantSmem {
    unsigned char* stages;
    float* merge_o;      // [W][NC columns][kMergeStride]
    float* merge_m;      // [W][NC]
    float* merge_l;      // [W][NC]
    uint64_t* full;
    uint64_t* empty;
    uint64_t* group;         // all consumers
    uint64_t* stashed;       // the merge slots hold every warp's columns of a segment
    uint64_t* combined;      // they have been merged and may be written again
    int* stage_len;          // rows per head of the stage inside the sequence; -1: every row counts
    unsigned* stage_pages;   // bit i: page i of the stage was copied
    volatile int* abort;
    int* last_flag;      // [2]
    int* seq_prefix;     // [B + 1] exclusive prefix of the sequences' places (of one unit each)
    int* seq_len;        // [B]
};

template <class Gm>
__device__ __forceinline__ QuantSmem quant_carve(unsigned char* raw) {
    QuantSmem s;
    unsigned char* base = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    s.stages = base;
    unsigned char* p = base + Gm::kStages * Gm::kStageBytes;
    s.full = reinterpret_cast<uint64_t*>(p);
    s.empty = s.full + Gm::kMaxStages;
    s.group = s.empty + Gm::kMaxStages;
    s.stashed = s.group + 1;
    s.combined = s.stashed + 1;
    s.stage_len = reinterpret_cast<int*>(s.combined + 1);
    s.stage_pages = reinterpret_cast<unsigned*>(s.stage_len + Gm::kMaxStages);
    s.abort = reinterpret_cast<volatile int*>(s.stage_pages + Gm::kMaxStages);
    s.last_flag = const_cast<int*>(s.abort) + 1;
    p += Gm::kMiscBytes;
    s.merge_o = reinterpret_cast<float*>(p);
    s.merge_m = s.merge_o + Gm::W * Gm::NC * Gm::kMergeStride;
    s.merge_l = s.merge_m + Gm::W * Gm::NC;
    s.seq_prefix = reinterpret_cast<int*>(s.merge_l + Gm::W * Gm::NC);
    s.seq_len = s.seq_prefix + kMaxPagedBatch + 1;
    return s;
}

struct QuantUnit {
    int b, g, u;     // sequence, group of kh KV heads, unit index
    int len, nt;     // live rows, stages
    int base;        // place of the first stage
};

// The unit of stage t; a whole warp calls it.  The sequence is the last b with seq_prefix[b] * units per
// sequence <= t: a ballot over every 32nd candidate, then one over the 32 in between.
__device__ __forceinline__ QuantUnit quant_locate(const QuantParams& p, const QuantSmem& sm, int t) {
    const int upb = p.upb, lane = threadIdx.x & 31;
    int b = 0;
    for (int hop = (p.B + 31) / 32 > 1 ? 32 : 1; hop > 0; hop = hop == 32 ? 1 : 0) {
        const int c = b + lane * hop;
        const bool at = c < p.B && sm.seq_prefix[c] * upb <= t;
        b += (__popc(__ballot_sync(0xffffffffu, at)) - 1) * hop;
    }
    QuantUnit U;
    U.b = b;
    const int places = sm.seq_prefix[b + 1] - sm.seq_prefix[b];
    U.nt = places - p.unit_pad;
    const int r = t - sm.seq_prefix[b] * upb;
    U.g = r / places;
    U.u = b * upb + U.g;
    U.len = sm.seq_len[b];
    U.base = sm.seq_prefix[b] * upb + U.g * places;
    return U;
}

// The stages [0, N) over C CTAs: the first N % C take one more than the others.
struct QuantSplit {
    int q, r;
    __device__ __forceinline__ int first(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int owner(int t) const {
        const int longer = r * (q + 1);
        return t < longer ? t / (q + 1) : r + (t - longer) / q;
    }
};

// The unit after U: the next head group, or the next sequence with rows; past the last unit, one that
// begins at `end`.
__device__ __forceinline__ QuantUnit quant_next(const QuantParams& p, const QuantSmem& sm, QuantUnit U,
                                                int end) {
    U.base += U.nt + p.unit_pad;
    if (U.base >= end) {
        U.base = end;
        return U;
    }
    ++U.u;
    if (++U.g == p.upb) {
        U.g = 0;
        do {
            ++U.b;
            U.nt = sm.seq_prefix[U.b + 1] - sm.seq_prefix[U.b];
            if (U.nt == 0) U.u += p.upb;
        } while (U.nt == 0);
        U.nt -= p.unit_pad;
        U.len = sm.seq_len[U.b];
    }
    return U;
}

// mbar_wait_warp that naps between its polls, so that a waiting warp leaves the scheduler's issue slots
// to the others (the twelve consumer warps of the 4-bit kernel are bound by them).
// Gives up after about a second, or when another thread of the CTA has raised *abort.
template <unsigned NAP_NS>
__device__ __forceinline__ bool quant_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    bool done = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, done)) {
        const uint64_t t0 = global_timer_ns();
        for (unsigned polls = 1; !done && !*abort; ++polls) {
            __nanosleep(NAP_NS);
            done = mbar_try_wait(bar, parity);
            if (polls % 64 == 0 && global_timer_ns() - t0 > kWaitLimitNs) break;
        }
        done = __all_sync(0xffffffffu, done);
    }
    return done;
}
constexpr unsigned kNapConsumer = 40, kNapCopy = 200, kNapGroup = 20;

__device__ __forceinline__ bool quant_sync(const QuantSmem& sm, uint32_t& phase, unsigned* err) {
    mbar_arrive(sm.group);
    const bool ok = quant_wait<kNapGroup>(sm.group, phase, sm.abort);
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

// D = A * B
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// N consecutive words (aligned to their size, at most 16 bytes a load)
template <int N>
__device__ __forceinline__ void lds(const unsigned char* at, uint32_t (&r)[N]) {
    if constexpr (N == 1) {
        r[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        r[0] = x.x;
        r[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + 4 * i);
            r[i] = x.x;
            r[i + 1] = x.y;
            r[i + 2] = x.z;
            r[i + 3] = x.w;
        }
    }
}

// Row of a 16-row tile (0..7; +8 for the second half) that stands at fragment row i: neighbouring
// fragment rows lie in rows of unlike parity (the K loads of a quarter warp then cover all banks at
// 64 bytes a row) and the rows 2 t, t = 0..3, are the first four (two of each parity for the V loads).
__device__ __forceinline__ int quant_tile_row(int i) { return ((i >> 1) ^ (i & 1)) | ((i & 1) << 2); }

constexpr float kQuantUnset = -3.402823466e38f;   // reference of a column that has seen no row

template <class Gm>
struct QuantWarp {
    static constexpr int D = Gm::D, BITS = Gm::BITS, NG = Gm::NG, NT = Gm::NT, UT = Gm::UT;
    static constexpr int S = D / 16;             // 16-element slices: MMA k-steps of a K row, m-tiles of V
    static constexpr int KW = Gm::RB / 16;       // words of a K row per lane
    static constexpr int VW = Gm::RB / 32;       // words of a V row per lane
    static constexpr int PW = 2 * NG;            // parameter words of a row
    // powers of two of the code operands: 2^-24, and 2^-20 for the upper codes of the 4-bit pairs
    static constexpr float kUnit = 16777216.f;
    static constexpr float kUnitHi = BITS == 4 ? 1048576.f : 16777216.f;
    // the middle code, taken off the V codes again (see the file's head), and as code operands
    static constexpr int kMid = BITS == 4 ? 8 : 128;
    static constexpr uint32_t kMidLo = kMid * 0x00010001u, kMidHi = (BITS == 4 ? 16 : 1) * kMidLo;

    int lane, gq, qd;                // fragment row, quad lane
    int col0;                        // first query column
    uint32_t qf[S][NT][2];           // Q^T fragments (fp16, scaled by a power of two per column)
    // pairs: columns 2 qd and 2 qd + 1 of an n-tile
    f2 qsum[NG][NT];                 // sum of a column's scaled elements per group, in code units
    f2 cf[NT];                       // score units -> log2 domain
    float o[S][NT][4];               // O^T: rows gq (element 16 m + 2 gq) and gq + 8 (element + 1)
    f2 z[NG][NT];                    // this lane's share of sum p * (vmin + kMid * vs)
    float w0[NG][NT][4];             // kMid * sum of the fp16 weights, in o's units
    f2 l[NT];                        // this lane's share of sum p
    f2 nm[NT], f[NT];                // -m and 2^(m - M)
    float M[NT][2];
    int tok[NT][2];                  // query token of the column (causal)
    int koff, voff[2], poff;         // lane offsets inside a tile: K row, V rows, parameters
    int half_k, half_p;              // from a row of the tile's first half to its second half

    // (lane, gq, qd and col0 are set)
    __device__ __forceinline__ void init(int sq, int half_k_, int half_p_) {
        koff = quant_tile_row(gq) * Gm::RB + qd * (4 * KW);
        voff[0] = quant_tile_row(2 * qd) * Gm::RB + gq * (4 * VW);
        voff[1] = quant_tile_row(2 * qd + 1) * Gm::RB + gq * (4 * VW);
        poff = quant_tile_row(gq) * Gm::PB;
        half_k = half_k_;
        half_p = half_p_;
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
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] = f2_of(0.f, 0.f);
            nm[nt] = f2_of(-kQuantUnset, -kQuantUnset);
            f[nt] = f2_of(1.f, 1.f);
            M[nt][0] = M[nt][1] = kQuantUnset;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                z[g][nt] = f2_of(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) w0[g][nt][e] = 0.f;
            }
        }
    }

    // Query rows row0 .. row0 + cols - 1 (columns at or past cols are zero): elements 16 s + 4 qd .. + 3
    // of column gq of each n-tile
    __device__ __forceinline__ void fetch_q(const QuantParams& p, size_t row0, uint2 (&raws)[NT][S]) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = col0 + nt * 8 + gq;
            const bool ok = c < p.cols;
            const uint2* row = reinterpret_cast<const uint2*>(p.q + (row0 + (ok ? c : 0)) * D);
#pragma unroll
            for (int s = 0; s < S; ++s) raws[nt][s] = ok ? __ldg(row + 4 * s + qd) : make_uint2(0u, 0u);
        }
    }
    __device__ __forceinline__ void set_q(float scale_log2, const uint2 (&raws)[NT][S]) {
        auto larger = [](uint32_t a, uint32_t b) {   // per half: the larger magnitude
            const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a),
                                             __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
            return *reinterpret_cast<const uint32_t*>(&m);
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint2(&raw)[S] = raws[nt];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < S; ++s) top = larger(larger(top, raw[s].x), raw[s].y);
            top = larger(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = larger(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top = max(top >> 16, top & 0xffffu);
            // the largest element goes to [2^14, 2^15) (an infinity stays one, a NaN spoils its row)
            const int ex = min(max(static_cast<int>(top >> 7), 27), 254);
            const float up = __int_as_float((268 - ex) << 23);
            const float down = __int_as_float((ex - 14) << 23);
            // 4 bits: a word holds two slices; its masked pairs are codes i and i + 4, at 2^-24 for even
            // i and at 2^-20 for odd i, whose Q elements are therefore scaled by 2^-4 more
            constexpr float kOdd = BITS == 4 ? 0.0625f : 1.0f;
            const f2 up2 = f2_of(up, up * kOdd);
            f2 v[S][2], gs[NG];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                v[s][0] = f2_mul(f2_of(bf16_lo_to_f32(raw[s].x), bf16_hi_to_f32(raw[s].x)), up2);
                v[s][1] = f2_mul(f2_of(bf16_lo_to_f32(raw[s].y), bf16_hi_to_f32(raw[s].y)), up2);
                const f2 both = f2_add(v[s][0], v[s][1]);
                gs[s * NG / S] = s % (S / NG) == 0 ? both : f2_add(gs[s * NG / S], both);
            }
            if (BITS == 8) {
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[s][nt][i] = pack_f16x2(f2_get(v[s][i], 0), f2_get(v[s][i], 1));
            } else {
#pragma unroll
                for (int w = 0; w < S / 2; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            qf[2 * w + h][nt][i] = pack_f16x2(f2_get(v[2 * w][i], h), f2_get(v[2 * w + 1][i], h));
            }
            // to the score fragment's columns 2 qd, 2 qd + 1 (held here by the quads of those rows)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float x = __fmaf_rn(f2_get(gs[g], 1), 1.f / kOdd, f2_get(gs[g], 0));
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x *= 1.f / kUnit;
                qsum[g][nt] = f2_of(__shfl_sync(0xffffffffu, x, 8 * qd), __shfl_sync(0xffffffffu, x, 8 * qd + 4));
            }
            const float c2 = scale_log2 * down * kUnit;
            cf[nt] = f2_of(__shfl_sync(0xffffffffu, c2, 8 * qd), __shfl_sync(0xffffffffu, c2, 8 * qd + 4));
        }
    }

    // Raises the references to the maxima of these tiles (and of all tiles before).  x: scores before
    // the factor cf; ls: log2 of a row's largest scale; hidden(u, nt, e): the element does not count.
    template <class Hidden>
    __device__ __forceinline__ void raise(const f2 (&x)[UT][NT][2], const float (&ls)[UT][2], Hidden hidden) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float al[2], ao[2], nf[2], nn[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float c = f2_get(cf[nt], e), m = -f2_get(nm[nt], e);
                float a = m, b = M[nt][e];
#pragma unroll
                for (int u = 0; u < UT; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (hidden(u, nt, e + 2 * i)) continue;
                        const float y = f2_get(x[u][nt][i], e);
                        a = fmaxf(a, y * c);
                        b = fmaxf(b, __fmaf_rn(y, c, ls[u][i]));
                    }
#pragma unroll
                for (int off = 4; off < 32; off *= 2) {
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
                }
                al[e] = fast_exp2(m - a);
                ao[e] = fast_exp2(M[nt][e] - b);
                nf[e] = fast_exp2(a - b);
                nn[e] = -a;
                M[nt][e] = b;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    w0[g][nt][e] *= ao[e];
                    w0[g][nt][e + 2] *= ao[e];
                }
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    o[i][nt][e] *= ao[e];
                    o[i][nt][e + 2] *= ao[e];
                }
            }
            nm[nt] = f2_of(nn[0], nn[1]);
            f[nt] = f2_of(nf[0], nf[1]);
            const f2 al2 = f2_of(al[0], al[1]);
            l[nt] = f2_mul(l[nt], al2);
#pragma unroll
            for (int g = 0; g < NG; ++g) z[g][nt] = f2_mul(z[g][nt], al2);
        }
    }

    // This lane's places in a tile whose K codes, V codes and parameters begin at byte k, v, par of a
    // stage: its K row, the V rows of its two keys, its parameters (those of the tile's second half
    // lie half_k and half_p further).
    struct TileAt {
        int k, va, vb, par;
    };
    __device__ __forceinline__ TileAt tile_at(int k, int v, int par) const {
        return {k + koff, v + voff[0], v + voff[1], par + poff};
    }

    // UT 16-row tiles of one KV head in a stage.
    // MASKED: bit r of rows[u] = row r of the tile counts, and column c sees keys up to last + tok[c].
    template <bool MASKED>
    __device__ __forceinline__ void tiles(const unsigned char* stage, const TileAt (&at)[UT],
                                          const uint32_t (&rows)[UT], const int (&key0)[UT], int last) {
        // from a row to the one 8 further: a constant unless pages have 8 rows, whose stages always come
        // masked
        const int hk = MASKED ? half_k : 8 * Gm::RB, hp = MASKED ? half_p : 8 * Gm::PB;
        uint32_t pa[UT][2][PW];           // parameters of the rows at gq and at gq + 8
        f2 x[UT][NT][2];                  // scores before the factor cf, the same rows
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            uint32_t ka[KW], kb[KW];
            lds<KW>(stage + at[u].k, ka);
            lds<KW>(stage + at[u].k + hk, kb);
            lds<PW>(stage + at[u].par, pa[u][0]);
            lds<PW>(stage + at[u].par + hp, pa[u][1]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float acc[NT][4];
#pragma unroll
                for (int w = g * KW / NG; w < (g + 1) * KW / NG; ++w) {
                    const bool first = w == g * KW / NG;
                    if constexpr (BITS == 4) {
                        const uint32_t a8 = ka[w] >> 8, b8 = kb[w] >> 8;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t mask = h ? 0x00f000f0u : 0x000f000fu;
                            const uint32_t a0 = ka[w] & mask, a1 = kb[w] & mask, a2 = a8 & mask,
                                           a3 = b8 & mask;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (first && h == 0)
                                    mma_f16_16816_first(acc[nt], a0, a1, a2, a3, qf[2 * w][nt][0],
                                                        qf[2 * w][nt][1]);
                                else
                                    mma_f16_16816(acc[nt], a0, a1, a2, a3, qf[2 * w + h][nt][0],
                                                  qf[2 * w + h][nt][1]);
                            }
                        }
                    } else {
                        const uint32_t a0 = __byte_perm(ka[w], 0u, 0x4140),
                                       a1 = __byte_perm(kb[w], 0u, 0x4140),
                                       a2 = __byte_perm(ka[w], 0u, 0x4342),
                                       a3 = __byte_perm(kb[w], 0u, 0x4342);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (first)
                                mma_f16_16816_first(acc[nt], a0, a1, a2, a3, qf[w][nt][0], qf[w][nt][1]);
                            else
                                mma_f16_16816(acc[nt], a0, a1, a2, a3, qf[w][nt][0], qf[w][nt][1]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float ks = bf16_lo_to_f32(pa[u][i][2 * g]), kn = bf16_hi_to_f32(pa[u][i][2 * g]);
                    const f2 ks2 = f2_of(ks, ks), kn2 = f2_of(kn, kn);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const f2 base = g == 0 ? f2_mul(kn2, qsum[g][nt]) : f2_fma(kn2, qsum[g][nt], x[u][nt][i]);
                        x[u][nt][i] = f2_fma(ks2, f2_of(acc[nt][2 * i], acc[nt][2 * i + 1]), base);
                    }
                }
            }
        }

        // rows that do not count may hold anything, NaN parameters too
        bool ok[UT][2];
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                ok[u][i] = !MASKED || ((rows[u] >> (quant_tile_row(gq) + 8 * i)) & 1u) != 0u;
        auto hidden = [&](int u, int nt, int e) -> bool {
            return MASKED && (!ok[u][e / 2] ||
                              key0[u] + quant_tile_row(gq) + 8 * (e / 2) - tok[nt][e & 1] > last);
        };
        f2 vs[UT][NG][2], vn[UT][NG][2];      // scale and middle value of the rows at gq and at gq + 8
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float a = bf16_lo_to_f32(pa[u][i][2 * g + 1]);
                    float b = __fmaf_rn(a, kMid, bf16_hi_to_f32(pa[u][i][2 * g + 1]));
                    if (!ok[u][i]) a = b = 0.f;
                    vs[u][g][i] = f2_of(a, a);
                    vn[u][g][i] = f2_of(b, b);
                }

        // weights: p for the sums, p * f * vs for the product; all of them are non-negative, so a bound
        // on their sum bounds each (a NaN fails the comparison and takes the careful path)
        f2 pe[UT][NT][2], wt[UT][NG][NT][2], sum;
        auto weights = [&]() {
            sum = f2_of(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < UT; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const f2 y = f2_fma(x[u][nt][i], cf[nt], nm[nt]);
                        float a = fast_exp2(f2_get(y, 0)), b = fast_exp2(f2_get(y, 1));
                        if (hidden(u, nt, 2 * i)) a = 0.f;
                        if (hidden(u, nt, 2 * i + 1)) b = 0.f;
                        pe[u][nt][i] = f2_of(a, b);
                        sum = f2_add(sum, pe[u][nt][i]);
                        const f2 pf = f2_mul(pe[u][nt][i], f[nt]);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            f2 w = f2_mul(pf, vs[u][g][i]);
                            // a key that the column does not see adds nothing, whatever its row holds
                            if (MASKED)
                                w = f2_of(hidden(u, nt, 2 * i) ? 0.f : f2_get(w, 0),
                                          hidden(u, nt, 2 * i + 1) ? 0.f : f2_get(w, 1));
                            wt[u][g][nt][i] = w;
                            sum = f2_add(sum, w);
                        }
                    }
        };
        weights();
        if (__any_sync(0xffffffffu, !(f2_get(sum, 0) + f2_get(sum, 1) <= 256.f))) {
            float ls[UT][2];
#pragma unroll
            for (int u = 0; u < UT; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float y = f2_get(vs[u][0][i], 0);
#pragma unroll
                    for (int g = 1; g < NG; ++g) y = fmaxf(y, f2_get(vs[u][g][i], 0));
                    // a scale's exponent within [-64, 120]: 0 has none, and 2^(m - M) stays normal
                    ls[u][i] = fminf(fmaxf(fast_log2(y), -64.f), 120.f);
                }
            raise(x, ls, hidden);
            weights();
        }
        uint32_t pb[UT][NG][NT][2];
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                l[nt] = f2_add(l[nt], f2_add(pe[u][nt][0], pe[u][nt][1]));
#pragma unroll
                for (int g = 0; g < NG; ++g) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (MASKED) {
                            const f2 y = f2_mul(pe[u][nt][i], vn[u][g][i]);
                            z[g][nt] = f2_add(z[g][nt], f2_of(hidden(u, nt, 2 * i) ? 0.f : f2_get(y, 0),
                                                              hidden(u, nt, 2 * i + 1) ? 0.f : f2_get(y, 1)));
                        } else {
                            z[g][nt] = f2_fma(pe[u][nt][i], vn[u][g][i], z[g][nt]);
                        }
                        pb[u][g][nt][i] = movmatrix_trans(
                            pack_f16x2(f2_get(wt[u][g][nt][i], 0), f2_get(wt[u][g][nt][i], 1)));
                    }
                    mma_f16_16816(w0[g][nt], kMidLo, kMidHi, kMidLo, kMidHi, pb[u][g][nt][0],
                                  pb[u][g][nt][1]);
                }
            }

        // O^T += V^T P^T: pairs of keys for one element from the words of two rows
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            uint32_t va[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                lds<VW>(stage + (i & 1 ? at[u].vb : at[u].va) + (i < 2 ? 0 : hk), va[i]);
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7632u : 0x5410u;
                    const uint32_t lo = __byte_perm(va[0][w], va[1][w], sel);
                    const uint32_t hi = __byte_perm(va[2][w], va[3][w], sel);
                    if constexpr (BITS == 4) {
                        const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
                        const int t = 4 * w + 2 * h, ga = t * NG / S, gb = (t + 1) * NG / S;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16_16816(o[t][nt], lo & 0x000f000fu, lo & 0x00f000f0u,
                                          hi & 0x000f000fu, hi & 0x00f000f0u, pb[u][ga][nt][0],
                                          pb[u][ga][nt][1]);
                            mma_f16_16816(o[t + 1][nt], lo8 & 0x000f000fu, lo8 & 0x00f000f0u,
                                          hi8 & 0x000f000fu, hi8 & 0x00f000f0u, pb[u][gb][nt][0],
                                          pb[u][gb][nt][1]);
                        }
                    } else {
                        const int t = 2 * w + h, ga = t * NG / S;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(o[t][nt], lo & 0x00ff00ffu, (lo >> 8) & 0x00ff00ffu,
                                          hi & 0x00ff00ffu, (hi >> 8) & 0x00ff00ffu, pb[u][ga][nt][0],
                                          pb[u][ga][nt][1]);
                    }
                }
        }
    }

    // Ends a segment: sums over the lanes, and o becomes sum p V relative to m (its final value but
    // for the division by l), so that m, l and o merge like any softmax state.
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            auto over_lanes = [&](f2 v) {
#pragma unroll
                for (int off = 4; off < 32; off *= 2) v = f2_add(v, __shfl_xor_sync(0xffffffffu, v, off));
                return v;
            };
            l[nt] = over_lanes(l[nt]);
            const float back[2] = {fast_exp2(M[nt][0] + f2_get(nm[nt], 0)),
                                   fast_exp2(M[nt][1] + f2_get(nm[nt], 1))};
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const f2 zz = over_lanes(z[g][nt]);
#pragma unroll
                for (int i = g * S / NG; i < (g + 1) * S / NG; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        o[i][nt][e] = __fmaf_rn((o[i][nt][e] - w0[g][nt][e]) * kUnit, back[e], f2_get(zz, e));
                        o[i][nt][e + 2] = __fmaf_rn((o[i][nt][e + 2] - w0[g][nt][e + 2]) * kUnitHi, back[e],
                                                    f2_get(zz, e));
                    }
            }
        }
    }

    // This warp's columns to its merge slot.
    __device__ __forceinline__ void stash(const QuantSmem& sm, int warp) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = warp * Gm::NC + nt * 8 + 2 * qd + e;
                if (gq == 0) {
                    sm.merge_m[c] = -f2_get(nm[nt], e);
                    sm.merge_l[c] = f2_get(l[nt], e);
                }
                float* row = sm.merge_o + c * Gm::kMergeStride + 2 * gq;
#pragma unroll
                for (int i = 0; i < S; ++i)
                    *reinterpret_cast<float2*>(row + 16 * i) = make_float2(o[i][nt][e], o[i][nt][e + 2]);
            }
    }
};

__device__ __forceinline__ void store_row4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Merges the nseg partial rows of a unit by log-sum-exp in segment order and stores its output.  A
// thread keeps the loads of kAhead segments of kRows rows in flight: a unit costs one trip to L2 per kAhead
// segments and kRows * kConsumers / (D / 4) rows (twice the segments of half the rows: 51.4 instead of 50.2 us
// for 64 columns of 32 ragged sequences; twice as many in flight costs the streaming loop registers: 53).
template <class Gm>
__device__ __forceinline__ void quant_merge_unit(const QuantParams& p, size_t row0, int first_seg,
                                                 int nseg) {
    constexpr int D4 = Gm::D / 4, kAhead = 4, kRows = 2 * Gm::NT, kHop = Gm::kConsumers / D4;
    const int SH = p.cols << p.kh_shift, d4 = threadIdx.x % D4;
    const float* lse = p.part_lse + static_cast<size_t>(first_seg) * SH;
    const float4* o = reinterpret_cast<const float4*>(p.part_o + static_cast<size_t>(first_seg) * SH * Gm::D) + d4;
#pragma unroll 1
    for (int r0 = threadIdx.x / D4; r0 < SH; r0 += kRows * kHop) {
        float top[kRows], sum[kRows];
        float4 acc[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            top[j] = -CUDART_INF_F;
            sum[j] = 0.f;
            acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int k0 = 0; k0 < nseg; k0 += kAhead) {
            float e[kRows][kAhead];
            float4 y[kRows][kAhead];
#pragma unroll
            for (int j = 0; j < kRows; ++j)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int r = r0 + j * kHop;
                    const size_t at = static_cast<size_t>(k0 + k) * SH + r;
                    const bool in = r < SH && k0 + k < nseg;
                    e[j][k] = in ? __ldcg(lse + at) : -CUDART_INF_F;
                    y[j][k] = in ? __ldcg(o + at * D4) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                float best = top[j];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) best = fmaxf(best, e[j][k]);
                const float back = top[j] == -CUDART_INF_F ? 0.f : fast_exp2(top[j] - best);
                top[j] = best;
                sum[j] *= back;
                acc[j] = make_float4(acc[j].x * back, acc[j].y * back, acc[j].z * back, acc[j].w * back);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    // an empty piece weighs nothing
                    const float w = e[j][k] == -CUDART_INF_F ? 0.f : fast_exp2(e[j][k] - best);
                    sum[j] += w;
                    acc[j] = fma4(w, y[j][k], acc[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int r = r0 + j * kHop;
            const float inv = sum[j] == 0.f ? 0.f : 1.0f / sum[j];
            if (r < SH)
                store_row4(p.out + (row0 + r) * Gm::D + 4 * d4,
                           make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv));
        }
    }
}

template <int D, int BITS, int NG, int NC>
__global__ void __launch_bounds__(QuantGeometry<D, BITS, NG, NC>::kThreads, 1)
quant_attn_kernel(const QuantParams p) {
    using Gm = QuantGeometry<D, BITS, NG, NC>;
    extern __shared__ unsigned char smem_raw[];
    const QuantSmem sm = quant_carve<Gm>(smem_raw);
    // (broadcast, so that the compiler knows it to be the same on every lane)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Gm::kStages; ++s) {
            mbar_init(sm.full + s, 1u);
            mbar_init(sm.empty + s, Gm::WG);
        }
        mbar_init(sm.group, Gm::kConsumers);
        mbar_init(sm.stashed, Gm::W);
        mbar_init(sm.combined, Gm::WG);
        *sm.abort = 0;
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    allow_dependent_launch();

    // ---- schedule
    const int kh_shift = p.kh_shift, kh = 1 << kh_shift, P = p.page_size;
    const int tok = Gm::kStageRows >> kh_shift;  // rows of one KV head in a stage
    {
        const int cap = p.max_pages * P;
        for (int b = threadIdx.x; b < p.B; b += Gm::kThreads) {
            const unsigned raw = __ldg(p.kv_lens + static_cast<size_t>(b) * p.kv_stride);
            const int len = raw > static_cast<unsigned>(cap) ? cap : static_cast<int>(raw);
            sm.seq_len[b] = len;
            sm.seq_prefix[b + 1] = len == 0 ? 0 : ((len + tok - 1) >> (31 - __clz(tok))) + p.unit_pad;
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
    const int N = sm.seq_prefix[p.B] * p.upb;
    const int C = min(static_cast<int>(gridDim.x), N);
    int t0 = 0, t1 = 0;
    QuantSplit split{1, 0};
    if (static_cast<int>(blockIdx.x) < C) {
        split.q = N / C;
        split.r = N - C * split.q;
        t0 = split.first(blockIdx.x);
        t1 = split.first(blockIdx.x + 1);
    }
    const int pe = min(P, tok);                  // rows of one page in a stage
    const int page_shift = 31 - __clz(P), pe_shift = 31 - __clz(pe);
    const int block = pe * Gm::ROW;              // bytes of one (page, head) in a stage

    if (warp >= Gm::W) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Gm::kCopyRegs));
        // ================================================================ copying warp
        const int npg = tok >> pe_shift;         // pages of a stage (<= 32)
        bool ok = true;
        int it = 0;
        const int pw = warp - Gm::W;
        if (pw == 3) {
            // a warp without copies: zero output rows for sequences without rows
            const size_t n = static_cast<size_t>(p.Hq) * p.sq * D / 8;
            for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
                if (sm.seq_len[b] != 0) continue;
                uint4* to = reinterpret_cast<uint4*>(p.out) + b * n;
                for (size_t i = lane; i < n; i += 32) to[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        if (pw >= Gm::kCopyWarps) return;
        it = pw;
        QuantUnit U{};
        int nxt = -1;                            // this lane's page of the warp's next stage
        int t = t0;
        if (t < t1) {
            U = quant_locate(p, sm, t);
            if (t >= U.base + U.nt) {            // a range may begin behind a unit's last stage
                U = quant_next(p, sm, U, t1);
                t = U.base;
            }
        }
        // n stages further: t1 when the range has no more
        auto advance = [&](int n) {
            while (t < t1) {
                const int here = min(t1, U.base + U.nt) - t;
                if (n < here) {
                    t += n;
                    return;
                }
                n -= here;
                U = quant_next(p, sm, U, t1);
                t = U.base;
            }
        };
        auto fetch = [&]() {
            if (t >= t1) return;
            const int slot = ((t - U.base) * tok >> page_shift) + lane;
            const bool in = lane < npg && slot < ((U.len + P - 1) >> page_shift);
            nxt = in ? __ldg(p.block_table + static_cast<size_t>(U.b) * p.max_pages + slot) : -1;
        };
        advance(pw);
        fetch();
        for (; t < t1; it += Gm::kCopyWarps) {
            const int s = it % Gm::kStages;
            const uint32_t ph = (it / Gm::kStages) & 1;
            const int page = nxt, g = U.g, len = U.len, key0 = (t - U.base) * tok;
            advance(Gm::kCopyWarps);
            fetch();                             // arrives while this stage's slot frees
            if (!quant_wait<kNapCopy>(sm.empty + s, ph ^ 1u, sm.abort)) { ok = false; break; }
            const bool good = page >= 0 && page < p.num_pages;
            const unsigned pages = __ballot_sync(0xffffffffu, good);
            unsigned char* dst = sm.stages + s * Gm::kStageBytes;
            if (lane == 0) {
                // plain: every row of the stage counts for every column, in pages of 16 rows or more
                const bool plain = pe >= 16 && __popc(pages) == npg && key0 + tok <= len - (p.causal ? p.sq - 1 : 0);
                sm.stage_len[s] = plain ? -1 : min(tok, len - key0);
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
                for (int k = it - Gm::kCopyWarps; k >= 0 && k >= it - Gm::kStages; k -= Gm::kCopyWarps)
                    if (!mbar_wait(sm.full + (k % Gm::kStages), (k / Gm::kStages) & 1, nullptr, kWaitLimitNs)) {
                        record_error(p.err, kErrDrain);
                        break;
                    }
            }
        }
        return;
    }

    // ==================================================================== consumer warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Gm::kConsumerRegs));
    // Warp w of group w / WG; inside the group: column slice, KV head, share of that head's tiles.
    const int gw = warp % Gm::WG, grp = warp / Gm::WG;
    const int cs = gw & ((1 << p.slices_shift) - 1);
    const int wt = gw >> p.slices_shift, WT = Gm::WG >> p.slices_shift;
    const int head = wt & (kh - 1);
    uint32_t gphase = 0;

    auto unit_row0 = [&](const QuantUnit& U) -> size_t {   // first q / out row of the unit
        return (static_cast<size_t>(U.b) * p.Hkv + U.g * kh) * p.cols;
    };
    QuantUnit U{};
    QuantWarp<Gm> cw;
    uint2 first[Gm::NT][D / 16];        // the first unit's query rows, on their way during the set-up
    cw.lane = lane;
    cw.gq = lane >> 2;
    cw.qd = lane & 3;
    cw.col0 = cs * NC;
    int t = t0;
    if (t < t1) {
        U = quant_locate(p, sm, t);
        if (t >= U.base + U.nt) {
            U = quant_next(p, sm, U, t1);
            t = U.base;
        }
    }
    if (t < t1) {
        cw.fetch_q(p, unit_row0(U) + head * p.cols, first);
    }
    // the second eight rows of a tile: next in the page, or on the next page (8-row pages)
    cw.init(p.sq, pe >= 16 ? 8 * Gm::RB : kh * block, pe >= 16 ? 8 * Gm::PB : kh * block);
    // Tile i of a stage; the places of the warp's first UT tiles never change
    auto place = [&](int i) {
        const int r0 = (i >> kh_shift) * 16;               // first row of the tile
        const int blk = ((r0 >> pe_shift) * kh + head) * block, rr = r0 & (pe - 1);
        return cw.tile_at(blk + rr * Gm::RB, blk + (pe + rr) * Gm::RB, blk + 2 * pe * Gm::RB + rr * Gm::PB);
    };
    typename QuantWarp<Gm>::TileAt own[Gm::TPW][Gm::UT];
#pragma unroll
    for (int j = 0; j < Gm::TPW; ++j)
#pragma unroll
        for (int u = 0; u < Gm::UT; ++u) own[j][u] = place(wt + (j * Gm::UT + u) * WT);
    if (t < t1) cw.set_q(p.scale_log2, first);
    int stage = grp;                    // the group takes every kGroups-th stage of the CTA's range
    uint32_t phase = 0;
    int pend_u[2], pend_first[2], pend_n[2], npend = 0;   // units of which this CTA stored a piece
    size_t pend_row[2];
    int skip = grp;                     // stages until the group's next one
    uint32_t round = 0;                 // segments merged so far
    int done = 0;                       // stages of the range in earlier segments
    while (t < t1) {
        const int tend = min(t1, U.base + U.nt);
        done += tend - t;
        const bool whole = t == U.base && tend == U.base + U.nt;
        // rows a causal column may see: keys up to last + its token; without masking, every row
        const int last = p.causal ? U.len - p.sq : 0x7fffffff;
        cw.reset();
        for (t += skip; t < tend; t += Gm::kGroups) {
            if (!quant_wait<kNapConsumer>(sm.full + stage, phase, sm.abort)) {
                *sm.abort = 1;
                record_error(p.err, kErrWaitFull);
                return;
            }
            const int nvalid = sm.stage_len[stage];
            const unsigned char* base = sm.stages + stage * Gm::kStageBytes;
            auto take = [&](int i, const typename QuantWarp<Gm>::TileAt (&at)[Gm::UT]) {
                uint32_t rows[Gm::UT];
                int key[Gm::UT];
#pragma unroll
                for (int u = 0; u < Gm::UT; ++u) {
                    rows[u] = 0xffffu;
                    key[u] = 0;
                }
                if (nvalid < 0) {
                    cw.template tiles<false>(base, at, rows, key, 0);
                    return;
                }
                const unsigned pages = sm.stage_pages[stage];
                uint32_t any = 0u;
#pragma unroll
                for (int u = 0; u < Gm::UT; ++u) {
                    const int r0 = ((i + u * WT) >> kh_shift) * 16, pg = r0 >> pe_shift;
                    const int n = nvalid - r0;
                    key[u] = (t - U.base) * tok + r0;
                    rows[u] = n >= 16 ? 0xffffu : n > 0 ? (1u << n) - 1u : 0u;
                    if (!((pages >> pg) & 1u)) rows[u] &= pe >= 16 ? 0u : 0xff00u;
                    if (pe < 16 && !((pages >> (pg + 1)) & 1u)) rows[u] &= 0x00ffu;
                    any |= rows[u];
                }
                if (any != 0u) cw.template tiles<true>(base, at, rows, key, last);
            };
#pragma unroll
            for (int j = 0; j < Gm::TPW; ++j) take(wt + j * Gm::UT * WT, own[j]);
            // with the columns split over several warps, each has more tiles
            for (int i = wt + Gm::TPW * Gm::UT * WT; i < Gm::kTiles; i += WT * Gm::UT) {
                typename QuantWarp<Gm>::TileAt at[Gm::UT];
#pragma unroll
                for (int u = 0; u < Gm::UT; ++u) at[u] = place(i + u * WT);
                take(i, at);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.empty + stage);
            stage += Gm::kGroups;
            if (stage >= Gm::kStages) {
                stage -= Gm::kStages;
                phase ^= 1u;
            }
        }
        skip = t - tend;
        t = tend;

        // ---- end of the segment: every warp leaves its columns in its merge slot and goes on to the
        // next unit; the group that took the segment's last stage merges them when all are there (after
        // the CTA's last segment every group takes part: nothing else is left to do).  With all warps
        // waiting for one another here a segment cost 6000 to 7500 cycles of streaming.
        const QuantUnit next = quant_next(p, sm, U, t1);
        t = next.base;
        const bool more = t < t1;
        uint2 raw[Gm::NT][D / 16];          // the next unit's query rows, on their way during the merge
        cw.settle();
        if (round > 0 && !quant_wait<kNapGroup>(sm.combined, (round - 1) & 1, sm.abort)) {
            *sm.abort = 1;
            record_error(p.err, kErrWaitGroup);
            return;
        }
        cw.stash(sm, warp);
        if (more) cw.fetch_q(p, unit_row0(next) + head * p.cols, raw);
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.stashed);
        const size_t row0 = unit_row0(U);
        int first_seg = 0, nseg = 1;
        if (!whole) {
            first_seg = split.owner(U.base) + U.u;
            nseg = split.owner(U.base + U.nt - 1) + U.u - first_seg + 1;
        }
        if (!more || grp == (done - 1) % Gm::kGroups) {
            if (!quant_wait<kNapGroup>(sm.stashed, round & 1, sm.abort)) {
                *sm.abort = 1;
                record_error(p.err, kErrWaitGroup);
                return;
            }
            // Output rows of the unit: (KV head, column); the pieces of one lie in the slots of the warps
            // that shared the head's tiles and hold the column.
            constexpr int D4 = D / 4;
            const int SH = kh * p.cols;
            const size_t seg0 = static_cast<size_t>(static_cast<int>(blockIdx.x) + U.u) * SH;
            const int pieces_shift = p.slices_shift + kh_shift;
            const int KS = (Gm::WG >> pieces_shift) * Gm::kGroups;
            const int tid = more ? gw * 32 + lane : static_cast<int>(threadIdx.x);
            const int hop = (more ? Gm::WG * 32 : Gm::kConsumers) / D4;   // rows between a thread's own
            const int d4 = tid % D4;
            int h = 0, col = tid / D4;
            while (col >= p.cols) { col -= p.cols; ++h; }
#pragma unroll 2
            for (int r = tid / D4; r < SH; r += hop) {
                // slot of piece k: warp (k << pieces_shift) | (h << slices_shift) | slice (a group's
                // warps are a multiple of 1 << pieces_shift), column col % NC
                const int slot0 = ((h << p.slices_shift) | (col / NC)) * NC + col % NC;
                const int step = NC << pieces_shift;
                float pm[Gm::W], top = kQuantUnset;
#pragma unroll
                for (int k = 0; k < Gm::W; ++k) {
                    pm[k] = k < KS ? sm.merge_m[slot0 + k * step] : kQuantUnset;
                    top = fmaxf(top, pm[k]);
                }
                float sum = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < Gm::W; ++k) {
                    if (k >= KS) break;
                    const int slot = slot0 + k * step;
                    const float w = fast_exp2(pm[k] - top);
                    sum += w * sm.merge_l[slot];
                    acc = fma4(w, *reinterpret_cast<const float4*>(
                                      sm.merge_o + slot * Gm::kMergeStride + 4 * d4), acc);
                }
                const float inv = sum == 0.f ? 0.f : 1.0f / sum;   // no row at all: zeros
                const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                if (whole) {
                    store_row4(p.out + (row0 + r) * D + 4 * d4, v);
                } else {
                    *reinterpret_cast<float4*>(p.part_o + (seg0 + r) * D + 4 * d4) = v;
                    if (d4 == 0) p.part_lse[seg0 + r] = sum == 0.f ? -CUDART_INF_F : top + fast_log2(sum);
                }
                col += hop;
                while (col >= p.cols) { col -= p.cols; ++h; }
            }
            __syncwarp();
            if (more && lane == 0) mbar_arrive(sm.combined);
        }
        ++round;
        if (!whole) {                       // at most twice: the range's first and last unit
            const int k = npend++;
            if (k == 0) {
                pend_u[0] = U.u; pend_first[0] = first_seg; pend_n[0] = nseg; pend_row[0] = row0;
            } else {
                pend_u[1] = U.u; pend_first[1] = first_seg; pend_n[1] = nseg; pend_row[1] = row0;
            }
        }
        if (more) cw.set_q(p.scale_log2, raw);
        U = next;
    }

    // ---- count the stored pieces, once after the whole range, and merge the units they complete.
    // The barrier orders every partial store before these releases.
    if (npend == 0) return;
    if (!quant_sync(sm, gphase, p.err)) return;
    if (threadIdx.x < npend) {
        const int k = threadIdx.x;
        const unsigned prev = atomic_add_acq_rel_gpu(p.counters + (k ? pend_u[1] : pend_u[0]));
        sm.last_flag[k] = prev == static_cast<unsigned>((k ? pend_n[1] : pend_n[0]) - 1) ? 1 : 0;
    }
    if (!quant_sync(sm, gphase, p.err)) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k >= npend || !sm.last_flag[k]) continue;
        quant_merge_unit<Gm>(p, pend_row[k], pend_first[k], pend_n[k]);
        if (threadIdx.x == 0) p.counters[pend_u[k]] = 0u;
    }
}

// Launches the instantiation for head dim D and BITS-bit codes: groups = D / group, narrow: at
// most 8 query columns per KV head.
template <int D, int BITS>
cudaError_t launch_quant(int groups, bool narrow, const QuantParams& p, int grid, cudaStream_t st);

// The tcgen05 kernel (quant_tc.cu): one group per row, 33 to 64 query columns per KV head.
cudaError_t launch_quant_tc(int D, int bits, const QuantParams& p, int grid, cudaStream_t st);

template <int D, int BITS, int NG, int NC>
cudaError_t launch_quant_as(const QuantParams& p, int grid, cudaStream_t st) {
    using Gm = QuantGeometry<D, BITS, NG, NC>;
    const void* kernel = reinterpret_cast<const void*>(&quant_attn_kernel<D, BITS, NG, NC>);
    // The consumers' share of registers must be there: a build that gives the launch fewer (other compiler
    // flags) would leave them waiting for it.
    static std::atomic<int> launch_regs{0};
    if (launch_regs.load() == 0) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
        if (e != cudaSuccess) return e;
        launch_regs.store(a.numRegs);
    }
    if (launch_regs.load() != Gm::kLaunchRegs) return cudaErrorInvalidConfiguration;
    void* args[] = {const_cast<QuantParams*>(&p)};
    return launch_configured(kernel, Gm::kSmemBytes, grid, Gm::kThreads, st, args);
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
