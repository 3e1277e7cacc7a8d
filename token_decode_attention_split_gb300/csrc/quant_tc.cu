// Decode attention over the quantised paged cache on the fifth-generation tensor cores (tcgen05), for 33 to
// 64 query columns per KV head and one group per row.  quant_attn.cuh has the other shapes, the formulas and
// the split of the work over CTAs, which are the same here, with one KV head a unit and stages of 64 rows.
//
// Why a second kernel.  The warp MMAs of quant_attn.cuh hold 16 columns, so wider units expand the codes
// once per 16 columns, and their matrix work alone takes 141 ns per 16-row tile and SM at 64 columns (with
// everything else 292).  Here the codes of 64 rows (a tile) are expanded once, into shared memory:
//     S = Q K^T    A: Q in tensor memory (fp16, columns on lanes 0 .. 63), B: K codes, fp16 subnormals
//     O += P V     A: the weights P in tensor memory (over the scores they came from), B: V codes
// V codes are stored less their middle code, as numbers, so O needs no correction.  A thread owns a query
// column (a TMEM lane): its softmax has no exchange between lanes.
//
// Inside a CTA (10 warps; warp w issues on scheduler w % 4 and reaches TMEM lanes 32 (w % 4) .. + 31):
//   warps 0 .. 3    softmax: warps 0 and 1 the first 32 rows of every tile, 32 columns each, warps 2 and 3 the
//                   last 32.  Q stands in lanes 64 .. 127 again, and either half's weights are zero in the
//                   other half's rows, so lanes c and 64 + c of O are two shares of column c; they are put
//                   together at a segment's end
//   warps 4 .. 7    expand the codes and parameters of a stage into an operand buffer; they bring a segment's
//                   query rows to TMEM before its first tile
//   warp 8          TMEM and the MMAs: S of up to three tiles ahead, P V of this one
//   warp 9          bulk copies of pages into a ring of stages
//
// What bounds it.  196 ns per 16-row tile and SM with the cache in L2 (D = 128, 4 bits; HBM needs 48), for
// any number of columns: 1500 cycles per 64 rows, of which the softmax warps work 1100 to 1270 and the
// expanding warps 830 to 1100, each limited by its own latencies (47% of the issue slots, 46% of the integer
// pipe, 56% of shared memory's cycles and 32% of the tensor pipe's are used).  Tried: one pair of softmax
// warps for all rows, 221 ns; pairs for odd and even tiles with an O each, 201, but dearer segment ends;
// eight expanding warps (128 registers a thread), 232; one polling lane a warp with naps, 315.  The MMA
// operands must be uniform values of the whole warp: issued by one diverged lane an MMA took 75 cycles, 25
// so.
//
// Every wait is bounded (about a second) and raises the CTA's abort flag; all warps meet at the end on every
// path, with the MMAs drained, before the tensor memory is freed.
#include "quant_attn.cuh"

#include <type_traits>

namespace da {
namespace {

constexpr int kRows = 64;                        // rows of a stage and of an operand buffer
constexpr int kThreads = 320;
constexpr int kExpand = 4;                       // expanding warps
constexpr int kMaxCols = 64;
constexpr uint32_t kTmemCols = 512;              // Q: 2 x 64 columns, S (and P): 4 x 64, O: 128
constexpr uint32_t kColS = 128, kColO = 384;
constexpr int kScores = 4;                       // S buffers
constexpr int kMaxBuffers = 4, kMaxStages = 8;
constexpr float kRaiseAt = 256.f;                // sum of a tile's p, and any weight

template <int D_, int BITS_>
struct TcQuant {
    static constexpr int D = D_, BITS = BITS_;
    static constexpr int kBuffers = D == 128 && BITS == 8 ? 3 : 4;   // operand buffers
    static constexpr int NT = 2, kConsumers = kThreads;      // for quant_merge_unit: rows ahead, threads
    static constexpr int RB = kQuantRowCodes(D, BITS), PB = kQuantRowParams(D, D);
    static constexpr int ROW = 2 * RB + PB;
    static constexpr int kStageBytes = kRows * ROW;
    static constexpr int kTileBytes = kRows * D * 2;         // one operand
    static constexpr int kParamBytes = 4 * kRows * 4;        // k scale, k min, v scale, v middle
    static constexpr int kMid = BITS == 4 ? 8 : 128;
    static constexpr int kPer = 32 / BITS;                   // codes of a word
    static constexpr int kOffParam = kBuffers * 2 * kTileBytes;
    static constexpr int kRowStride = D / 2 + 4;             // floats between the rows handed over
    static constexpr int kOffHalf = kOffParam + kBuffers * kParamBytes;
    static constexpr int kOffRing = kOffHalf + 2 * kMaxCols * kRowStride * 4;
    static constexpr int kMiscBytes = 3 * 1024;
    static constexpr int kSchedBytes = (2 * kMaxPagedBatch + 2) * 4;
    static constexpr int kFit = (kSmemBudget - 1024 - kOffRing - kMiscBytes - kSchedBytes) / kStageBytes;
    static constexpr int kStages = kFit > kMaxStages ? kMaxStages : kFit;
    static constexpr int kOffMisc = kOffRing + kStages * kStageBytes;
    static constexpr int kOffSched = kOffMisc + kMiscBytes;
    static constexpr int kSmemBytes = 1024 + kOffSched + kSchedBytes;
    static_assert(kStages >= 4 && kStageBytes % 128 == 0 && kSmemBytes <= kSmemBudget, "shared memory");

    // Place of a code in an expanded row: word j of the codes becomes kPer places, pairs of the codes i
    // and i + kPer / 2 (the halves of a masked word).
    __host__ __device__ static constexpr int place(int code) {
        const int j = code / kPer, r = code % kPer;
        return j * kPer + 2 * (r % (kPer / 2)) + r / (kPer / 2);
    }
    // place of element e of a V row
    __host__ __device__ static constexpr int v_place(int e) {
        return place(((e % 16 / 2) * (D / 16) + e / 16) * 2 + e % 2);
    }
    // element of a K row at place n, and whether its code is expanded at 2^-20 instead of 2^-24
    __host__ __device__ static constexpr int k_elem(int n) {
        const int j = n / kPer, r = n % kPer, code = j * kPer + r / 2 + (r % 2) * (kPer / 2);
        return 16 * (code / 4 % (D / 16)) + 4 * (code / (4 * (D / 16))) + code % 4;
    }
    __host__ __device__ static constexpr bool k_high(int n) { return BITS == 4 && (n % kPer / 2) % 2 == 1; }
};

struct TcQuantBars {
    uint64_t full[kMaxStages], empty[kMaxStages];   // ring: copied (bytes) / expanded (expanding warps)
    uint64_t tile_ready[kMaxBuffers];        // operand buffer written (expanding warps)
    uint64_t tile_free[kMaxBuffers];         // its P V done (commit)
    uint64_t s_ready[kScores];               // scores written (commit)
    uint64_t p_ready[kScores];               // weights written (softmax warps)
    uint64_t q_ready[2];                     // query rows in TMEM (their warps)
    uint64_t q_free[2];                      // their scores done (commit), factors read (softmax warps)
    uint64_t half_sums, half_rows;           // a segment's sums / rows handed over (softmax warps)
    uint64_t drain;
    unsigned tile_mask[kMaxBuffers][2];      // rows of the buffer that count
    int stage_len[kMaxStages];
    unsigned stage_pages[kMaxStages];
    uint32_t tmem_base;
    int abort;
    int last_flag[2];
    int npend, pend_u[2], pend_first[2], pend_n[2];
    size_t pend_row[2];
    float q_cf[2][kMaxCols], q_sum[2][kMaxCols];
    float half_m[2][kMaxCols], half_l[2][kMaxCols];
};
static_assert(sizeof(TcQuantBars) <= 3 * 1024, "barrier block");

// kind::f16 with fp16 operands, A K-major (tensor memory), B K-major or MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem]; issued by one thread, runs asynchronously.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// true on one lane of the (whole) warp, the same one every time
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t half2_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Sixteen bytes of codes x as fp16: chunk w of the result is out[w] (4 bits: four chunks, 8 bits: two).
template <int BITS, bool V>
__device__ __forceinline__ uint4 expand(const uint32_t (&x)[4], int w) {
    uint32_t o[4];
    if (BITS == 4) {
        const uint32_t a = x[w], b = a >> 8;
        o[0] = a & 0x000f000fu;
        o[1] = a & 0x00f000f0u;
        o[2] = b & 0x000f000fu;
        o[3] = b & 0x00f000f0u;
        if (V) {
            // under the bits of 1024: 1024 + c, or 1024 + 16 c; less the middle code, exactly
            const __half2 lo = __float2half2_rn(-1032.f), sixteenth = __float2half2_rn(0.0625f),
                          hi = __float2half2_rn(-72.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 y = as_half2(o[i] | 0x64006400u);
                o[i] = half2_bits(i % 2 == 0 ? __hadd2(y, lo) : __hfma2(y, sixteenth, hi));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o[2 * i] = x[2 * w + i] & 0x00ff00ffu;
            o[2 * i + 1] = (x[2 * w + i] >> 8) & 0x00ff00ffu;
        }
        if (V) {
            const __half2 mid = __float2half2_rn(-1152.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = half2_bits(__hadd2(as_half2(o[i] | 0x64006400u), mid));
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Whether the phase with the given parity has completed; the same answer on every lane.
__device__ __forceinline__ bool tc_test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return __all_sync(0xffffffffu, done);
}

// The stages of a CTA's range one after another, with the segment (unit piece) they belong to.
struct TcWalk {
    QuantUnit U;
    int t, seg, start;   // start: the segment's first stage
    __device__ __forceinline__ int end(int t1) const { return min(t1, U.base + U.nt); }
    __device__ __forceinline__ void next_segment(const QuantParams& p, const QuantSmem& sm, int t1) {
        U = quant_next(p, sm, U, t1);
        t = U.base;
        ++seg;
        start = t;
    }
    __device__ __forceinline__ void advance(const QuantParams& p, const QuantSmem& sm, int t1) {
        if (++t >= end(t1)) next_segment(p, sm, t1);
    }
};

// Fills seq_len and seq_prefix; every thread of the CTA calls it.  (The other kernel has these lines in its
// body: as a function of both, its loop lost 15%.)
__device__ __forceinline__ void tc_schedule(const QuantParams& p, const QuantSmem& sm) {
    const int cap = p.max_pages * p.page_size, lane = threadIdx.x & 31;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const unsigned raw = __ldg(p.kv_lens + static_cast<size_t>(b) * p.kv_stride);
        const int len = raw > static_cast<unsigned>(cap) ? cap : static_cast<int>(raw);
        sm.seq_len[b] = len;
        sm.seq_prefix[b + 1] = len == 0 ? 0 : (len + kRows - 1) / kRows + p.unit_pad;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
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
    __syncthreads();
}

// This CTA's range [t0, t1) of the N places.  No more CTAs take part than leaves about kLeast places to each,
// since the one that merges a unit reads 32 KB for each of its pieces (one sequence of 4000 rows and 64
// columns: 48 us in ranges of one place, 22 of four, 20 of eight; of 1000 rows: 20, 15, 17).
__device__ __forceinline__ void tc_range(int N, QuantSplit& split, int& t0, int& t1) {
    constexpr int kLeast = 6;
    const int C = min(static_cast<int>(gridDim.x), (N + kLeast - 1) / kLeast);
    if (static_cast<int>(blockIdx.x) >= C) return;
    split.q = N / C;
    split.r = N - C * split.q;
    t0 = split.first(blockIdx.x);
    t1 = split.first(blockIdx.x + 1);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) quant_tc_kernel(const QuantParams p) {
    using Gm = TcQuant<D, BITS>;
    constexpr int kBuffers = Gm::kBuffers;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TcQuantBars& bar = *reinterpret_cast<TcQuantBars*>(base + Gm::kOffMisc);
    QuantSmem sm{};
    sm.seq_prefix = reinterpret_cast<int*>(base + Gm::kOffSched);
    sm.seq_len = sm.seq_prefix + kMaxPagedBatch + 1;
    volatile int* abort = &bar.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Gm::kStages; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], kExpand);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&bar.tile_ready[i], kExpand);
            mbar_init(&bar.tile_free[i], 1);
        }
        for (int i = 0; i < kScores; ++i) {
            mbar_init(&bar.s_ready[i], 1);
            mbar_init(&bar.p_ready[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_ready[i], 4);
            mbar_init(&bar.q_free[i], 4 + 1);
        }
        mbar_init(&bar.half_sums, 4);
        mbar_init(&bar.half_rows, 4);
        mbar_init(&bar.drain, 1);
        bar.abort = 0;
        bar.npend = 0;
        fence_mbarrier_init();
    }
    if (warp == 8) {
        tmem_alloc(&bar.tmem_base, kTmemCols);
        tmem_relinquish_alloc_permit();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    tc_fence_before_sync();
    tc_schedule(p, sm);      // (two CTA barriers)
    tc_fence_after_sync();
    const uint32_t tmem = bar.tmem_base;
    const int N = sm.seq_prefix[p.B] * p.upb;
    QuantSplit split{1, 0};
    int t0 = 0, t1 = 0;
    tc_range(N, split, t0, t1);
    const int P = p.page_size, pe = min(P, kRows);
    const int page_shift = 31 - __clz(P), pe_shift = 31 - __clz(pe);
    const int block = pe * Gm::ROW;

    TcWalk at{};
    at.t = t0;
    if (t0 < t1) {
        at.U = quant_locate(p, sm, t0);
        if (at.t >= at.U.base + at.U.nt) {       // a range may begin behind a unit's last stage
            at.U = quant_next(p, sm, at.U, t1);
            at.t = at.U.base;
        }
    }
    at.start = at.t;
    auto unit_row0 = [&](const QuantUnit& U) -> size_t {
        return (static_cast<size_t>(U.b) * p.Hkv + U.g) * p.cols;
    };
    bool ok = true;
    uint32_t err = kErrWaitFull;

    if (warp == 9) {
        // ================================================================ copies
        // A lane looks up page lane % 8 of stage lane / 8 of the next four stages of the segment.
        const int npg = kRows >> pe_shift;       // pages of a stage: 1, 2, 4 or 8
        auto fetch = [&](const TcWalk& w) -> int {
            if (w.t >= t1) return -1;
            const int st = lane >> 3, k = lane & 7;
            const int slot = (((w.t + st - w.U.base) * kRows) >> page_shift) + k;
            const bool in = k < npg && w.t + st < w.end(t1) && slot < ((w.U.len + P - 1) >> page_shift);
            return in ? __ldg(p.block_table + static_cast<size_t>(w.U.b) * p.max_pages + slot) : -1;
        };
        int page = fetch(at), n = 0;
        err = kErrWaitEmpty;
        const size_t page_bytes = static_cast<size_t>(P) * Gm::ROW;
        while (ok && at.t < t1) {
            const TcWalk cur = at;
            const int here = min(4, at.end(t1) - at.t);
            at.t += here;
            if (at.t >= at.end(t1)) at.next_segment(p, sm, t1);
            const int mine = page;
            page = fetch(at);                    // arrives while these stages' slots free
            for (int i = 0; i < here; ++i, ++n) {
                const int s = n % Gm::kStages;
                if (!quant_wait<100>(&bar.empty[s], ((n / Gm::kStages) & 1) ^ 1u, abort)) {
                    ok = false;
                    break;
                }
                const bool good = lane >> 3 == i && mine >= 0 && mine < p.num_pages;
                const unsigned pages = (__ballot_sync(0xffffffffu, good) >> (8 * i)) & 0xffu;
                const int key0 = (cur.t + i - cur.U.base) * kRows;
                unsigned char* dst = base + Gm::kOffRing + s * Gm::kStageBytes;
                if (lane == 0) {
                    bar.stage_len[s] = min(kRows, cur.U.len - key0);
                    bar.stage_pages[s] = pages;
                    mbar_arrive_expect_tx(&bar.full[s], __popc(pages) * block);
                }
                __syncwarp();
                if (P <= kRows) {
                    if (good)
                        bulk_load(dst + (lane & 7) * block,
                                  p.pool + (static_cast<size_t>(mine) * p.Hkv + cur.U.g) * page_bytes, block,
                                  &bar.full[s]);
                } else if (pages) {
                    const int pg = __shfl_sync(0xffffffffu, mine, 8 * i), r0 = key0 & (P - 1);
                    const unsigned char* src = p.pool + (static_cast<size_t>(pg) * p.Hkv + cur.U.g) * page_bytes;
                    if (lane < 2)
                        bulk_load(dst + lane * pe * Gm::RB, src + (lane * P + r0) * Gm::RB, pe * Gm::RB,
                                  &bar.full[s]);
                    else if (lane == 2)
                        bulk_load(dst + 2 * pe * Gm::RB, src + 2 * P * Gm::RB + r0 * Gm::PB, pe * Gm::PB,
                                  &bar.full[s]);
                }
                __syncwarp();
            }
        }
        if ((!ok || *abort) && lane == 0) {
            // every copy issued lands before the CTA can exit
            for (int k = n - 1; k >= 0 && k >= n - Gm::kStages; --k)
                if (!mbar_wait(&bar.full[k % Gm::kStages], (k / Gm::kStages) & 1, nullptr, kWaitLimitNs)) {
                    record_error(p.err, kErrDrain);
                    break;
                }
        }
    } else if (warp >= 4 && warp < 8) {
        // ================================================================ expansion
        const int uw = warp - 4, ut = uw * 32 + lane;
        constexpr int CPR = Gm::RB / 16;                     // 16-byte chunks of a row of codes
        constexpr int kTasks = kRows * CPR / (32 * kExpand);
        static_assert(kTasks * 32 * kExpand == kRows * CPR, "shares");
        constexpr int kOut = BITS == 4 ? 4 : 2;              // fp16 chunks of one
        // the segment's query rows, column c on lanes c and 64 + c
        // (brought to fp16 by a power of two as in quant_attn.cuh)
        auto load_q = [&](const TcWalk& w) -> bool {
            const int c = (warp & 1) * 32 + lane, qb = w.seg & 1;
            uint32_t raw[D / 2];
            const uint4* row = reinterpret_cast<const uint4*>(p.q + (unit_row0(w.U) + (c < p.cols ? c : 0)) * D);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint4 y = c < p.cols ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
                raw[4 * i] = y.x;
                raw[4 * i + 1] = y.y;
                raw[4 * i + 2] = y.z;
                raw[4 * i + 3] = y.w;
            }
            __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
#pragma unroll
            for (int i = 0; i < D / 2; ++i)
                top2 = __hmax2(top2, __habs2(*reinterpret_cast<__nv_bfloat162*>(&raw[i])));
            const uint32_t tb = *reinterpret_cast<const uint32_t*>(&top2);
            const uint32_t top = max(tb >> 16, tb & 0xffffu);
            // the largest element goes to [2^14, 2^15) (an infinity stays one, a NaN spoils its row)
            const int ex = min(max(static_cast<int>(top >> 7), 27), 254);
            const float up = __int_as_float((268 - ex) << 23), down = __int_as_float((ex - 14) << 23);
            float sum = 0.f;
            auto elem = [&](int e) {
                return (e % 2 ? bf16_hi_to_f32(raw[e / 2]) : bf16_lo_to_f32(raw[e / 2])) * up;
            };
#pragma unroll
            for (int e = 0; e < D; ++e) sum += elem(e);
            if (!mbar_wait_warp(&bar.q_free[qb], ((w.seg >> 1) & 1) ^ 1u, abort)) return false;
            tc_fence_after_sync();
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint32_t x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int n0 = 64 * h + 2 * i;
                    const float f = Gm::k_high(n0) ? 0.0625f : 1.f;
                    x[i] = pack_f16x2(elem(Gm::k_elem(n0)) * f, elem(Gm::k_elem(n0 + 1)) * f);
                }
                tmem_st32(tmem + (static_cast<uint32_t>((warp - 4) * 32) << 16) + qb * 64 + 32 * h, x);
            }
            tmem_wait_st();
            if (warp < 6) {
                bar.q_cf[qb][c] = p.scale_log2 * down * 16777216.f;
                bar.q_sum[qb][c] = sum * (1.f / 16777216.f);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_ready[qb]);
            return true;
        };
        int n = 0;
        for (TcWalk w = at; w.t < t1; w.advance(p, sm, t1), ++n) {
            if (w.t == w.start && !load_q(w)) {
                ok = false;
                break;
            }
            const int s = n % Gm::kStages, b = n % kBuffers;
            if (!mbar_wait_warp(&bar.full[s], (n / Gm::kStages) & 1, abort) ||
                !mbar_wait_warp(&bar.tile_free[b], ((n / kBuffers) & 1) ^ 1u, abort)) {
                ok = false;
                break;
            }
            const unsigned char* stage = base + Gm::kOffRing + s * Gm::kStageBytes;
            unsigned char* tile = base + b * 2 * Gm::kTileBytes;
            if (uw < 2) {
                const int r = ut, rr = r & (pe - 1);
                const bool in = r < bar.stage_len[s] && ((bar.stage_pages[s] >> (r >> pe_shift)) & 1u);
                const unsigned m = __ballot_sync(0xffffffffu, in);
                uint2 q = make_uint2(0u, 0u);
                if (in)
                    q = *reinterpret_cast<const uint2*>(stage + (r >> pe_shift) * block + 2 * pe * Gm::RB +
                                                        rr * Gm::PB);
                float* par = reinterpret_cast<float*>(base + Gm::kOffParam + b * Gm::kParamBytes);
                par[r] = bf16_lo_to_f32(q.x);
                par[kRows + r] = bf16_hi_to_f32(q.x);
                par[2 * kRows + r] = bf16_lo_to_f32(q.y);
                par[3 * kRows + r] = __fmaf_rn(static_cast<float>(Gm::kMid), bf16_lo_to_f32(q.y),
                                               bf16_hi_to_f32(q.y));
                if (lane == 0) bar.tile_mask[b][uw] = m;
            }
#pragma unroll
            for (int i = 0; i < kTasks; ++i) {
                const int task = ut + 32 * kExpand * i, r = task / CPR, c = task % CPR;
                const unsigned char* src = stage + (r >> pe_shift) * block + (r & (pe - 1)) * Gm::RB + c * 16;
                // the lanes whose results lie in the second half of a row write them in another order, so that
                // the eight of one access fall in different banks
                const int hi = D == 128 ? c / (CPR / 2) : 0;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const uint4 y = *reinterpret_cast<const uint4*>(src + v * pe * Gm::RB);
                    const uint32_t x[4] = {hi ? y.z : y.x, hi ? y.w : y.y, hi ? y.x : y.z, hi ? y.y : y.w};
#pragma unroll
                    for (int k = 0; k < kOut; ++k) {
                        const int j = kOut * c + (k ^ (hi * (kOut / 2)));
                        *reinterpret_cast<uint4*>(tile + v * Gm::kTileBytes + (j >> 3) * (kRows * 128) + r * 128 +
                                                  (((j ^ r) & 7) << 4)) =
                            v ? expand<BITS, true>(x, k) : expand<BITS, false>(x, k);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar.empty[s]);
                mbar_arrive(&bar.tile_ready[b]);
            }
        }
    } else if (warp == 8) {
        // ================================================================ MMAs
        {
            // zero output rows for sequences without rows
            const size_t n = static_cast<size_t>(p.Hq) * p.sq * D / 8;
            for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
                if (sm.seq_len[b] != 0) continue;
                uint4* to = reinterpret_cast<uint4*>(p.out) + b * n;
                for (size_t i = lane; i < n; i += 32) to[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        // The whole warp goes through the loop with values that are the same on every lane (broadcast), so
        // that they can stand in uniform registers, where the MMA takes its operands from; one elected lane
        // issues.
        constexpr uint32_t kIdS = idesc_f16(128, kRows, false), kIdO = idesc_f16(128, D, true);
        auto same = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
        const uint32_t tm = same(tmem), tiles_s = same(smem_u32(base));
        TcWalk ws = at, wp = at;                 // next scores, next P V
        int ns = 0, n = 0;
        uint64_t since = 0, idle0 = 0;            // polls without work, and when they began
        while (wp.t < t1) {
            // Scores of the next tile, if it is there, at most kScores - 1 tiles ahead (its buffer held the
            // weights of tile ns - kScores, whose P V was issued before).
            if (ws.t < t1 && ns < n + kScores &&
                tc_test(&bar.tile_ready[ns % kBuffers], (ns / kBuffers) & 1)) {
                const int sb = ns % kScores, qb = ws.seg & 1;
                // (the tile's expanding warps have brought its query rows before)
                if (ws.t == ws.start && !mbar_wait_warp(&bar.q_ready[qb], (ws.seg >> 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t k_s = same(tiles_s + (ns % kBuffers) * 2 * Gm::kTileBytes),
                               d = same(tm + kColS + sb * kRows), a = same(tm + qb * 64);
                const bool last = ws.t + 1 >= ws.end(t1);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        umma_f16_ts(d, a + ks * 8,
                                    umma_desc_sw128(k_s + (ks >> 2) * (kRows * 128) + (ks & 3) * 32, 16, 1024),
                                    kIdS, ks > 0 ? 1u : 0u);
                    umma_commit(&bar.s_ready[sb]);
                    if (last) umma_commit(&bar.q_free[qb]);
                }
                __syncwarp();
                ws.advance(p, sm, t1);
                ++ns;
                since = 0;
            }
            if (n < ns && tc_test(&bar.p_ready[n % kScores], (n / kScores) & 1)) {
                tc_fence_after_sync();
                const int b = n % kBuffers;
                const uint32_t v_s = same(tiles_s + b * 2 * Gm::kTileBytes + Gm::kTileBytes),
                               a = same(tm + kColS + (n % kScores) * kRows),
                               more = same(wp.t != wp.start ? 1u : 0u);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kRows / 16; ++ks)
                        umma_f16_ts(tm + kColO, a + ks * 8,
                                    umma_desc_sw128(v_s + ks * 16 * 128, kRows * 128, 1024), kIdO,
                                    ks > 0 ? 1u : more);
                    umma_commit(&bar.tile_free[b]);
                }
                __syncwarp();
                wp.advance(p, sm, t1);
                ++n;
                since = 0;
            } else if (++since % 256 == 0) {     // nothing to do: about a second of it ends the wait
                if (since == 256) idle0 = global_timer_ns();
                const bool late = *abort || global_timer_ns() - idle0 > kWaitLimitNs;
                if (__any_sync(0xffffffffu, late)) {
                    ok = false;
                    break;
                }
            }
        }
        if (!ok) *abort = 1;
        // every MMA issued completes before the tensor memory is freed
        if (elect_one()) umma_commit(&bar.drain);
        __syncwarp();
        if (!mbar_wait_warp(&bar.drain, 0, nullptr) && lane == 0) record_error(p.err, kErrDrain);
        __syncwarp();
    } else {
        // ================================================================ softmax and output
        const int half = warp >> 1;              // rows 32 half .. + 31 of every tile
        const int c = (warp & 1) * 32 + lane;    // query column
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const uint32_t t_o = t_lane + kColO;
        const int tok = c % p.sq;
        int n = 0;                               // tile of the range
        uint32_t round = 0;                      // segments before this one
        TcWalk w = at;
        while (ok && w.t < t1) {
            const int tbeg = w.t, tend = w.end(t1);
            const bool whole = tbeg == w.U.base && tend == w.U.base + w.U.nt;
            const int qb = w.seg & 1;
            if (!mbar_wait_warp(&bar.q_ready[qb], (w.seg >> 1) & 1, abort)) {
                ok = false;
                break;
            }
            const float cf = bar.q_cf[qb][c], qs = bar.q_sum[qb][c];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_free[qb]);
            const f2 cf2 = f2_of(cf, cf), qs2 = f2_of(qs, qs);
            float m = kQuantUnset, M = kQuantUnset, f = 1.f, l = 0.f, z = 0.f;
            const int see = p.causal ? w.U.len - p.sq + tok + 1 : 0x7fffffff;   // rows this column may see
            for (int t = tbeg; t < tend; ++t, ++n) {
                const int b = n % kBuffers, sb = n % kScores, key0 = (t - w.U.base) * kRows + 32 * half;
                if (!mbar_wait_warp(&bar.tile_ready[b], (n / kBuffers) & 1, abort) ||
                    !mbar_wait_warp(&bar.s_ready[sb], (n / kScores) & 1, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                // this warp's 32 rows: k scales, k minima, v scales, v middles, four rows a load
                const ulonglong2* par =
                    reinterpret_cast<const ulonglong2*>(base + Gm::kOffParam + b * Gm::kParamBytes) + 8 * half;
                constexpr int kNext = kRows / 4;
                unsigned seen = bar.tile_mask[b][half];
                const bool full = seen == ~0u && (!p.causal || key0 + 32 <= w.U.len - p.sq + 1);
                if (see - key0 < 32) seen &= see > key0 ? (1u << (see - key0)) - 1u : 0u;
                uint32_t pk[16];
                f2 lt, zt;
                __half2 wm;
                auto load_s = [&](uint32_t (&sr)[32]) {
                    tmem_ld32(t_lane + kColS + sb * kRows + 32 * half, sr);
                    tmem_wait_ld();
                };
                auto score = [&](const uint32_t (&sr)[32], int k, f2 ks, f2 kmin, f2 add) {   // rows 2 k, 2 k + 1
                    const f2 s = f2_of(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1]));
                    return f2_fma(f2_fma(kmin, qs2, f2_mul(ks, s)), cf2, add);
                };
                auto pass = [&](auto masked) {
                    constexpr bool kMasked = decltype(masked)::value;
                    const f2 nm = f2_of(-m, -m), f2f = f2_of(f, f);
                    uint32_t sr[32];
                    load_s(sr);
                    lt = f2_of(0.f, 0.f);
                    zt = lt;
                    wm = __float2half2_rn(0.f);
#pragma unroll
                    for (int k4 = 0; k4 < 8; ++k4) {
                        const ulonglong2 ks4 = par[k4], km4 = par[kNext + k4], vs4 = par[2 * kNext + k4],
                                         zv4 = par[3 * kNext + k4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int k = 2 * k4 + i;
                            const f2 x = score(sr, k, i ? ks4.y : ks4.x, i ? km4.y : km4.x, nm);
                            f2 vs = i ? vs4.y : vs4.x, zv = i ? zv4.y : zv4.x;
                            float x0 = f2_get(x, 0), x1 = f2_get(x, 1);
                            if (kMasked) {
                                const bool a = (seen >> (2 * k)) & 1u, e = (seen >> (2 * k + 1)) & 1u;
                                x0 = a ? x0 : -CUDART_INF_F;
                                x1 = e ? x1 : -CUDART_INF_F;
                                vs = f2_of(a ? f2_get(vs, 0) : 0.f, e ? f2_get(vs, 1) : 0.f);
                                zv = f2_of(a ? f2_get(zv, 0) : 0.f, e ? f2_get(zv, 1) : 0.f);
                            }
                            const f2 pr = f2_of(fast_exp2(x0), fast_exp2(x1));
                            lt = f2_add(lt, pr);
                            zt = f2_fma(pr, zv, zt);
                            const f2 wt = f2_mul(f2_mul(pr, vs), f2f);
                            // weights to fp16: half a step, 2^-11
                            pk[k] = pack_f16x2(f2_get(wt, 0), f2_get(wt, 1));
                            wm = __hmax2(wm, as_half2(pk[k]));
                        }
                    }
                };
                for (int attempt = 0;; ++attempt) {
                    if (full) pass(std::false_type{});
                    else pass(std::true_type{});
                    if (attempt) break;
                    const bool over = f2_get(lt, 0) + f2_get(lt, 1) > kRaiseAt ||
                                      fmaxf(__low2float(wm), __high2float(wm)) > kRaiseAt;
                    if (!__any_sync(0xffffffffu, over)) break;
                    // Raise the references to this tile's maxima (at most 126 apart, so that f stays a normal
                    // number), rescale what was summed and weigh the tile again.
                    float mt = m, Mt = M;
                    uint32_t sr[32];
                    load_s(sr);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const f2* pp = reinterpret_cast<const f2*>(par) + k;
                        const f2 x = score(sr, k, pp[0], pp[2 * kNext], f2_of(0.f, 0.f));
                        const f2 vs = pp[4 * kNext];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float y = (seen >> (2 * k + i)) & 1u ? f2_get(x, i) : -CUDART_INF_F;
                            mt = fmaxf(mt, y);
                            Mt = fmaxf(Mt, y + fast_log2(f2_get(vs, i)));
                        }
                    }
                    Mt = fminf(fmaxf(Mt, mt - 126.f), mt + 126.f);
                    const float back = mt == m ? 1.f : fast_exp2(m - mt);
                    l *= back;
                    z *= back;
                    const float ob = Mt == M ? 1.f : fast_exp2(M - Mt);
                    m = mt;
                    M = Mt;
                    f = fast_exp2(m - M);
                    if (t > tbeg && __any_sync(0xffffffffu, ob != 1.f)) {
                        const int last = n - 1;
                        if (!mbar_wait_warp(&bar.tile_free[last % kBuffers], (last / kBuffers) & 1, abort)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int cb = 0; cb < D / 32; ++cb) {
                            uint32_t o[32];
                            tmem_ld32(t_o + cb * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * ob);
                            tmem_st32(t_o + cb * 32, o);
                        }
                        tmem_wait_st();
                    }
                }
                if (!ok) break;
                l += f2_get(lt, 0) + f2_get(lt, 1);
                z += f2_get(zt, 0) + f2_get(zt, 1);
                {
                    // the other half's rows weigh nothing here
                    uint32_t x[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] = half ? 0u : pk[i];
                        x[16 + i] = half ? pk[i] : 0u;
                    }
                    tmem_st32(t_lane + kColS + sb * kRows, x);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready[sb]);
            }
            if (!ok) break;
            // ---- the segment's rows: the two halves' shares put together, either warp of a column half the
            // elements
            bar.half_m[half][c] = m;
            bar.half_l[half][c] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.half_sums);
            const int last = n - 1;
            if (!mbar_wait_warp(&bar.tile_free[last % kBuffers], (last / kBuffers) & 1, abort) ||
                !mbar_wait_warp(&bar.half_sums, round & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const float m1 = bar.half_m[1 - half][c], l1 = bar.half_l[1 - half][c], top = fmaxf(m, m1);
            const float wa = l == 0.f ? 0.f : fast_exp2(m - top), wb = l1 == 0.f ? 0.f : fast_exp2(m1 - top);
            const float total = half ? l1 * wb + l * wa : l * wa + l1 * wb;
            const float mine = total == 0.f ? 0.f : wa / total;      // no row at all: zeros
            const float a = fast_exp2(M - m) * mine, zz = z * mine;
            constexpr int C = D / 64, kRun = 512 / D;    // 32-place chunks of either warp, elements of a run
            // chunk cb holds elements 16 i + kRun cb .. + kRun - 1
            auto chunk = [&](int cb, uint32_t (&o)[32]) {
                tmem_ld32(t_o + cb * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)             // (no row: the accumulator may hold anything)
                    o[j] = l == 0.f ? 0u : __float_as_uint(__fmaf_rn(__uint_as_float(o[j]), a, zz));
            };
            auto run4 = [&](const uint32_t (&o)[32], int i, int e) {
                return make_float4(__uint_as_float(o[Gm::v_place(16 * i + e)]),
                                   __uint_as_float(o[Gm::v_place(16 * i + e + 1)]),
                                   __uint_as_float(o[Gm::v_place(16 * i + e + 2)]),
                                   __uint_as_float(o[Gm::v_place(16 * i + e + 3)]));
            };
            float* rows = reinterpret_cast<float*>(base + Gm::kOffHalf) + c * Gm::kRowStride;
            float4* give = reinterpret_cast<float4*>(rows + (1 - half) * kMaxCols * Gm::kRowStride);
            const float4* take = reinterpret_cast<const float4*>(rows + half * kMaxCols * Gm::kRowStride);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                uint32_t o[32];
                chunk((1 - half) * C + j, o);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < kRun; e += 4) give[(i * C * kRun + j * kRun + e) / 4] = run4(o, i, e);
            }
            uint32_t o[C][32];
#pragma unroll
            for (int j = 0; j < C; ++j) chunk(half * C + j, o[j]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.half_rows);
            if (!mbar_wait_warp(&bar.half_rows, round & 1, abort)) {
                ok = false;
                break;
            }
            const size_t row0 = unit_row0(w.U);
            int first_seg = 0, nseg = 1;
            if (!whole) {
                first_seg = split.owner(w.U.base) + w.U.u;
                nseg = split.owner(w.U.base + w.U.nt - 1) + w.U.u - first_seg + 1;
            }
            const size_t seg = static_cast<size_t>(static_cast<int>(blockIdx.x) + w.U.u) * p.cols + c;
            if (c < p.cols) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int j = 0; j < C; ++j)
#pragma unroll
                        for (int e = 0; e < kRun; e += 4) {
                            const float4 x = run4(o[j], i, e), y = take[(i * C * kRun + j * kRun + e) / 4];
                            const float4 v = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                            const int el = 16 * i + kRun * (half * C + j) + e;
                            if (whole) store_row4(p.out + (row0 + c) * D + el, v);
                            else *reinterpret_cast<float4*>(p.part_o + seg * D + el) = v;
                        }
                if (!whole && half == 0)
                    p.part_lse[seg] = total == 0.f ? -CUDART_INF_F : top + fast_log2(total);
            }
            if (!whole && threadIdx.x == 0) {
                const int k = bar.npend++;       // at most two: the range's first and last unit
                bar.pend_u[k] = w.U.u;
                bar.pend_first[k] = first_seg;
                bar.pend_n[k] = nseg;
                bar.pend_row[k] = row0;
            }
            // (O is read before the next P V overwrites it: the fence of the next weights' arrival)
            ++round;
            w.next_segment(p, sm, t1);
        }
    }
    if (!ok) {
        *abort = 1;
        if (lane == 0) record_error(p.err, err);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 8) tmem_dealloc(tmem, kTmemCols);
    const int npend = bar.npend;
    if (npend == 0 || *abort) return;
    // ---- count the stored pieces and merge the units they complete (the barrier above orders every
    // partial store before these releases)
    if (threadIdx.x < npend) {
        const int k = threadIdx.x;
        const unsigned prev = atomic_add_acq_rel_gpu(p.counters + bar.pend_u[k]);
        bar.last_flag[k] = prev == static_cast<unsigned>(bar.pend_n[k] - 1) ? 1 : 0;
    }
    __syncthreads();
    for (int k = 0; k < npend; ++k) {
        if (!bar.last_flag[k]) continue;
        quant_merge_unit<Gm>(p, bar.pend_row[k], bar.pend_first[k], bar.pend_n[k]);
        if (threadIdx.x == 0) p.counters[bar.pend_u[k]] = 0u;
    }
}

template <int D, int BITS>
cudaError_t launch_as(const QuantParams& p, int grid, cudaStream_t st) {
    void* args[] = {const_cast<QuantParams*>(&p)};
    return launch_configured(reinterpret_cast<const void*>(&quant_tc_kernel<D, BITS>),
                             TcQuant<D, BITS>::kSmemBytes, grid, kThreads, st, args);
}

}  // namespace

cudaError_t launch_quant_tc(int D, int bits, const QuantParams& p, int grid, cudaStream_t st) {
    if (D == 64) return bits == 4 ? launch_as<64, 4>(p, grid, st) : launch_as<64, 8>(p, grid, st);
    return bits == 4 ? launch_as<128, 4>(p, grid, st) : launch_as<128, 8>(p, grid, st);
}

}  // namespace da
