// Writing and reading the quantised paged cache (layout: quant_format.h).
//   decode_attn_append_paged_quant  new bf16 rows are quantised into their slots.
//   decode_attn_read_paged_quant    the rows of given slots come back as bf16.
// Both move each byte once and are bound by memory (append: 4 D bytes in per row and KV head, the
// quantised row out; read: the reverse) and, for a few rows, by the latency of one launch.  A row
// of codes is D * bits / 32 words; that many lanes of a warp take one (row, KV head), each lane
// one word of the stored K row and the same word of the stored V row, gathering the bf16 elements
// that the stored order puts there (pieces of 8 and 4 bytes; the lanes of one instruction cover
// whole 32-byte sectors).
//
// Quantisation of a group of `group` elements x (all arithmetic fp32):
//     min = smallest x (+0 for -0), range = largest x - min
//     scale = range / (2^bits - 1) rounded up to bf16; 0 when that is below 2^-126
//     code = (x - min) / scale rounded to the nearest integer, ties to even; 0 when scale is 0
// bf16 holds min exactly (it is one of the inputs), and a scale rounded up keeps every code in
// range and every error within scale / 2.  A group with a NaN or an infinity (or a range past the
// largest fp32) gets NaN for both parameters, so it reads as NaN throughout, never as numbers.
//
// The nearest code without a division per element: inv = 1 / scale rounded toward zero, and
//     k0  = x' * inv rounded to an integer           (x' = x - min)
//     res = x' - k0 * scale                          (exact: both have few bits)
//     code = (k0 + res * inv) rounded to an integer
// scale has 8 significant bits, so x' / scale is an exact tie k + 1/2 or (unless x' needs all its
// 24 bits) more than 2^-22 away from one, and only exact ties need care: there inv <= 1 / scale
// makes k0 the lower (or the even) neighbour, k0 + res * inv rounds to exactly k0 + 1/2 for
// k0 >= 1 and stays at most 1/2 for k0 = 0, and the last rounding takes the even neighbour.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decode_attn.h"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "quant_format.h"

namespace {

using da::f2;
using da::f2_add;
using da::f2_fma;
using da::f2_get;
using da::f2_of;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct CacheArgs {
    const __nv_bfloat16* k_new;   // append: rows [T] of [Hkv, D], k_stride / v_stride elements apart
    const __nv_bfloat16* v_new;
    int64_t k_stride, v_stride;
    __nv_bfloat16* k_out;         // read: [T, Hkv, D]
    __nv_bfloat16* v_out;
    unsigned char* pool;
    const int64_t* slots;
    int64_t rows;                 // T
    int64_t num_slots;
    int Hkv;
    int span;                     // KV heads that a warp takes of a row
    int parts;                    // pieces of span heads in a row
    int page_shift, page_size;
    int page_bytes;
};

// Adding and subtracting 1.5 * 2^23 rounds a number below 2^22 to an integer (ties to even); the
// sum's low bits are that integer.
constexpr float kRound = 12582912.0f;
constexpr uint32_t kRoundBits = 0x4b400000u;

// The largest float at or below 1 / s, for a normal s below 2^126: an approximate reciprocal, one
// Newton step, and a step of one unit down where the (exactly signed) residual says it is above.
__device__ __forceinline__ float below_reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = __fmaf_rn(r, __fmaf_rn(-s, r, 1.0f), r);
    return __fmaf_rn(-s, r, 1.0f) < 0.f ? __uint_as_float(__float_as_uint(r) - 1u) : r;
}

template <int D, int BITS>
struct RowShape {
    static constexpr int kWords = D * BITS / 32;          // words of a stored row = lanes per row
    static constexpr int kPer = 32 / BITS;                // codes per word
    static constexpr int S = D / 16;                      // 16-element slices
    static constexpr int kRowsPerWarp = 32 / kWords;
    // Element of the first code of stored word j.  A word holds quads (K) or pairs (V) of consecutive
    // 16-element slices of one lane part, so its i-th quad or pair lies 16 i elements further.
    __device__ static int k_elem(int j) {
        const int quad = j * (kPer / 4);
        return 16 * (quad % S) + 4 * (quad / S);
    }
    __device__ static int v_elem(int j) {
        const int pair = j * (kPer / 2);
        return 16 * (pair % S) + 2 * (pair / S);
    }
};

// Reads the kPer elements of stored word j of a bf16 row as raw bits (K: runs of 4 elements, V: of 2).
template <int D, int BITS, bool V>
__device__ __forceinline__ void load_elems(const __nv_bfloat16* row, int j,
                                           uint32_t (&x)[RowShape<D, BITS>::kPer / 2]) {
    using R = RowShape<D, BITS>;
    if (V) {
#pragma unroll
        for (int i = 0; i < R::kPer / 2; ++i)
            x[i] = __ldg(reinterpret_cast<const uint32_t*>(row + R::v_elem(j) + 16 * i));
    } else {
#pragma unroll
        for (int i = 0; i < R::kPer / 4; ++i) {
            const uint2 y = __ldg(reinterpret_cast<const uint2*>(row + R::k_elem(j) + 16 * i));
            x[2 * i] = y.x;
            x[2 * i + 1] = y.y;
        }
    }
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
    return *reinterpret_cast<__nv_bfloat162*>(&x);
}

// Quantises stored word j of one row; the kWords lanes of the row call it together.  Returns the
// packed codes; par[q] = scale | min << 16 (bf16 bits) of each group that this lane's word touches.
template <int D, int BITS, int GROUP, bool V>
__device__ __forceinline__ uint32_t quantise_word(
    const uint32_t (&x)[RowShape<D, BITS>::kPer / 2], uint32_t (&par)[2]) {
    using R = RowShape<D, BITS>;
    // 16-element slices with elements in one word, and 32-element groups
    constexpr int kSlices = V ? R::kPer / 2 : R::kPer / 4;      // 4 (V 4-bit), 2, 2, 1
    constexpr int kQ = (kSlices >= 4 && GROUP == 32) ? 2 : 1;   // groups of this word
    constexpr int kX = R::kPer / 2 / kQ;                        // bf16 pairs per group of the word
    uint32_t packed = 0;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        __nv_bfloat162 lo = as_bf162(x[q * kX]), hi = lo;
#pragma unroll
        for (int i = 1; i < kX; ++i) {
            lo = __hmin2_nan(lo, as_bf162(x[q * kX + i]));
            hi = __hmax2_nan(hi, as_bf162(x[q * kX + i]));
        }
        // The lanes that share the group: stored words are [lane part][slice part]; a group takes
        // every lane part and GROUP / 16 slices, kSlices of them in each word.
        constexpr int kWordsPerPart = R::S / kSlices;           // words of one lane part
        constexpr int kGroupWords = GROUP / 16 >= kSlices ? GROUP / 16 / kSlices : 1;
        auto fold = [&](int off) {
            uint32_t l = *reinterpret_cast<uint32_t*>(&lo), h = *reinterpret_cast<uint32_t*>(&hi);
            l = __shfl_xor_sync(0xffffffffu, l, off);
            h = __shfl_xor_sync(0xffffffffu, h, off);
            lo = __hmin2_nan(lo, as_bf162(l));
            hi = __hmax2_nan(hi, as_bf162(h));
        };
#pragma unroll
        for (int off = 1; off < kGroupWords; off *= 2) fold(off);
#pragma unroll
        for (int off = kWordsPerPart; off < R::kWords; off *= 2) fold(off);
        const float mn = __bfloat162float(__hmin_nan(lo.x, lo.y)) + 0.0f;
        const float mx = __bfloat162float(__hmax_nan(hi.x, hi.y));
        const float range = mx - mn;
        const bool fine = range <= 3.4028234e38f;               // false for NaN and infinity
        // range / (2^bits - 1), correctly rounded (Markstein: one residual correction with a correctly
        // rounded reciprocal of the constant)
        constexpr float kMax = static_cast<float>((1 << BITS) - 1), kInv = 1.0f / kMax;
        const float s0 = range * kInv;
        float s = __fmaf_rn(__fmaf_rn(-kMax, s0, range), kInv, s0);
        s = __uint_as_float((__float_as_uint(s) + 0xffffu) & 0xffff0000u);
        if (!fine || s < 1.17549435e-38f) s = 0.f;
        par[q] = fine ? (__float_as_uint(s) >> 16) | (__float_as_uint(mn) & 0xffff0000u)
                      : 0x7fc07fc0u;
        const float inv = s > 0.f ? below_reciprocal(s) : 0.f;
        const float base = fine ? mn : 0.f;
        const f2 inv2 = f2_of(inv, inv), down = f2_of(-base, -base), minus = f2_of(-s, -s);
        const f2 up = f2_of(kRound, kRound), back = f2_of(-kRound, -kRound);
        uint32_t word = 0;     // sum of (kRoundBits + code) << position, modulo 2^32
        uint32_t bias = 0;     // the kRoundBits in it
#pragma unroll
        for (int i = kX - 1; i >= 0; --i) {
            const uint32_t w = x[q * kX + i];
            const f2 d = f2_add(f2_of(da::bf16_lo_to_f32(w), da::bf16_hi_to_f32(w)), down);
            const f2 k0 = f2_add(f2_fma(d, inv2, up), back);
            const f2 res = f2_fma(k0, minus, d);
            const f2 c = f2_add(f2_fma(res, inv2, k0), up);
            word = (word * (1u << BITS) + __float_as_uint(f2_get(c, 1))) * (1u << BITS) +
                   __float_as_uint(f2_get(c, 0));
            bias = (bias * (1u << BITS) + kRoundBits) * (1u << BITS) + kRoundBits;
        }
        packed |= (fine ? word - bias : 0u) << (q * kX * 2 * BITS);
    }
    if (kQ == 1) par[1] = par[0];
    return packed;
}

// Where stored word j of a row lies among its row's lanes and groups.
template <int D, int BITS, int GROUP, bool V>
struct WordPlace {
    using R = RowShape<D, BITS>;
    static constexpr int kSlices = V ? R::kPer / 2 : R::kPer / 4;
    static constexpr int kWordsPerPart = R::S / kSlices;
    static constexpr int kQ = (kSlices >= 4 && GROUP == 32) ? 2 : 1;
    static constexpr int kGroupWords = GROUP / 16 >= kSlices ? GROUP / 16 / kSlices : 1;
    // first group of word j, and whether its lane stores that group's parameters
    __device__ static int group(int j) { return (j % kWordsPerPart) * kSlices * 16 / GROUP; }
    __device__ static bool stores(int j) {
        return j < kWordsPerPart && (j % kGroupWords) == 0;
    }
};

// Block of KV head 0 of the page of slot w, and the row in it; null where the slot says to skip it.
__device__ __forceinline__ unsigned char* slot_block(const CacheArgs& a, int64_t w, int& row) {
    if (w < 0 || w >= a.num_slots) return nullptr;
    row = static_cast<int>(w & (a.page_size - 1));
    return a.pool + (w >> a.page_shift) * a.Hkv * a.page_bytes;
}

// Work of both kernels: a unit is `span` KV heads of one row, a warp takes one unit after another;
// 32 / kWords heads go through the warp at a time, so many times, with the loads of all steps in flight
// together.  The writer issues about 150 instructions per (row, KV head), a third of them for the groups'
// minima, maxima and scales, and is bound by issue and the latency of its first loads; it is fastest with
// two steps and twice the CTAs that fit, so that new ones load while old ones compute (8192 rows of 8
// heads in groups of 32, with the rows read back: 21.9 us; four steps 24.5, one step 24.4, a grid of
// resident CTAs 25.1).  The reader is bound by memory: four steps on a resident grid (131071 rows of 8
// heads: 109.6 us, 6.28 TB/s; two steps 116.5, twice the CTAs 115.2).
constexpr int kCtasPerSm = 4;
constexpr int kReadSteps = 4, kAppendSteps = 2;
constexpr int kReadWaves = 1, kAppendWaves = 2;

template <int D, int BITS, int GROUP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) quant_append_kernel(const CacheArgs a) {
    using R = RowShape<D, BITS>;
    using PK = WordPlace<D, BITS, GROUP, false>;
    using PV = WordPlace<D, BITS, GROUP, true>;
    constexpr int RB = da::kQuantRowCodes(D, BITS), PB = da::kQuantRowParams(D, GROUP);
    constexpr int X = R::kPer / 2;
    da::grid_dependency_wait();
    da::allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int j = lane % R::kWords, sub = lane / R::kWords;
    const int64_t units = a.rows * a.parts;
    // everything that decides the trip counts is the same on every lane of a warp (the shuffles need
    // all of them)
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
         u += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = a.parts == 1 ? u : u / a.parts;
        const int h0 = static_cast<int>(u - t * a.parts) * a.span;
        const int h1 = min(h0 + a.span, a.Hkv);
        const int64_t slot = a.slots[t];
        const __nv_bfloat16* kr = a.k_new + t * a.k_stride;
        const __nv_bfloat16* vr = a.v_new + t * a.v_stride;
        uint32_t xk[kAppendSteps][X], xv[kAppendSteps][X];
#pragma unroll
        for (int i = 0; i < kAppendSteps; ++i) {
            const int h = min(h0 + i * R::kRowsPerWarp + sub, h1 - 1);
            if (h0 + i * R::kRowsPerWarp >= h1) break;
            load_elems<D, BITS, false>(kr + h * D, j, xk[i]);
            load_elems<D, BITS, true>(vr + h * D, j, xv[i]);
        }
        int row = 0;
        unsigned char* page = slot_block(a, slot, row);
        if (page == nullptr) continue;
#pragma unroll
        for (int i = 0; i < kAppendSteps; ++i) {
            const int h = h0 + i * R::kRowsPerWarp + sub;
            if (h0 + i * R::kRowsPerWarp >= h1) break;
            uint32_t pk[2], pv[2];
            const uint32_t ck = quantise_word<D, BITS, GROUP, false>(xk[i], pk);
            const uint32_t cv = quantise_word<D, BITS, GROUP, true>(xv[i], pv);
            if (h >= h1) continue;
            unsigned char* block = page + h * a.page_bytes;
            *reinterpret_cast<uint32_t*>(block + row * RB + 4 * j) = ck;
            *reinterpret_cast<uint32_t*>(block + (a.page_size + row) * RB + 4 * j) = cv;
            unsigned char* par = block + 2 * a.page_size * RB + row * PB;
            if (PK::stores(j)) *reinterpret_cast<uint32_t*>(par + 8 * PK::group(j)) = pk[0];
            if (PV::stores(j)) {
#pragma unroll
                for (int q = 0; q < PV::kQ; ++q)
                    *reinterpret_cast<uint32_t*>(par + 8 * (PV::group(j) + q) + 4) = pv[q];
            }
        }
    }
}

// The bf16 values of stored word w; par: scale | min << 16 of the group (or two) of its codes.
template <int D, int BITS, int GROUP, bool V>
__device__ __forceinline__ void restore_word(uint32_t w, const uint32_t (&par)[2],
                                             uint32_t (&x)[RowShape<D, BITS>::kPer / 2]) {
    using R = RowShape<D, BITS>;
    using P = WordPlace<D, BITS, GROUP, V>;
    constexpr int kX = R::kPer / 2 / P::kQ;
    const f2 back = f2_of(-8388608.f, -8388608.f);
    // even and odd codes of a 4-bit word as bytes; a byte permute under the bits of 2^23 makes floats
    const uint32_t even = BITS == 4 ? w & 0x0f0f0f0fu : w;
    const uint32_t odd = BITS == 4 ? (w >> 4) & 0x0f0f0f0fu : w;
#pragma unroll
    for (int q = 0; q < P::kQ; ++q) {
        const float s = da::bf16_lo_to_f32(par[q]), mn = da::bf16_hi_to_f32(par[q]);
        const f2 s2 = f2_of(s, s), mn2 = f2_of(mn, mn);
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int pair = q * kX + i;
            const uint32_t lo = __byte_perm(even, 0x4b000000u, 0x7440 | (BITS == 4 ? pair : 2 * pair));
            const uint32_t hi = __byte_perm(odd, 0x4b000000u, 0x7440 | (BITS == 4 ? pair : 2 * pair + 1));
            const f2 c = f2_add(f2_of(__uint_as_float(lo), __uint_as_float(hi)), back);
            const f2 v = f2_fma(s2, c, mn2);
            x[pair] = da::pack_bf16x2(f2_get(v, 0), f2_get(v, 1));
        }
    }
}

template <int D, int BITS, int GROUP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) quant_read_kernel(const CacheArgs a) {
    using R = RowShape<D, BITS>;
    using PK = WordPlace<D, BITS, GROUP, false>;
    using PV = WordPlace<D, BITS, GROUP, true>;
    constexpr int RB = da::kQuantRowCodes(D, BITS), PB = da::kQuantRowParams(D, GROUP);
    constexpr int X = R::kPer / 2;
    da::grid_dependency_wait();
    da::allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int j = lane % R::kWords, sub = lane / R::kWords;
    const int64_t units = a.rows * a.parts, stride = static_cast<int64_t>(gridDim.x) * kWarps;
    int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (u >= units) return;
    int64_t t = a.parts == 1 ? u : u / a.parts;
    int64_t slot = a.slots[t];
    while (true) {
        const int h0 = static_cast<int>(u - t * a.parts) * a.span;
        const int h1 = min(h0 + a.span, a.Hkv);
        int row = 0;
        const unsigned char* page = slot_block(a, slot, row);
        uint32_t ck[kReadSteps], cv[kReadSteps], pk[kReadSteps][2], pv[kReadSteps][2];
#pragma unroll
        for (int i = 0; i < kReadSteps; ++i) {
            ck[i] = cv[i] = pk[i][0] = pk[i][1] = pv[i][0] = pv[i][1] = 0u;   // a skipped row: zeros
            const int h = h0 + i * R::kRowsPerWarp + sub;
            if (page == nullptr || h >= h1) continue;
            const unsigned char* block = page + h * a.page_bytes;
            const unsigned char* par = block + 2 * a.page_size * RB + row * PB;
            ck[i] = __ldg(reinterpret_cast<const uint32_t*>(block + row * RB + 4 * j));
            cv[i] = __ldg(reinterpret_cast<const uint32_t*>(block + (a.page_size + row) * RB + 4 * j));
            pk[i][0] = __ldg(reinterpret_cast<const uint32_t*>(par + 8 * PK::group(j)));
#pragma unroll
            for (int q = 0; q < PV::kQ; ++q)
                pv[i][q] = __ldg(reinterpret_cast<const uint32_t*>(par + 8 * (PV::group(j) + q) + 4));
        }
        // the next unit's slot travels while this one is restored
        const int64_t un = u + stride;
        const int64_t tn = un < units ? (a.parts == 1 ? un : un / a.parts) : t;
        slot = a.slots[tn];
        __nv_bfloat16* ko = a.k_out + t * a.Hkv * D;
        __nv_bfloat16* vo = a.v_out + t * a.Hkv * D;
#pragma unroll
        for (int i = 0; i < kReadSteps; ++i) {
            const int h = h0 + i * R::kRowsPerWarp + sub;
            if (h >= h1) continue;
            uint32_t xk[X], xv[X];
            restore_word<D, BITS, GROUP, false>(ck[i], pk[i], xk);
            restore_word<D, BITS, GROUP, true>(cv[i], pv[i], xv);
#pragma unroll
            for (int e = 0; e < R::kPer / 4; ++e)
                *reinterpret_cast<uint2*>(ko + h * D + R::k_elem(j) + 16 * e) =
                    make_uint2(xk[2 * e], xk[2 * e + 1]);
#pragma unroll
            for (int e = 0; e < X; ++e)
                *reinterpret_cast<uint32_t*>(vo + h * D + R::v_elem(j) + 16 * e) = xv[e];
        }
        if (un >= units) break;
        u = un;
        t = tn;
    }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

using Kernel = void (*)(const CacheArgs);

template <bool READ, int D, int BITS>
Kernel pick_group(int group) {
    switch (group) {
        case 32: return READ ? quant_read_kernel<D, BITS, 32> : quant_append_kernel<D, BITS, 32>;
        case 64: return READ ? quant_read_kernel<D, BITS, 64> : quant_append_kernel<D, BITS, 64>;
        default:
            if constexpr (D == 128)
                return READ ? quant_read_kernel<D, BITS, 128> : quant_append_kernel<D, BITS, 128>;
            return nullptr;
    }
}

template <bool READ>
Kernel pick(int D, int bits, int group) {
    if (D == 64) return bits == 4 ? pick_group<READ, 64, 4>(group) : pick_group<READ, 64, 8>(group);
    return bits == 4 ? pick_group<READ, 128, 4>(group) : pick_group<READ, 128, 8>(group);
}

da_status check(const void* pool, const int64_t* slots, int64_t T, int Hkv, int D, int page_size,
                int64_t num_pages, int bits, int group) {
    if (!pool || !slots || !aligned(pool, 16) || !aligned(slots, 8)) return DA_ERR_INVALID_ARGUMENT;
    if (T < 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0) return DA_ERR_INVALID_ARGUMENT;
    if (!da::quant_format_ok(D, page_size, bits, group)) return DA_ERR_UNSUPPORTED;
    // keeps rows * heads * elements and pages * heads * bytes inside 63 bits
    if (T >= (1ll << 40) || num_pages >= (1ll << 31) || Hkv >= (1 << 12)) return DA_ERR_UNSUPPORTED;
    return DA_OK;
}

da_status launch(Kernel kernel, bool read, CacheArgs& a, void* pool, const int64_t* slots, int64_t T, int Hkv,
                 int D, int page_size, int64_t num_pages, int bits, int group, void* stream) {
    if (T == 0) return DA_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return DA_ERR_CUDA;
    a.pool = static_cast<unsigned char*>(pool);
    a.slots = slots;
    a.rows = T;
    a.num_slots = num_pages * page_size;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.page_shift = 0;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.page_bytes = page_size * da::kQuantRowBytes(D, bits, group);
    const int steps = read ? kReadSteps : kAppendSteps;
    // Heads of a unit: all that the kernel's steps cover, unless that leaves SMs without a warp of
    // their own (few rows: the heads of a row then go to more warps).
    const int at_once = 32 / (D * bits / 32);
    a.span = steps * at_once;
    if (T * ((Hkv + a.span - 1) / a.span) < sms) a.span = at_once;
    a.parts = (Hkv + a.span - 1) / a.span;
    const int64_t want = (T * a.parts + kWarps - 1) / kWarps;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t most = static_cast<int64_t>(kCtasPerSm) * (read ? kReadWaves : kAppendWaves) * sms;
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const CacheArgs>(a)) == cudaSuccess
               ? DA_OK
               : DA_ERR_CUDA;
}

}  // namespace

extern "C" size_t decode_attn_quant_page_bytes(int D, int page_size, int bits, int group) {
    if (!da::quant_format_ok(D, page_size, bits, group)) return 0;
    return static_cast<size_t>(page_size) * da::kQuantRowBytes(D, bits, group);
}

extern "C" da_status decode_attn_append_paged_quant(
    const void* k_new, const void* v_new, int64_t k_row_stride, int64_t v_row_stride, void* pool,
    const int64_t* slot_mapping, int64_t T, int Hkv, int D, int page_size, int64_t num_pages,
    int bits, int group, void* stream) {
    const da_status st = check(pool, slot_mapping, T, Hkv, D, page_size, num_pages, bits, group);
    if (st != DA_OK) return st;
    if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16)) return DA_ERR_INVALID_ARGUMENT;
    const int64_t row = static_cast<int64_t>(Hkv) * D;
    if (k_row_stride < row || v_row_stride < row) return DA_ERR_INVALID_ARGUMENT;
    if (k_row_stride % 8 != 0 || v_row_stride % 8 != 0) return DA_ERR_UNSUPPORTED;
    if (T > 0 && (k_row_stride > (1ll << 61) / T || v_row_stride > (1ll << 61) / T))
        return DA_ERR_UNSUPPORTED;
    CacheArgs a{};
    a.k_new = static_cast<const __nv_bfloat16*>(k_new);
    a.v_new = static_cast<const __nv_bfloat16*>(v_new);
    a.k_stride = k_row_stride;
    a.v_stride = v_row_stride;
    return launch(pick<false>(D, bits, group), false, a, pool, slot_mapping, T, Hkv, D, page_size,
                  num_pages, bits, group, stream);
}

extern "C" da_status decode_attn_read_paged_quant(const void* pool, const int64_t* slot_mapping,
                                                  void* k_out, void* v_out, int64_t T, int Hkv,
                                                  int D, int page_size, int64_t num_pages, int bits,
                                                  int group, void* stream) {
    const da_status st = check(pool, slot_mapping, T, Hkv, D, page_size, num_pages, bits, group);
    if (st != DA_OK) return st;
    if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return DA_ERR_INVALID_ARGUMENT;
    CacheArgs a{};
    a.k_out = static_cast<__nv_bfloat16*>(k_out);
    a.v_out = static_cast<__nv_bfloat16*>(v_out);
    return launch(pick<true>(D, bits, group), true, a, const_cast<void*>(pool), slot_mapping, T, Hkv, D,
                  page_size, num_pages, bits, group, stream);
}
