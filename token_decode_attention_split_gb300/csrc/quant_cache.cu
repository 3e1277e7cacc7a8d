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
#include "ptx.cuh"
#include "quant_format.h"

namespace {

constexpr int kThreads = 256;

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
    int page_shift, page_size;
    int page_bytes;
};

// Adding and subtracting 1.5 * 2^23 rounds a number below 2^22 to an integer (ties to even); the
// sum's low bits are that integer.
constexpr float kRound = 12582912.0f;

template <int D, int BITS>
struct RowShape {
    static constexpr int kWords = D * BITS / 32;          // words of a stored row = lanes per row
    static constexpr int kPer = 32 / BITS;                // codes per word
    static constexpr int S = D / 16;                      // 16-element slices
    static constexpr int kRowsPerWarp = 32 / kWords;
    // element index of code i of stored word j
    __device__ static constexpr int k_elem(int j, int i) {
        const int pos = j * kPer + i, quad = pos / 4;
        return 16 * (quad % S) + 4 * (quad / S) + pos % 4;
    }
    __device__ static constexpr int v_elem(int j, int i) {
        const int pos = j * kPer + i, pair = pos / 2;
        return 16 * (pair % S) + 2 * (pair / S) + pos % 2;
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
            x[i] = __ldg(reinterpret_cast<const uint32_t*>(row + R::v_elem(j, 2 * i)));
    } else {
#pragma unroll
        for (int i = 0; i < R::kPer / 4; ++i) {
            const uint2 y = __ldg(reinterpret_cast<const uint2*>(row + R::k_elem(j, 4 * i)));
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
        float s = __fdiv_rn(range, static_cast<float>((1 << BITS) - 1));
        s = __uint_as_float((__float_as_uint(s) + 0xffffu) & 0xffff0000u);
        if (!fine || s < 1.17549435e-38f) s = 0.f;
        par[q] = fine ? (__float_as_uint(s) >> 16) | (__float_as_uint(mn) & 0xffff0000u)
                      : 0x7fc07fc0u;
        const float inv = s > 0.f ? __frcp_rz(s) : 0.f;
        const float base = fine ? mn : 0.f;
#pragma unroll
        for (int i = 0; i < kX; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t w = x[q * kX + i];
                const float v = e ? da::bf16_hi_to_f32(w) : da::bf16_lo_to_f32(w);
                const float d = v - base;
                const float k0 = __fadd_rn(__fmaf_rn(d, inv, kRound), -kRound);
                const float res = __fmaf_rn(-k0, s, d);
                const float c = __fadd_rn(__fmaf_rn(res, inv, k0), kRound);
                const uint32_t code = __float_as_uint(c) & ((1u << BITS) - 1u);
                packed |= (fine ? code : 0u) << (((q * kX + i) * 2 + e) * BITS);
            }
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

// The page block and row of item (new row t, KV head h), or null where the slot says to skip it.
__device__ __forceinline__ unsigned char* item_block(const CacheArgs& a, int64_t t, int h, int& row) {
    const int64_t w = a.slots[t];
    if (w < 0 || w >= a.num_slots) return nullptr;
    const int64_t page = w >> a.page_shift;
    row = static_cast<int>(w & (a.page_size - 1));
    return a.pool + (page * a.Hkv + h) * a.page_bytes;
}

template <int D, int BITS, int GROUP>
__global__ void __launch_bounds__(kThreads) quant_append_kernel(const CacheArgs a) {
    using R = RowShape<D, BITS>;
    using PK = WordPlace<D, BITS, GROUP, false>;
    using PV = WordPlace<D, BITS, GROUP, true>;
    constexpr int RB = da::kQuantRowCodes(D, BITS), PB = da::kQuantRowParams(D, GROUP);
    da::grid_dependency_wait();
    da::allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int j = lane % R::kWords, sub = lane / R::kWords;
    const int64_t items = a.rows * a.Hkv;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * R::kRowsPerWarp;
    // the loop bound is the same on every lane of a warp (the shuffles need all of them)
    for (int64_t it0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) *
                       R::kRowsPerWarp;
         it0 < items; it0 += step) {
        const int64_t it = it0 + sub < items ? it0 + sub : items - 1;
        const int64_t t = it / a.Hkv;
        const int h = static_cast<int>(it - t * a.Hkv);
        uint32_t xk[R::kPer / 2], xv[R::kPer / 2], pk[2], pv[2];
        load_elems<D, BITS, false>(a.k_new + t * a.k_stride + h * D, j, xk);
        load_elems<D, BITS, true>(a.v_new + t * a.v_stride + h * D, j, xv);
        int row = 0;
        unsigned char* block = item_block(a, t, h, row);
        const uint32_t ck = quantise_word<D, BITS, GROUP, false>(xk, pk);
        const uint32_t cv = quantise_word<D, BITS, GROUP, true>(xv, pv);
        if (block == nullptr || it0 + sub >= items) continue;
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

// The bf16 values of stored word w; par(i): scale | min << 16 of the group of code i.
template <int D, int BITS, int GROUP, bool V>
__device__ __forceinline__ void restore_word(uint32_t w, int j, const unsigned char* par,
                                             uint32_t (&x)[RowShape<D, BITS>::kPer / 2]) {
    using R = RowShape<D, BITS>;
    using P = WordPlace<D, BITS, GROUP, V>;
    constexpr int kX = R::kPer / 2 / P::kQ;
#pragma unroll
    for (int q = 0; q < P::kQ; ++q) {
        const uint32_t p = __ldg(reinterpret_cast<const uint32_t*>(par + 8 * (P::group(j) + q) +
                                                                   (V ? 4 : 0)));
        const float s = da::bf16_lo_to_f32(p), mn = da::bf16_hi_to_f32(p);
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t code = (w >> (((q * kX + i) * 2 + e) * BITS)) & ((1u << BITS) - 1u);
                const float c = __uint_as_float(0x4b400000u | code) - kRound;
                v[e] = __fmaf_rn(s, c, mn);
            }
            x[q * kX + i] = da::pack_bf16x2(v[0], v[1]);
        }
    }
}

template <int D, int BITS, int GROUP>
__global__ void __launch_bounds__(kThreads) quant_read_kernel(const CacheArgs a) {
    using R = RowShape<D, BITS>;
    constexpr int RB = da::kQuantRowCodes(D, BITS), PB = da::kQuantRowParams(D, GROUP);
    da::grid_dependency_wait();
    da::allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int j = lane % R::kWords, sub = lane / R::kWords;
    const int64_t items = a.rows * a.Hkv;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * R::kRowsPerWarp;
    for (int64_t it = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) *
                          R::kRowsPerWarp + sub;
         it < items; it += step) {
        const int64_t t = it / a.Hkv;
        const int h = static_cast<int>(it - t * a.Hkv);
        int row = 0;
        const unsigned char* block = item_block(a, t, h, row);
        uint32_t xk[R::kPer / 2], xv[R::kPer / 2];
        if (block != nullptr) {
            const uint32_t ck = __ldg(reinterpret_cast<const uint32_t*>(block + row * RB + 4 * j));
            const uint32_t cv = __ldg(
                reinterpret_cast<const uint32_t*>(block + (a.page_size + row) * RB + 4 * j));
            const unsigned char* par = block + 2 * a.page_size * RB + row * PB;
            restore_word<D, BITS, GROUP, false>(ck, j, par, xk);
            restore_word<D, BITS, GROUP, true>(cv, j, par, xv);
        } else {
#pragma unroll
            for (int i = 0; i < R::kPer / 2; ++i) xk[i] = xv[i] = 0u;
        }
        __nv_bfloat16* ko = a.k_out + it * D;
        __nv_bfloat16* vo = a.v_out + it * D;
#pragma unroll
        for (int i = 0; i < R::kPer / 4; ++i)
            *reinterpret_cast<uint2*>(ko + R::k_elem(j, 4 * i)) = make_uint2(xk[2 * i], xk[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < R::kPer / 2; ++i)
            *reinterpret_cast<uint32_t*>(vo + R::v_elem(j, 2 * i)) = xv[i];
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

da_status launch(Kernel kernel, CacheArgs& a, void* pool, const int64_t* slots, int64_t T, int Hkv,
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
    const int64_t per_block = kThreads / (D * bits / 32);
    const int64_t want = (T * Hkv + per_block - 1) / per_block;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < 8LL * sms ? want : 8LL * sms));
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
    return launch(pick<false>(D, bits, group), a, pool, slot_mapping, T, Hkv, D, page_size,
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
    return launch(pick<true>(D, bits, group), a, const_cast<void*>(pool), slot_mapping, T, Hkv, D,
                  page_size, num_pages, bits, group, stream);
}
