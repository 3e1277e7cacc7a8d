// The quantised paged cache: its layout in memory.  Shared by the writer, the reader and the
// attention kernel, and by the host checks.
//
// pool: uint8 [num_pages, Hkv, page_bytes].  One page of one KV head is contiguous, so one bulk
// copy brings everything an attention stage needs of it:
//     K codes     page_size rows of D * bits / 8 bytes
//     V codes     page_size rows of D * bits / 8 bytes
//     parameters  page_size rows of D / group quadruples of bf16: k_scale, k_min, v_scale, v_min
// Code c of a group stands for min + scale * c.
//
// A row's codes are stored in the order in which the attention kernel's lanes hold them, so that
// each lane reads its codes with one wide load: a K row of [D/16][4][4] elements is stored as
// [4][D/16][4] (lane t of a quad holds elements 16 s + 4 t + i of every 16-element slice s), a V
// row of [D/16][8][2] elements as [8][D/16][2] (the lanes of row g hold elements 16 m + 2 g + i of
// every 16-element tile m).  Two 4-bit codes share a byte, the first one in its low half.
#pragma once

#include <cstddef>
#include <cstdint>

namespace da {

// bytes of a K (or V) row of codes, of a row's parameters, and of a whole row
__host__ __device__ constexpr int kQuantRowCodes(int D, int bits) { return D * bits / 8; }
__host__ __device__ constexpr int kQuantRowParams(int D, int group) { return D / group * 8; }
__host__ __device__ constexpr int kQuantRowBytes(int D, int bits, int group) {
    return 2 * kQuantRowCodes(D, bits) + kQuantRowParams(D, group);
}

// Whether the kernels have the format (page sizes: powers of two from 8 to 256).
constexpr bool quant_format_ok(int D, int page_size, int bits, int group) {
    return (D == 64 || D == 128) && (bits == 4 || bits == 8) &&
           (group == 32 || group == 64 || group == 128) && group <= D && page_size >= 8 &&
           page_size <= 256 && (page_size & (page_size - 1)) == 0;
}

}  // namespace da
