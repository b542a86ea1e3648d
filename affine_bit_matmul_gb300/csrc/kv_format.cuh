// Format of the paged 4-bit key/value cache, shared by the kernels that write,
// read and attend over it.
//
// A page holds page_size tokens.  Its block for one key/value head is
//   K codes | K pairs | V codes | V pairs
// with page_size * D / 2 bytes of codes and one (bf16 scale, bf16 bias) pair
// per token and group of G values, [page_size][D / G].  Codes are stored in
// slabs of 8 tokens x DS = min(D, 128) values, in the order in which a warp's
// lanes feed them to m16n8k16 matrix instructions: lane 4 r + i owns DS / 32
// consecutive words, word u being
//   K: token r,                values 32 u + 8 i + 0..7   (lowest nibble first)
//   V: tokens 2 i and 2 i + 1, values 32 u + r + 8 n, n = 0..3: token 2 i in
//      the low half, token 2 i + 1 in the high half.
// So a lane's operands of 8 tokens are one 16-byte load without bank
// conflicts, a K word's nibbles pair up along the values (0 with 4, 1 with 5,
// ...) and a V word's along the tokens, and four masks and one shift make the
// pairs of a word four registers of f16 operands.
#pragma once

#include <cstdint>

#include "mxq_device.cuh"

namespace mxq {

__host__ __device__ constexpr int kv_code_bytes(int D, int page) { return page * (D / 2); }
__host__ __device__ constexpr int kv_pair_bytes(int D, int G, int page) {
    return page * (D / G) * 4;
}
// Bytes of one page for one key/value head.
__host__ __device__ constexpr int kv_block_bytes(int D, int G, int page) {
    return 2 * (kv_code_bytes(D, page) + kv_pair_bytes(D, G, page));
}

// Byte offset, within the K codes of a block, of the word that holds values
// v .. v + 7 (v a multiple of 8) of token t.
__device__ __forceinline__ int kv_k_word(int D, int t, int v) {
    const int ds = D < 128 ? D : 128, words = ds / 32;
    const int lane = (t & 7) * 4 + ((v >> 3) & 3);
    return ((((t >> 3) * (D / ds) + v / ds) * 32 + lane) * words + (v % ds) / 32) * 4;
}

// Byte offset, within the V codes, of the half word that holds values
// v + r + 8 n, n = 0..3 (v a multiple of 32), of token t.
__device__ __forceinline__ int kv_v_half(int D, int t, int v, int r) {
    const int ds = D < 128 ? D : 128, words = ds / 32;
    const int lane = r * 4 + ((t & 7) >> 1);
    return ((((t >> 3) * (D / ds) + v / ds) * 32 + lane) * words + (v % ds) / 32) * 4 +
           (t & 1) * 2;
}

}  // namespace mxq
