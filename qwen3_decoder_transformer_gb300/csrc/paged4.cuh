// The paged KV cache held in 4 bits: layout of a page and the address of a token in it.
//
// pages [n_pages][Hkv][page_bytes]: one page holds `page` tokens (a power of two, 16..256) of one kv head, first their codes
// [page][dh / 2] (two a byte, the lower nibble first), then [page][dh / 64] pairs (scale, minimum) in bf16, one for
// 64 dims of a token: value = minimum + scale * code. A page of a head is contiguous and a multiple of 16 bytes, so it is
// fetched by untiled bulk copies; the codes of one token and head are contiguous, so one token can be appended at a time.
#pragma once

#include "common.cuh"

namespace q3 {

constexpr int kP4Group = 64;  // dims that share a scale and a minimum

struct Paged4 {
    const uint8_t *k, *v;
    const int* table;  // [sequences][max_pages]
    int n_pages, max_pages, page_log;
};

__host__ __device__ constexpr int p4_token_bytes(int dh) { return dh / 2 + dh / kP4Group * 4; }
__host__ __device__ constexpr size_t p4_page_bytes(int page, int dh) { return (size_t)page * p4_token_bytes(dh); }

}  // namespace q3
