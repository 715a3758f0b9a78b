// kv_index.h — where a token's row lies in a paged cache. Plain C++ with no CUDA header, so that
// the index arithmetic is the same on the device and in the host tests. Internal to libcolimoe.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define COLI_HD __host__ __device__ __forceinline__
#else
#define COLI_HD inline
#endif

namespace colimoe {

struct KvShape {
    int64_t page_stride, token_stride, head_stride;  // elements
    int32_t pages, page_size;
};

enum KvWhy : int { kKvOk = 0, kKvBadPage = 1, kKvBadPosition = 2 };

// The page and the slot of token t, where row[0..width) are the sequence's pages; page -1 if there is
// none, and why.
COLI_HD int kv_place(const KvShape &c, const int32_t *row, int32_t width, int32_t t, int32_t &page, int32_t &slot) {
    page = -1;
    slot = 0;
    if (t < 0) return kKvBadPosition;
    const uint32_t i = (uint32_t)t / (uint32_t)c.page_size;
    if (i >= (uint32_t)width) return kKvBadPosition;
    const int32_t p = row[i];
    if ((uint32_t)p >= (uint32_t)c.pages) return kKvBadPage;
    page = p;
    slot = (int32_t)((uint32_t)t - i * (uint32_t)c.page_size);
    return kKvOk;
}

// Element offset of token t's row of kv head h; -1 (and why) if there is none. Products are 64-bit: a
// pool may hold more than 2^31 elements.
COLI_HD int64_t kv_row(const KvShape &c, const int32_t *row, int32_t width, int32_t t, int32_t h, int &why) {
    int32_t page, slot;
    why = kv_place(c, row, width, t, page, slot);
    if (why) return -1;
    return (int64_t)page * c.page_stride + (int64_t)slot * c.token_stride + (int64_t)h * c.head_stride;
}

// Division of t in [0, 2^31) by a page size: with l = ceil(log2 size) and mul = ceil(2^(31 + l) / size),
// (t * mul) >> (31 + l) is exact, as mul * size - 2^(31 + l) < size <= 2^l.
struct KvDivide {
    uint32_t mul, shift;
};
inline KvDivide kv_divide_by(int32_t size) {
    uint32_t l = 0;
    while (((int64_t)1 << l) < size) l++;
    return {(uint32_t)((((uint64_t)1 << (31 + l)) + size - 1) / (uint32_t)size), 31 + l};
}
COLI_HD int32_t kv_quotient(KvDivide d, int32_t t) { return (int32_t)(((uint64_t)(uint32_t)t * d.mul) >> d.shift); }

// The tokens [first, end) of a sequence of n cached tokens that the new token sees; n is clamped to
// what the table can name (and flagged).
COLI_HD void kv_span(int32_t n, int32_t width, int32_t page_size, int32_t window, int32_t &first, int32_t &end,
                     int &why) {
    const int64_t most = (int64_t)width * page_size;
    why = (n < 0 || n > most) ? kKvBadPosition : kKvOk;
    end = n < 0 ? 0 : n > most ? (int32_t)most : n;
    first = (window > 0 && end > window) ? end - window : 0;
}

// Units of `unit` tokens (the last one ragged) that hold `tokens` of them, and the token at place `at` of unit u
// behind `first`. A sequence may end at 2^31 - 1, and the places of its last unit behind the end pass 2^31: sums
// are unsigned.
COLI_HD int32_t kv_units(int32_t tokens, int32_t unit) {
    return (int32_t)(((uint32_t)tokens + (uint32_t)unit - 1) / (uint32_t)unit);
}
COLI_HD bool kv_unit_token(int32_t first, int32_t end, int32_t unit, int32_t u, int32_t at, int32_t &t) {
    const uint32_t x = (uint32_t)first + (uint32_t)u * (uint32_t)unit + (uint32_t)at;
    t = (int32_t)x;
    return x < (uint32_t)end;
}

}  // namespace colimoe
