// Where the tokens of a paged cache lie, and how a decode call shares them out.
// Plain arithmetic, also compiled by the host compiler, where it is checked.
//
// Tokens are read in tiles of 32, two units of 16; a page is a whole number of
// units, so that a unit lies in one page and its rows are consecutive there.
#pragma once

#include <cstddef>
#include <cstdint>

#if defined(__HIPCC__)
#define FQ_PAGED_FN __host__ __device__ __forceinline__
#else
#define FQ_PAGED_FN inline
#endif

namespace fq {

constexpr int32_t kDecodeMaxLen = 1 << 30;  // of a sequence (sums of a length and a tile stay an int32)
constexpr int kDecodeUnit = 16;
constexpr int kDecodeTile = 2 * kDecodeUnit;
constexpr int kDecodeWaves = 4;    // of a workgroup; they take the tiles of its part in turn
constexpr int kDecodeHeads = 16;   // query heads of a workgroup
constexpr int kDecodeWgs = 1024;   // workgroups that a call is split into, where the cache is long enough

// Tokens that a sequence sees.
FQ_PAGED_FN int32_t paged_len(int32_t len, int32_t max_pages, int32_t page_size) {
    const int32_t most = max_pages * page_size;
    return len < 0 ? 0 : len > most ? most : len;
}

// Parts that a sequence of up to max_len tokens is split into, at most: as many as
// give kDecodeWgs workgroups, and no part shorter than a tile for each wave.
FQ_PAGED_FN int32_t decode_splits(int64_t pairs, int32_t max_len) {
    const int32_t step = kDecodeTile * kDecodeWaves;
    const int64_t want = (kDecodeWgs + pairs - 1) / pairs, most = (int64_t(max_len) + step - 1) / step;
    return int32_t(want < most ? want : most);
}

// The tokens of each part of a sequence (whole tiles for each wave), and the parts it has.
struct DecodeParts {
    int32_t len, count;
};
FQ_PAGED_FN DecodeParts decode_parts(int32_t len, int32_t splits) {
    const int32_t step = kDecodeTile * kDecodeWaves;
    const int32_t steps = (len + step - 1) / step;
    const int32_t per = (steps + splits - 1) / splits;
    return DecodeParts{per * step, per ? (steps + per - 1) / per : 0};
}

// Pages by a multiplication: units of a page d = page_size / 16 <= 2^11, m = 2^37 / d + 1.
// The unit u < 2^26 lies in page u m / 2^37: m d - 2^37 is at most d, so u times it stays below 2^37.
FQ_PAGED_FN uint64_t paged_magic(int32_t page_size) { return (uint64_t(1) << 37) / uint32_t(page_size / kDecodeUnit) + 1; }
// Entry of the page table that holds token t's page (of the last token's where t lies behind it; len >= 1).
FQ_PAGED_FN int32_t paged_entry(int32_t t, int32_t len, uint64_t magic) {
    return int32_t((uint64_t(uint32_t((t < len ? t : len - 1) / kDecodeUnit)) * magic) >> 37);
}

// The unit of tokens t .. t + 15 (t a multiple of 16) of a sequence of `len` tokens, whose page is `page`,
// entry `entry` of the table.
struct PagedUnit {
    int32_t page, first;  // its first token's place; page 0 and token 0, which exist, where none is seen
    int32_t valid;        // tokens seen, the first ones
};
FQ_PAGED_FN PagedUnit paged_unit(int32_t page, int32_t entry, int32_t t, int32_t len, int32_t pages, int32_t page_size) {
    if (t >= len || page < 0 || page >= pages) return PagedUnit{0, 0, 0};
    const int32_t left = len - t;
    return PagedUnit{page, t - entry * page_size, left < kDecodeUnit ? left : kDecodeUnit};
}

// Index of a row of a head, in rows of head_dim values (and in scales).
FQ_PAGED_FN int64_t paged_row(int32_t page, int32_t place, int32_t head, int32_t kv_heads, int32_t page_size) {
    return (int64_t(page) * kv_heads + head) * page_size + place;
}

// Workspace of a decode call in rows of (head_dim + 2) floats: at least one for every
// sequence, query head and part, and never fewer for more sequences or tokens.
FQ_PAGED_FN size_t decode_part_rows(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t max_len) {
    const int32_t step = kDecodeTile * kDecodeWaves;
    const int64_t group = q_heads / kv_heads, per_seq = kv_heads * ((group + kDecodeHeads - 1) / kDecodeHeads);
    const int64_t by_len = int64_t(seqs) * ((int64_t(max_len) + step - 1) / step);
    const int64_t by_wgs = seqs + (kDecodeWgs + per_seq - 1) / per_seq;
    return size_t(by_len < by_wgs ? by_len : by_wgs) * size_t(q_heads);
}

}  // namespace fq
