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
// Workgroups that a call is split into, where the cache is long enough.  (512 / 1024 / 2048: 64 sequences of 0 to 8191
// tokens 26.2 / 25.0 / 25.1 us, 16 of 4000 31.7 / 32.8 / 35.5, one of 131071 95.8 / 98.0 / 102.8: more even out
// unequal lengths, fewer leave less to join.)
constexpr int kDecodeWgs = 1024;

// Tokens that a sequence sees.
FQ_PAGED_FN int32_t paged_len(int32_t len, int32_t max_pages, int32_t page_size) {
    const int32_t most = max_pages * page_size;
    return len < 0 ? 0 : len > most ? most : len;
}

// A call's sequences are cut into parts of one length, which the kernel finds from the
// lengths: as many parts as give kDecodeWgs workgroups, and no part shorter than a tile
// for each wave.  Parts are numbered through the sequences in turn; one of no tokens has a part too.
constexpr int32_t kDecodeStep = kDecodeTile * kDecodeWaves;
// Query heads share a key head's reads in workgroups of up to kDecodeHeads.
FQ_PAGED_FN int32_t decode_head_tiles(int32_t q_heads, int32_t kv_heads) {
    return (q_heads / kv_heads + kDecodeHeads - 1) / kDecodeHeads;
}
// Parts of the batch, aside from one that every sequence has.
FQ_PAGED_FN int32_t decode_target(int32_t kv_heads, int32_t head_tiles) {
    const int32_t n = kv_heads * head_tiles;
    return (kDecodeWgs + n - 1) / n;
}
// What a sequence adds to the batch's length, in 64 tokens.
FQ_PAGED_FN uint32_t decode_units(int32_t len) { return (uint32_t(len) + 63) / 64; }
// Tokens of a part, from the batch's sum of those: sum / target of them are at most target parts.
FQ_PAGED_FN int32_t decode_part_len(uint64_t units, int32_t target) {
    const uint32_t t = uint32_t(target);
    const uint64_t up = units + t - 1;  // (divided in 32 bits where it fits them)
    const uint64_t per = up >> 32 ? up / t : uint64_t(uint32_t(up) / t);
    const uint64_t steps = (per * 64 + kDecodeStep - 1) / kDecodeStep;
    return steps > uint64_t(kDecodeMaxLen / kDecodeStep) ? kDecodeMaxLen : steps ? int32_t(steps) * kDecodeStep : kDecodeStep;
}
FQ_PAGED_FN int32_t decode_count(int32_t len, int32_t part_len) { return len <= part_len ? 1 : (len + part_len - 1) / part_len; }
// Most parts that a call has, whatever the lengths.
FQ_PAGED_FN int64_t decode_parts(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t max_len) {
    const int64_t by_len = int64_t(seqs) * ((int64_t(max_len) + kDecodeStep - 1) / kDecodeStep);
    const int64_t by_target = int64_t(seqs) + decode_target(kv_heads, decode_head_tiles(q_heads, kv_heads));
    return by_len < by_target ? by_len : by_target;
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

// The last of n sorted entries that is not past a wanted one (-1: none), 64 of them looked at in a step, so that n up to
// 2^18 takes three steps; count(first, step, probes): how many of the entries first, first + step, ..., `probes` of
// them and at most 64, are not past it.  Whatever the entries are, only those of 0 .. n - 1 are looked at, and the steps end.
template <class Count>
FQ_PAGED_FN int32_t last_not_past(int32_t n, Count count) {
    int32_t first = 0;
    while (n > 64) {
        const int32_t step = (n + 63) / 64, k = count(first, step, (n + step - 1) / step);
        if (k == 0) return -1;
        first += (k - 1) * step;
        n = step < n - (k - 1) * step ? step : n - (k - 1) * step;
    }
    return first + count(first, 1, n) - 1;
}

// Workspace of a decode call, never smaller for more sequences or tokens: the first part and the
// parts of every sequence, and of the batch all parts and the tokens of one; then for every part and query head the
// maximum, the sum of weights and the output.
struct DecodeWorkspace {
    size_t stats, sums, bytes;  // offsets of the two, and the size
};
FQ_PAGED_FN DecodeWorkspace decode_workspace(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             int32_t max_len) {
    const size_t rows = size_t(decode_parts(seqs, q_heads, kv_heads, max_len)) * size_t(q_heads);
    const size_t stats = (size_t(seqs) * 8 + 8 + 255) / 256 * 256, sums = stats + (rows * 8 + 255) / 256 * 256;
    return DecodeWorkspace{stats, sums, (sums + rows * size_t(head_dim) * 4 + 255) / 256 * 256};
}

}  // namespace fq
