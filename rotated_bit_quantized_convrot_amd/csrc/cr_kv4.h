// Paged cache of keys and values held in 4 bits (KV4): layout, and the rules
// that place a sequence's tokens in it, shared by the writer, by attention
// over it (cr_kv4.hip) and by the host.
//
// A value of the cache is x'[d] = s (c - z), c in 0..15, s and z of its group
// of g along the head; x' is the head rotated (kv4 with rotate) or as it is.
//   codes   [page][K, V][head] blocks of S D / 2 bytes (S rows a page)
//     K     row r at r D / 2; dword i D / 32 + s of a row holds d = 32 s + 8 i
//           + 0..7, the MFMA operand of one lane: d + 2 j in bits 4 j,
//           d + 2 j + 1 in bits 16 + 4 j
//     V     16 rows at (r / 16) 8 D; byte (16 e + m) 16 + r % 16 holds
//           d = 32 e + m in its low nibble and d = 32 e + 16 + m in its high
//           one: a lane's 16 bytes are 16 tokens of its two d
//   scales  words [page][K, V][head][S][D / g]: the bits of the float32 s,
//           whose low four hold z.  A group that held an infinity or a NaN has
//           a NaN for s.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace cr {

constexpr uint32_t kKv4Nan = 0x7FC00000u;

struct Kv4 {
    uint8_t* codes;
    uint32_t* scales;
    int pages, page_log2, heads, dim, group, rotate;
    const int32_t* table;   // [B, width] page ids
    const int32_t* lens;    // [B] tokens in the cache, the call's own among them
    const int32_t* cu;      // [B + 1] first rows of the call's sequences
    int width, B, T;        // T: rows of the call's tensors
};

__host__ __device__ inline int clamp_int(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Sequence b of the call: its rows, and the tokens of it that the cache can
// hold.  Whatever the three device arrays say, rows stay inside 0..T and
// tokens inside the table.
struct Kv4Seq {
    int first, rows, tokens;
};
__host__ __device__ inline Kv4Seq kv4_seq(const Kv4& c, int b) {
    Kv4Seq s;
    s.first = clamp_int(c.cu[b], 0, c.T);
    s.rows = clamp_int(c.cu[b + 1], s.first, c.T) - s.first;
    const int64_t room = (int64_t)c.width << c.page_log2;
    s.tokens = clamp_int(c.lens[b], 0, room > 0x7FFFFFFF ? 0x7FFFFFFF : (int)room);
    return s;
}
// The page that holds token `pos` (0 <= pos < tokens) of sequence b, or -1:
// a table entry that is no page holds nothing.
__host__ __device__ inline int kv4_page(const Kv4& c, int b, int pos) {
    const int p = c.table[(size_t)b * c.width + (pos >> c.page_log2)];
    return p >= 0 && p < c.pages ? p : -1;
}
// Byte and word offsets of a page's K (which = 0) or V (1) of a head.
__host__ __device__ inline size_t kv4_codes_at(const Kv4& c, int page, int which, int head) {
    return ((((size_t)page * 2 + which) * c.heads + head) << c.page_log2) * (c.dim / 2);
}
__host__ __device__ inline size_t kv4_scales_at(const Kv4& c, int page, int which, int head) {
    return ((((size_t)page * 2 + which) * c.heads + head) << c.page_log2) * (c.dim / c.group);
}
__host__ __device__ inline int kv4_k_byte(int dim, int row, int dword) { return row * (dim / 2) + 4 * dword; }
__host__ __device__ inline int kv4_v_byte(int dim, int row, int pair) {
    return (row >> 4) * (8 * dim) + 16 * pair + (row & 15);
}

}  // namespace cr
