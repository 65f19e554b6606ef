// A paged cache of keys and values held in 4 bits (layout in cr_kv4.h): the
// writer, and attention over it.
//
//   x' = H x / sqrt D (rotate: H the Sylvester Hadamard matrix of the head, by
//   float32 butterflies of strides 1, 2, .. D / 2, a, b -> a + b, a - b, then
//   times float32(1 / sqrt D)) or x; for each group of g along the head
//   lo = min(0, min x'), hi = max(0, max x'), s = hi / 15 - lo / 15 to the
//   nearest float32 whose low four bits are 0, z = clamp(rint(-lo / s), 0, 15),
//   c = clamp(rint(x' / s) + z, 0, 15); both 0 where s = 0.
#include <algorithm>
#include <numeric>
#include <type_traits>

#include "cr_w4g.h"
#include "cr_kv4.h"

namespace cr {
namespace {

template <int D>
constexpr float kv4_norm() { return D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f; }

template <int M, int N>
__device__ __forceinline__ void rotate_lanes(float (&x)[N], int lane) {
    const float c = lane & M ? -1.0f : 1.0f;   // x + p, or p - x: one rounding either way
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float p;
        if constexpr (M == 32) p = __shfl_xor(x[i], 32);
        else p = lane_xor<M>(x[i]);
        x[i] = __builtin_fmaf(x[i], c, p);
    }
}

// Lane l holds d = l D / 64 and on.
template <int D>
__device__ __forceinline__ void rotate_head(float (&x)[D / 64]) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int h = 1; h < N; h <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & h) == 0) {
                const float a = x[i], b = x[i + h];
                x[i] = a + b;
                x[i + h] = a - b;
            }
    rotate_lanes<1>(x, lane);
    rotate_lanes<2>(x, lane);
    rotate_lanes<4>(x, lane);
    rotate_lanes<8>(x, lane);
    rotate_lanes<16>(x, lane);
    rotate_lanes<32>(x, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= kv4_norm<D>();
}

struct AppendArgs {
    Kv4 c;
    const uint16_t* x[2];        // K, V
    int64_t row[2], head[2];     // their strides in values
};

// 16 rows of the cache (of one page) that take new tokens: rows r0 up to r1 of
// the call's are positions pos0 and on, all in the 16 from pos0 & ~15.
struct AppendWork {
    int b, r0, r1, pos0;
};
__device__ __forceinline__ bool append_work(const Kv4& c, int index, AppendWork* w) {
    const int lane = threadIdx.x & 63;
    for (int b0 = 0; b0 < c.B; b0 += 64) {
        const Kv4Seq s = kv4_seq(c, min(b0 + lane, c.B - 1));
        // rows that come before token 0 are left out
        const int rows = b0 + lane < c.B ? min(s.rows, s.tokens) : 0, from = s.tokens - rows;
        const int n = rows > 0 ? (s.tokens - 1) / 16 - from / 16 + 1 : 0;
        const int upto = wave_scan(n, add_ints);
        const uint64_t after = __ballot(upto > index);
        if (after) {
            const int l = __builtin_ctzll(after);
            auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            const int first = of(from), end = of(s.tokens), row = of(s.first + s.rows - rows);
            const int block = first / 16 + index - of(upto - n), lo = max(first, block * 16), hi = min(end, block * 16 + 16);
            w->b = b0 + l;
            w->pos0 = lo;
            w->r0 = row + (lo - first);
            w->r1 = w->r0 + (hi - lo);
            return true;
        }
        index -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// One wave 16 rows of the cache, a head, K or V; lane 4 t + p holds token t's
// d = 32 s + 8 p + 0..7: the strides of the rotation are among j (1, 2, 4),
// among the four lanes (8, 16), among s (32 ..); K's bytes of a lane lie side
// by side, V's go through LDS to have the 16 tokens of a pair of d side by side.
// 1220 tokens, 8 heads of 128, rotated: 6.9 us, loads that wait for each other
// (lengths, page, rows); 16384 tokens: 29 us for 86 MB, its arithmetic (bound at
// 4.7 TB/s: 18 us).
template <class T, int D, int NG>
__global__ __launch_bounds__(256) void k_kv4_append(AppendArgs a) {
    constexpr int KS = D / 32, SPG = KS / NG;
    __shared__ __align__(16) uint8_t pairs[4][8 * D];
    const int lane = threadIdx.x & 63, wave = wave_of_block(), t = lane >> 2, p = lane & 3;
    const int hw = blockIdx.x * 4 + wave;
    if (hw >= 2 * a.c.heads) return;
    const int which = hw >= a.c.heads, h = hw - which * a.c.heads;
    AppendWork w;
    if (!append_work(a.c, blockIdx.y + blockIdx.z * gridDim.y, &w)) return;
    const int page = kv4_page(a.c, w.b, w.pos0);
    if (page < 0) return;
    // lanes of rows that take no token repeat the first's or the last's
    const int base = w.pos0 & ~15, r = min(max(w.r0 + base + t - w.pos0, w.r0), w.r1 - 1);
    const bool mine = base + t >= w.pos0 && base + t < w.pos0 + (w.r1 - w.r0);
    const uint16_t* src = a.x[which] + r * a.row[which] + h * a.head[which] + 8 * p;
    float x[KS][8];
#pragma unroll
    for (int s = 0; s < KS; ++s) w4g_values<T>(src + 32 * s, x[s]);
    if (a.c.rotate) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
            for (int m = 1; m < 8; m <<= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if ((j & m) == 0) {
                        const float u = x[s][j], v = x[s][j + m];
                        x[s][j] = u + v;
                        x[s][j + m] = u - v;
                    }
            rotate_lanes<1>(x[s], lane);
            rotate_lanes<2>(x[s], lane);
        }
#pragma unroll
        for (int m = 1; m < KS; m <<= 1)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if ((s & m) == 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float u = x[s][j], v = x[s + m][j];
                        x[s][j] = u + v;
                        x[s + m][j] = u - v;
                    }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[s][j] *= kv4_norm<D>();
    }
    uint32_t word[NG], code[KS];   // code: d + 2 j in bits 4 j, d + 2 j + 1 in bits 16 + 4 j
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        float lo = 0.0f, hi = 0.0f, bad = 0.0f;
#pragma unroll
        for (int s = n * SPG; s < (n + 1) * SPG; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                lo = fminf(lo, x[s][j]);
                hi = fmaxf(hi, x[s][j]);
                bad = __builtin_fmaf(x[s][j], 0.0f, bad);   // NaN from the first infinity or NaN on
            }
        lo = fminf(lo, lane_xor<1>(lo));
        lo = fminf(lo, lane_xor<2>(lo));
        hi = fmaxf(hi, lane_xor<1>(hi));
        hi = fmaxf(hi, lane_xor<2>(hi));
        bad += lane_xor<1>(bad);
        bad += lane_xor<2>(bad);
        const uint32_t sb = bad != bad ? kKv4Nan : (__float_as_uint(hi / 15.0f - lo / 15.0f) + 8) & ~15u;
        const float sc = __uint_as_float(sb);
        // x / s by a reciprocal and one exact correction: the same float32 as the division's.  With r = x inv off
        // x / s by e, at most 1.5 of its last places, x - r s is exact (s has 20 bits) and r + (x - r s) inv off x / s
        // by 2^-24 e at most, 2^-46 of it; and x / s, of 24 bits by 20, is no nearer than 2^-45 of itself to where the
        // rounding turns.  The products stay normal where the scale is between 2^-100 and 2^100 (the others divide; a
        // quotient under 1/2 is 0 either way).  With 0 for the reciprocal, a scale of 0 or NaN gives codes of 0.
        const float inv = sc > 0.0f ? 1.0f / sc : 0.0f;
        const float z = fminf(fmaxf(rintf(sc > 0.0f ? -lo / sc : 0.0f), 0.0f), 15.0f);
        word[n] = sb | (uint32_t)z;
        const bool divide = __any(sc > 0x1p100f || (sc > 0.0f && sc < 0x1p-100f));
#pragma unroll
        for (int s = n * SPG; s < (n + 1) * SPG; ++s) {
            float q[8];
            if (divide) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = sc > 0.0f ? x[s][j] / sc : 0.0f;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float r = x[s][j] * inv;
                    q[j] = __builtin_fmaf(__builtin_fmaf(-r, sc, x[s][j]), inv, r);
                }
            }
            code[s] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                code[s] |= (uint32_t)fminf(fmaxf(rintf(q[j]) + z, 0.0f), 15.0f) << (4 * (j >> 1) + 16 * (j & 1));
        }
    }
    const int row = (base + t) & ((1 << a.c.page_log2) - 1);
    if (mine) {
        uint32_t* to = a.c.scales + kv4_scales_at(a.c, page, which, h) + row * NG;
#pragma unroll
        for (int n = 0; n < NG; ++n)
            if ((n & 3) == p) to[n] = word[n];
    }
    uint8_t* codes = a.c.codes + kv4_codes_at(a.c, page, which, h);
    if (which == 0) {
        if (mine) {
            uint32_t* to = reinterpret_cast<uint32_t*>(codes + kv4_k_byte(D, row, p * KS));
            if constexpr (KS == 2) *reinterpret_cast<uint2*>(to) = uint2{code[0], code[1]};
            else
#pragma unroll
                for (int s = 0; s < KS; s += 4)
                    *reinterpret_cast<u32x4*>(to + s) = u32x4{code[s], code[s + 1], code[s + 2], code[s + 3]};
        }
        return;
    }
    // pair 16 s + 8 p + j (p < 2): d = 32 s + 8 p + j, and that of lane p + 2
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const uint32_t other = (uint32_t)__float_as_int(lane_xor<2>(__uint_as_float(code[s])));
        // bytes of j = 0, 4, 1, 5 and 2, 6, 3, 7
        const uint32_t u = (code[s] & 0x0F0F0F0Fu) | (other & 0x0F0F0F0Fu) << 4;
        const uint32_t v = (code[s] >> 4 & 0x0F0F0F0Fu) | (other & 0xF0F0F0F0u);
        if (p < 2) {
            uint8_t* to = &pairs[wave][(16 * s + 8 * p) * 16 + t];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                to[16 * j] = (uint8_t)(((j & 2) ? v : u) >> (8 * (j >> 2) + 16 * (j & 1)));
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int row0 = base & ((1 << a.c.page_log2) - 1), from = w.pos0 - base, to = from + (w.r1 - w.r0);
#pragma unroll
    for (int i = 0; i < (D / 2 + 63) / 64; ++i) {
        const int pair = 64 * i + lane;
        if (pair >= D / 2) break;
        uint8_t* out = codes + kv4_v_byte(D, row0, pair);
        const uint8_t* in = &pairs[wave][pair * 16];
        if (to - from == 16) *reinterpret_cast<u32x4*>(out) = *reinterpret_cast<const u32x4*>(in);
        else
            for (int x = from; x < to; ++x) out[x] = in[x];   // the others' bytes are theirs
    }
}

// ---------------------------------------------------------------------------
// Attention over the cache
// ---------------------------------------------------------------------------
//
// Of a sequence's n query rows and a key head, the n G rows (row i, head of
// the group) go in tiles of 16, one to a column of MFMA 16x16x32; the tokens
// in spans over blocks, and a span's steps of 64 tokens over the block's waves.
//   S^T = K q^T      a lane holds 16 tokens' scores of one row: of step
//                    tokens 16 (lane / 16) + 0..15
//   O^T = V^T P^T    the weights are the second operand as they lie; V is laid
//                    out so that a lane's 16 bytes are these tokens of two d
// The operands hold u (1 + c / 16), the code put into the mantissa of
// u = 2^-10 (two instructions a pair); what that adds, (1 + z / 16) u sum q and
// u (1 + z / 16) sum p, is known and taken off in float32.  With 1 for u the
// sums of a head of 256 would pass float32 from q of some 2^118 on.
// q (rotated: float32) and the weights times V's scales go in as two bf16
// values of 8 bits each, in bf16's range whatever T.
constexpr uint32_t kUnitBf16 = 0x3A80u;
constexpr float kUnit = 0x1p-10f;
constexpr int kStep = 64;
constexpr int kMinSpan = 4 * kStep;
constexpr float kMostSpan = 2097152.0f;   // kMinSpans: twice of it hold the longest sequence, 2^30 tokens

template <int D>
constexpr int max_tiles() { return D == 64 ? 3 : D == 128 ? 2 : 1; }

// One block's work: tile group `tile` of sequence b (rows 16 RT tile ..),
// tokens span * chunk .. of it; its slot among all blocks of a head.
struct Kv4Work {
    int b, first, rows, tokens, tile, chunk, chunks, span, slot;
};
// The work of block `index` of `slots` (by_tile: of tile group `index`, its
// chunk 0).  Every wave counts for itself, 64 sequences at a time.
//   `fill` blocks of a head run at once (`few` where that is enough).  A block's start and end cost as much
// as some 500 tokens, so the spans are the shortest with which all blocks run
// at once, up to twice fill's share; of more than 64 sequences, which the lanes
// do not count at once, they are twice fill's share (us, 64 and 66 of 4000
// tokens: one key head 20.1 and 22.7, two 27.9 and 33.4).  Where that leaves them unlike (spans
// beyond 1.25 shares, the longest sequence beyond 1.25 times the mean) and a
// share is 2048 tokens and more, the spans are half a share and the blocks
// follow each other, at most 2 fill more than tile groups, which is what the
// grid has.  us, at once / half shares: 64 sequences of up to 30000 tokens
// 259 / 238, 100 of up to 6000 119.9 / 109.7; where both rules are off, 64 of
// 4000 77.2 / 82.7, 64 of 2048 39.3 / 47.4.  A sequence's spans are equal.
// slots = 0: one span takes everything.
template <int R>
__device__ __forceinline__ bool kv4_work(const Kv4& c, int G, int slots, int fill, int few, bool by_tile, int index, Kv4Work* w) {
    const int lane = threadIdx.x & 63;
    auto groups_of = [&](const Kv4Seq& s) { return (s.rows * G + R - 1) / R; };   // rows * G <= 2^30
    const Kv4Seq first = kv4_seq(c, min(lane, c.B - 1));
    int span = 0x40000000;
    if (slots > 0) {
        float total = 0.0f;   // of tokens, group by group
        int top = 0, groups = 0;   // the longest sequence; tile groups
        for (int b0 = 0; b0 < c.B; b0 += 64) {
            const Kv4Seq s = b0 == 0 ? first : kv4_seq(c, min(b0 + lane, c.B - 1));
            const int n = b0 + lane < c.B ? groups_of(s) : 0;
            total += __int_as_float(__builtin_amdgcn_readlane(wave_scan(__float_as_int((float)n * (float)s.tokens), add_floats), 63));
            top = max(top, __builtin_amdgcn_readlane(wave_scan(n > 0 ? s.tokens : 0, [](int x, int y) { return max(x, y); }), 63));
            groups += __builtin_amdgcn_readlane(wave_scan(n, add_ints), 63);
        }
        // A sequence or two are even by themselves: two blocks a CU do, with fewer starts, up to shares of some 2200
        // tokens.  us, 2 / 3 blocks: 20000 and 3000 tokens 14.0 / 14.5, 100000 33.2 / 33.9, 131072 40.3 / 40.8, 160000
        // 49.2 / 48.2, 250000 71.2 / 68.6, 500000 125 / 119; 3 ragged sequences 19.5 / 19.4, 32 70.6 / 56.4, 64 97.1 /
        // 72.7
        if (c.B < 3 && total < 2200.0f * (float)few) fill = few;
        const int n = lane < c.B ? groups_of(first) : 0;
        // in units of kMinSpan: fill's share, and twice it, with which at most fill / 2 blocks more than groups are
        // needed (the sum is rounded: a little more than it)
        const float e = fminf(total / (kMinSpan * (float)fill), kMostSpan);
        int lo = max((int)e, 1), hi = (int)(2.0f * e * 1.0001f) + 1;
        while (c.B <= 64 && lo < hi) {
            const int mid = (lo + hi) / 2;
            span = mid * kMinSpan;
            if (__builtin_amdgcn_readlane(wave_scan(n * max((first.tokens + span - 1) / span, 1), add_ints), 63) <= fill) hi = mid;
            else lo = mid + 1;
        }
        if (e >= 2048.0f / kMinSpan && e < kMostSpan && (float)hi > 1.25f * e && (float)top * (float)groups > 1.25f * total)
            hi = (int)(0.5f * e) + 1;
        span = hi * kMinSpan;
    }
    int at = 0, slot = 0;
    for (int b0 = 0; b0 < c.B; b0 += 64) {
        const Kv4Seq s = b0 == 0 ? first : kv4_seq(c, min(b0 + lane, c.B - 1));
        const int n = b0 + lane < c.B ? groups_of(s) : 0;
        const int chunks = max((s.tokens + span - 1) / span, 1);
        const int tiles = wave_scan(n, add_ints), all = wave_scan(n * chunks, add_ints);
        const uint64_t after = __ballot((by_tile ? at + tiles : slot + all) > index);
        if (after) {
            const int l = __builtin_ctzll(after);
            auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            w->b = b0 + l;
            w->first = of(s.first);
            w->rows = of(s.rows);
            w->tokens = of(s.tokens);
            w->chunks = of(chunks);
            w->span = ((w->tokens + w->chunks - 1) / w->chunks + kMinSpan - 1) / kMinSpan * kMinSpan;
            const int before = slot + of(all - n * chunks);
            if (by_tile) {
                w->tile = index - at - of(tiles - n);
                w->chunk = 0;
            } else {
                w->tile = (index - before) / w->chunks;
                w->chunk = (index - before) % w->chunks;
            }
            w->slot = before + w->tile * w->chunks + w->chunk;
            // (sequences that overlap can count past the grid and past 2^31: what has no slot is left out)
            return w->tile >= 0 && w->tile < of(n) && w->slot >= 0 && (slots == 0 || w->slot + (by_tile ? w->chunks : 1) <= slots);
        }
        at += __builtin_amdgcn_readlane(tiles, 63);
        slot += __builtin_amdgcn_readlane(all, 63);
    }
    return false;
}

// Partial results of a slot: averages [R][D], then the maxima and the sums of
// weights [R] each, R the rows of a block.
//   Averages, in LDS too, carry 2^-8, so that neither a code's offset nor
// turning them back passes float32 where the output does not.
constexpr float kPart = 1.0f / 256.0f;
// The maximum of a row whose tokens have all scored -infinity; that of a row
// that has seen none is -infinity.
constexpr float kNoScore = -3.402823466e38f;
template <int D, int R>
constexpr size_t part_words() { return R * (D + 2); }

// Four operand pairs of a dword of codes: u (1 + c / 16) in bf16.
// The constants come in registers: as literals they would cost an instruction
// more a pair.
struct Mantissa {
    uint32_t mask = 0x00780078u, one = kUnitBf16 * 0x10001u;
    __device__ __forceinline__ uint32_t operator()(uint32_t w) const { return (w & mask) | one; }
};
__device__ __forceinline__ Mantissa mantissa() {
    Mantissa m;
    asm("" : "+v"(m.mask), "+v"(m.one));
    return m;
}
__device__ __forceinline__ u32x4 kv4_operand(Mantissa m, uint32_t w) {
    return u32x4{m(w << 3), m(w >> 1), m(w >> 5), m(w >> 9)};
}
// 16 tokens of V (4 dwords, a byte a token): operand of tokens 8 u + 0..7 in
// the order 0 2, 1 3, 4 6, 5 7, of the bytes' low or high nibbles.
template <bool HIGH>
__device__ __forceinline__ u32x4 kv4_v_operand(Mantissa m, uint32_t a, uint32_t b) {
    if constexpr (HIGH) return u32x4{m(a >> 1), m(a >> 9), m(b >> 1), m(b >> 9)};
    else return u32x4{m(a << 3), m(a >> 5), m(b << 3), m(b >> 5)};
}
// x as hi + lo of 8 bits each (to 2^-17 of x).
__device__ __forceinline__ void split2(float a, float b, uint32_t* hi, uint32_t* lo) {
    *hi = pack_bf16x2(a, b);
    *lo = pack_bf16x2(a - __uint_as_float(*hi << 16), b - __uint_as_float(*hi & 0xFFFF0000u));
}

// Floats of a row in LDS, so that 16 rows' 16 bytes hit all banks; of the block.
template <int D>
constexpr int lds_row() { return D + 4; }
template <int D, int W, int TR>
constexpr int lds_words() { return W * TR * lds_row<D>(); }

// A step's scales s and 1 + z / 16 (of V: the operand, u (1 + z / 16), in its
// order of tokens).
template <int NG>
struct Stage {
    float ks[NG][kStep], kz[NG][kStep], vs[NG][kStep];
    uint16_t vz[NG][kStep];
};

template <int N>
struct Words {
    uint32_t w[N];
};

// 1 / x to a unit in the last place (sums of weights are 0 or some 1 and more),
// or 0: where all weights are 0, as those of a row that saw nothing, averages
// are.
__device__ __forceinline__ float reciprocal_or_0(float x) { return x == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(x); }

// y = the average, turned back; NaN where there are scores but no weight.
template <class T, int D>
__device__ __forceinline__ void kv4_finish(float (&x)[D / 64], float top, float total, int rotate, uint16_t* y) {
    const int lane = threadIdx.x & 63;
    if (total == 0.0f && top > -__builtin_inff()) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) x[i] = __uint_as_float(kKv4Nan);
    }
    if (rotate) rotate_head<D>(x);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) y[lane * (D / 64) + i] = T::from_f32(x[i] * (1.0f / kPart));
}

// Blocks of four waves that a CU holds, by their registers (three: 168 a lane;
// more key groups or 16 rows of them spill).
constexpr int blocks_a_cu(int dim, int groups, int rows) { return dim == 256 ? 1 : rows == 8 && dim * groups <= 256 ? 3 : 2; }

// RT tiles of TR rows.  TR = 16: a column of the products a row, and a second
// product where q has a second part (LO: rotated, or fp16's 11 bits) and for the
// weights' second part.  TR = 8: columns 8 and on take the second parts of rows
// 0 to 7, half the products (131072 tokens, 4 heads a
// key head: 37.6 -> 36.1 us, 32 ragged sequences 67.2 -> 64.3).
//   The bytes bound it where the cache is long: 131072 tokens of 8 key heads of
// 128 are 142.6 MB, 30.2 us at a large copy's 4.7 TB/s; 5.4 to 5.9 TB/s while all
// blocks read, and some 8 us before that (lengths, table, q's rotation, the first
// loads, each after the other).  Short calls are these waits.
//   Steps of loads in flight a wave: with three blocks a CU one is enough at
// D = 128 (1 / 2 / 3 steps, two blocks: 39.8 / 40.2 / 40.5); D = 64 has the
// registers for two (three blocks: 142).
//   Two and three tiles of several groups do not fit into 256 registers: they
// keep 120 and 228 bytes a lane in scratch memory at D = 64 (three tiles, groups
// of 32, LO false and true), 0 and 44, 68 and 208, 232 and 484 at D = 128 (two
// tiles, groups of 128, 64, 32); a tile of 16 rows 132 at D = 256 with LO and
// groups of 32.
template <class T, int D, int NG, int RT, int TR, bool LO, int W>
__global__ __launch_bounds__(64 * W, W == 4 ? blocks_a_cu(D, NG, TR) : D == 256 ? 1 : 2) void k_attn_kv4(Kv4 c, AttnArgs a, int slots,
                                                                                              int fill, int few, float* parts) {
    constexpr int KS = D / 32, SPG = KS / NG, DT = D / 16, DPG = DT / NG, R = TR * RT;
    constexpr bool HALF = TR == 8;
    constexpr float kMove = 8.0f;   // the maximum follows when weights would pass 2^8
    // From here on the maximum's own rounding shows in the exponents (by 2^-4 at 2^20, by 128 at 2^32).
    constexpr float kFar = 1048576.0f;
    constexpr int kRow = lds_row<D>(), DEPTH = RT == 1 && D == 64 ? 2 : 1;
    // the waves' scales of a step; then their sums of a tile
    extern __shared__ __align__(16) uint32_t lds[];
    static_assert(W * sizeof(Stage<NG>) <= 4 * lds_words<D, W, TR>(), "a step's scales fit where the sums go");
    float* lds_o = reinterpret_cast<float*>(lds);
    __shared__ float lds_top[W][16], lds_sum[W][16];
    const int lane = threadIdx.x & 63, wave = wave_of_block(), col = lane & 15, quad = lane >> 4;
    const int g = blockIdx.x, G = a.Hq / c.heads;
    Kv4Work w;
    if (!kv4_work<R>(c, G, slots, fill, few, false, blockIdx.y + blockIdx.z * gridDim.y, &w)) return;
    const int begin = w.chunk * w.span, end = min(begin + w.span, w.tokens);

    // page of the 16 tokens from `pos` on, -1 past the end
    auto page_at = [&](int pos) { return pos < end ? kv4_page(c, w.b, pos) : -1; };
    const int S1 = (1 << c.page_log2) - 1;
    const size_t code_page = ((size_t)2 * c.heads << c.page_log2) * (D / 2);
    const size_t word_page = ((size_t)2 * c.heads << c.page_log2) * NG;
    const uint8_t* codes_k = c.codes + kv4_codes_at(c, 0, 0, g);
    const uint8_t* codes_v = c.codes + kv4_codes_at(c, 0, 1, g);
    const uint32_t* words_k = c.scales + kv4_scales_at(c, 0, 0, g);
    const uint32_t* words_v = c.scales + kv4_scales_at(c, 0, 1, g);

    // steps in flight, each in registers of its own
    u32x4 vc[DEPTH][DT / 2];
    uint32_t kc[DEPTH][4][KS];
    Words<NG> kw[DEPTH], vw[DEPTH];
    int pv[DEPTH];   // pages of tokens 16 quad + 0..15
    // K rows: MFMA row m of tile (u, j) is token 16 (m / 4) + 8 u + 4 j + m % 4, so that a lane's four results are
    // tokens 16 quad + 8 u + 4 j + 0..3
    auto load_k = [&](int at, int pos, int page_k, int page_w) {
        const int row = ((pos + 16 * (col >> 2)) & S1) + (col & 3);
        const uint8_t* p = codes_k + (size_t)(page_k < 0 ? 0 : page_k) * code_page + kv4_k_byte(D, row, quad * KS);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const Words<KS> v = *reinterpret_cast<const Words<KS>*>(__builtin_assume_aligned(p + x * 4 * (D / 2), KS >= 4 ? 16 : 8));
#pragma unroll
            for (int s = 0; s < KS; ++s) kc[at][x][s] = v.w[s];
        }
        kw[at] = *reinterpret_cast<const Words<NG>*>(__builtin_assume_aligned(
            words_k + (size_t)(page_w < 0 ? 0 : page_w) * word_page + ((pos + lane) & S1) * NG, NG >= 4 ? 16 : 4 * NG));
    };
    auto load_v = [&](int at, int pos, int page) {
        const size_t p = (size_t)(page < 0 ? 0 : page);
        const uint8_t* q = codes_v + p * code_page + kv4_v_byte(D, (pos + 16 * quad) & S1, col);
#pragma unroll
        for (int e = 0; e < DT / 2; ++e) vc[at][e] = *reinterpret_cast<const u32x4*>(q + 256 * e);
        vw[at] = *reinterpret_cast<const Words<NG>*>(__builtin_assume_aligned(
            words_v + p * word_page + ((pos + lane) & S1) * NG, NG >= 4 ? 16 : 4 * NG));
    };
    const Mantissa man = mantissa();
    constexpr int kStride = W * kStep;
    int pos = begin + wave * kStep;
    int pk[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
        pk[i] = page_at(pos + i * kStride + 16 * (col >> 2));
        pv[i] = page_at(pos + i * kStride + 16 * quad);
    }
    int next_k = page_at(pos + DEPTH * kStride + 16 * (col >> 2)), next_v = page_at(pos + DEPTH * kStride + 16 * quad);
    // rows of the tiles: what they see, and q
    int seen[RT];
    u32x4 qh[RT][KS], ql[RT][LO && !HALF ? KS : 1];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        // a column past the last row repeats it
        const int r = min((w.tile * RT + t) * TR + (HALF ? col & 7 : col), w.rows * G - 1), i = r / G, h = g * G + r % G;
        seen[t] = w.tokens - w.rows + i + 1;
        const uint16_t* p = a.q + (w.first + i) * a.q_row + h * a.q_head + 8 * quad;
#pragma unroll
        for (int s = 0; s < KS; ++s) qh[t][s] = *reinterpret_cast<const u32x4*>(p + 32 * s);
    }
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
        if (pos + i * kStride < end) {
            load_k(i, pos + i * kStride, pk[i], pv[i]);
            load_v(i, pos + i * kStride, pv[i]);
        }
    // The Hadamard matrix as an operand: (-1)^popcount(d & d'), row m of tile u for d' = 32 (u / 2) + 8 (m / 4) +
    // 4 (u % 2) + m % 4, so that a lane's results are the d' = 32 s + 8 quad + 0..7 that it needs; here the bits of
    // d = 8 quad + j and of d' below 32.  Times 2^-4, so that no sum passes float32 where its turned value does not.
    u32x4 hadamard[2];
    if (LO && c.rotate) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v = 0x3D803D80u;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    v ^= (uint32_t)((__popc((2 * j + x) & (4 * u + (col & 3))) ^ __popc(quad & (col >> 2))) & 1) << (15 + 16 * x);
                hadamard[u][j] = v;
            }
    }
    float qs[RT][NG];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        float x[KS][8];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (a.scale < 0.0f) qh[t][s] ^= 0x80008000u;   // its sign goes to q
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[s][2 * j] = T::to_f32(qh[t][s][j] & 0xFFFFu);
                x[s][2 * j + 1] = T::to_f32(qh[t][s][j] >> 16);
            }
            if (a.scale == 0.0f) {   // goes to q, whose infinities and NaN it turns into NaN
#pragma unroll
                for (int j = 0; j < 8; ++j) x[s][j] *= 0.0f;
            }
        }
        if (LO && c.rotate) {
            u32x4 part[2][KS];
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t hi, lo;
                    split2(x[s][2 * j], x[s][2 * j + 1], &hi, &lo);
                    part[0][s][j] = hi;
                    part[1][s][j] = lo;
                }
#pragma unroll
            for (int u = 0; u < DT; ++u) {
                f32x4 acc = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const u32x4 sign = __builtin_popcount(s & (u / 2)) & 1 ? hadamard[u % 2] ^ 0x80008000u : hadamard[u % 2];
                    acc = Bf16::mfma(sign, part[0][s], acc);
                    // (fp16's second parts are exact, bf16 has none)
                    if constexpr (std::is_same_v<T, Fp16>) acc = Bf16::mfma(sign, part[1][s], acc);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) x[u / 2][4 * (u % 2) + j] = acc[j] * (16.0f * kv4_norm<D>());
            }
        }
        // u times the sums of what the operands hold, group by group
#pragma unroll
        for (int n = 0; n < NG; ++n) qs[t][n] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi, lo;
                split2(x[s][2 * j], x[s][2 * j + 1], &hi, &lo);
                if (HALF && col >= 8) hi = lo;
                qh[t][s][j] = hi;
                float v = kUnit * bf16_lo(hi) + kUnit * bf16_hi(hi);
                if constexpr (LO && !HALF) {
                    ql[t][s][j] = lo;
                    v += kUnit * bf16_lo(lo) + kUnit * bf16_hi(lo);
                }
                qs[t][s / SPG] += v;
            }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            qs[t][n] += __shfl_xor(qs[t][n], 16);
            qs[t][n] += __shfl_xor(qs[t][n], 32);
        }
    }

    f32x4 o[RT][DT] = {}, zp[RT][NG] = {};   // zp: sums of weights times u (1 + z / 16)
    uint32_t poison[RT] = {};                // bit n: group n of V is NaN
    constexpr uint32_t kSeen = 1u << 31;     // a token has scored -infinity where there was no other
    // bit n: group n of V has had a scale beyond kLarge, and its scales and sums carry kShrink from then on: below it
    // 2^30 tokens' sums, of weights of up to 2^8, stay under 2^110
    uint32_t shrunk = 0;
    constexpr uint32_t kLarge = 0x67800000u, kInfinity = 0x7F800000u;   // 2^80
    constexpr float kShrink = 0x1p-64f;
    float top[RT], sum[RT];
    bool far[RT];   // of some row of the tile: a maximum beyond kFar, or none yet
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        far[t] = true;
        top[t] = -__builtin_inff();
        sum[t] = 0.0f;
    }
    // masked scores become -infinity times cs; a scale of 0, which would make NaN of them, is in q
    const float cs = 16.0f / kUnit * (a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.4426950408889634f);

    Stage<NG>& stage = reinterpret_cast<Stage<NG>*>(lds)[wave];
    auto step = [&](auto slot) {
        constexpr int at = slot;
        // scales and 1 + z / 16 through LDS: a token's own lane has them, its 16 lanes need them; of tokens that are
        // not there, zeros
        uint64_t odd;   // tokens with a V of NaN or beyond kLarge
        {
            const bool there = pos + lane < end && pv[at] >= 0;
            const int place = (lane & ~7) | (lane & 4) | (lane & 1) << 1 | (lane >> 1 & 1);   // 0 2, 1 3, 4 6, 5 7
            uint32_t most = 0;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const uint32_t k = there ? kw[at].w[n] : 0, v = there ? vw[at].w[n] : 0;
                stage.ks[n][lane] = __uint_as_float(k & ~15u);
                stage.kz[n][lane] = __uint_as_float((k & 15u) << 19 | 0x3F800000u);
                stage.vs[n][lane] = __uint_as_float(v & ~15u);
                stage.vz[n][place] = (uint16_t)((v & 15u) << 3 | kUnitBf16);
                most = max(most, v);
            }
            odd = __ballot(most >= kLarge);
            if (odd != 0 || shrunk != 0) {
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    const uint32_t v = there ? vw[at].w[n] : 0;
                    const bool nan = v >= kInfinity;
                    if (!(shrunk >> n & 1) && __any(v >= kLarge && !nan)) {
                        shrunk |= 1u << n;
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            zp[t][n] *= kShrink;
#pragma unroll
                            for (int d = n * DPG; d < (n + 1) * DPG; ++d) o[t][d] *= kShrink;
                        }
                    }
                    stage.vs[n][lane] = nan ? 0.0f : __uint_as_float(v & ~15u) * (shrunk >> n & 1 ? kShrink : 1.0f);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        float s[RT][16];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            // one tile's sums at a time: made side by side, all 16 would take registers that there are not
            if (NG * RT > 1 && x > 0) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    asm volatile("" : "+v"(s[t][4 * x - 4]), "+v"(s[t][4 * x - 3]), "+v"(s[t][4 * x - 2]), "+v"(s[t][4 * x - 1]));
#pragma unroll
                for (int k = 0; k < KS; ++k) asm volatile("" : "+v"(kc[at][x][k]));
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const f32x4 sc = *reinterpret_cast<const f32x4*>(&stage.ks[n][16 * quad + 4 * x]);
                const f32x4 z = *reinterpret_cast<const f32x4*>(&stage.kz[n][16 * quad + 4 * x]);
                f32x4 acc[RT] = {};
#pragma unroll
                for (int k = n * SPG; k < (n + 1) * SPG; ++k) {
                    const u32x4 op = kv4_operand(man, kc[at][x][k]);
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        acc[t] = Bf16::mfma(op, qh[t][k], acc[t]);
                        if constexpr (LO && !HALF) acc[t] = Bf16::mfma(op, ql[t][k], acc[t]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const float d = __builtin_fmaf(-z[i], qs[t][n], acc[t][i]);
                        s[t][4 * x + i] = n == 0 ? sc[i] * d : __builtin_fmaf(sc[i], d, s[t][4 * x + i]);
                    }
            }
        }
        if constexpr (HALF) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[t][i] += lane_xor<8>(s[t][i]);   // the parts' scores together, in both
        }
        // a later step's K while this one's weights and V are at work
        const int page = pv[at], ahead = pos + DEPTH * kStride;
        if (ahead < end) load_k(at, ahead, next_k, next_v);
        pv[at] = next_v;
        next_k = page_at(ahead + kStride + 16 * (col >> 2));
        next_v = page_at(ahead + kStride + 16 * quad);

        int lim[RT];
        bool cut = false;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            lim[t] = page < 0 ? 0 : min(seen[t], end) - pos - 16 * quad;
            cut |= lim[t] < 16;
        }
        const bool masked = __any(cut);
        if (masked) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i >= lim[t]) s[t][i] = -__builtin_inff();
            asm volatile("");   // a branch, not 32 instructions of every step
        }
        // rows that see a token whose V is NaN: their sums are made NaN at the end (0 times it would reach the others)
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            if (odd == 0) break;
            const uint64_t nans = __ballot(pos + lane < end && page >= 0 && vw[at].w[n] >= kInfinity);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const uint32_t visible = lim[t] >= 16 ? 0xFFFFu : lim[t] > 0 ? (1u << lim[t]) - 1 : 0u;
                if ((uint32_t)(nans >> (16 * quad)) & visible) poison[t] |= 1u << n;
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float m = s[t][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) m = fmaxf(m, s[t][i]);
            m *= cs;
            if (__any(m > top[t] + kMove)) {
                m = fmaxf(m, __shfl_xor(m, 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                const float up = fmaxf(top[t], m), f = top[t] == up ? 1.0f : __builtin_amdgcn_exp2f(top[t] - up);
                top[t] = up;
                far[t] = __any(!(fabsf(up) <= kFar));
                sum[t] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[t][d] *= f;
#pragma unroll
                for (int n = 0; n < NG; ++n) zp[t][n] *= f;
            }
            float c1 = cs, off = -top[t];
            if (far[t]) {
                // The product is rounded as the maximum's was, so that the maximum's own exponent is 0; unrounded it
                // would be up to half of the maximum's last place.  The tile's other rows are not: their bits are
                // theirs alone.
                const float base = top[t] == -__builtin_inff() ? 0.0f : top[t];   // a row that has seen nothing yet
                const bool own = fabsf(base) > kFar;
                if (lim[t] > 0 && top[t] == -__builtin_inff()) poison[t] |= kSeen;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[t][i] = own ? s[t][i] * cs - base : __builtin_fmaf(s[t][i], cs, -base);
                c1 = 1.0f;
                off = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], c1, off));
                sum[t] += s[t][i];
            }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (NG * RT > 1) {   // as above
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(s[t][8 * u + i]));
                }
                // weights times scales, in V's order of tokens, and the operand u (1 + z / 16)
                const f32x4 sc[2] = {*reinterpret_cast<const f32x4*>(&stage.vs[n][16 * quad + 8 * u]),
                                     *reinterpret_cast<const f32x4*>(&stage.vs[n][16 * quad + 8 * u + 4])};
                const u32x4 zo = *reinterpret_cast<const u32x4*>(&stage.vz[n][16 * quad + 8 * u]);
                u32x4 hi[RT], lo[RT];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t0 = 4 * (j / 2) + j % 2, t1 = t0 + 2;
                    const float s0 = sc[j / 2][j % 2], s1 = sc[j / 2][j % 2 + 2];
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const float x0 = s[t][8 * u + t0] * s0, x1 = s[t][8 * u + t1] * s1;
                        uint32_t h, l;
                        split2(x0, x1, &h, &l);
                        hi[t][j] = HALF && col >= 8 ? l : h;
                        lo[t][j] = l;
                    }
                }
                if constexpr (NG * RT > 1) {
#pragma unroll
                    for (int t = 0; t < RT; ++t) asm volatile("" : "+v"(hi[t]), "+v"(lo[t]));
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    zp[t][n] = Bf16::mfma(zo, hi[t], zp[t][n]);
                    if constexpr (!HALF) zp[t][n] = Bf16::mfma(zo, lo[t], zp[t][n]);
                }
#pragma unroll
                for (int d = n * DPG; d < (n + 1) * DPG; ++d) {
                    const u32x4 op = d % 2 ? kv4_v_operand<true>(man, vc[at][d / 2][2 * u], vc[at][d / 2][2 * u + 1])
                                           : kv4_v_operand<false>(man, vc[at][d / 2][2 * u], vc[at][d / 2][2 * u + 1]);
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        o[t][d] = Bf16::mfma(op, hi[t], o[t][d]);
                        if constexpr (!HALF) o[t][d] = Bf16::mfma(op, lo[t], o[t][d]);
                    }
                }
            }
        }
        if (ahead < end) load_v(at, ahead, pv[at]);
        pos += kStride;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    while (pos < end) {
        step(std::integral_constant<int, 0>());
        if constexpr (DEPTH == 2) {
            if (pos >= end) break;
            step(std::integral_constant<int, 1>());
        }
    }

    // the waves' results joined: rows of the tile, wave by wave
    const bool whole = w.chunks == 1;
    float* part = parts + ((size_t)g * slots + w.slot) * part_words<D, R>();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        sum[t] += __shfl_xor(sum[t], 16);
        sum[t] += __shfl_xor(sum[t], 32);
        poison[t] |= __shfl_xor(poison[t], 16);
        poison[t] |= __shfl_xor(poison[t], 32);
        const float share = 16.0f / kUnit * kPart * reciprocal_or_0(sum[t]);
        __syncthreads();   // the words, or the last tile's rows, were read
        if (quad == 0) {
            lds_top[wave][col] = top[t] == -__builtin_inff() && (poison[t] & kSeen) ? kNoScore : top[t];
            lds_sum[wave][col] = sum[t];
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = poison[t] >> (d / DPG) & 1 ? __uint_as_float(kKv4Nan)
                                                  : (shrunk >> (d / DPG) & 1 ? share / kShrink : share) * (o[t][d][i] - zp[t][d / DPG][i]);
            if constexpr (HALF) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += lane_xor<8>(v[i]);
            }
            if (!HALF || col < 8) *reinterpret_cast<f32x4*>(lds_o + (wave * TR + col) * kRow + 16 * d + 4 * quad) = v;
        }
        __syncthreads();
        const int r0 = (w.tile * RT + t) * TR, n = min(TR, w.rows * G - r0);
        for (int r = wave; r < n; r += W) {
            float m = lds_top[0][r], total = 0.0f, x[D / 64] = {}, of[W];
#pragma unroll
            for (int k = 1; k < W; ++k) m = fmaxf(m, lds_top[k][r]);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                // a wave that has seen nothing has a sum of 0, or NaN
                of[k] = lds_sum[k][r] * (lds_top[k][r] == m || lds_top[k][r] == -__builtin_inff()
                                             ? 1.0f : __builtin_amdgcn_exp2f(lds_top[k][r] - m));
                total += of[k];
            }
            const float inv = reciprocal_or_0(total);
#pragma unroll
            for (int k = 0; k < W; ++k)
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    x[i] = __builtin_fmaf(of[k] * inv, lds_o[(k * TR + r) * kRow + lane * (D / 64) + i], x[i]);
            if (whole) {
                const int i0 = (r0 + r) / G, h = g * G + (r0 + r) % G;
                kv4_finish<T, D>(x, m, total, c.rotate, a.y + ((int64_t)(w.first + i0) * a.Hq + h) * D);
            } else {
                float* p = part + (TR * t + r) * D + lane * (D / 64);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) p[i] = x[i];
                if (lane == 0) {
                    part[R * D + TR * t + r] = m;
                    part[R * (D + 1) + TR * t + r] = total;
                }
            }
        }
    }
}

// The slots of a tile group's spans joined: a block a row, its waves every
// fourth span, 16 at a time, so that few loads wait for each other.
constexpr int kJoinWaves = 4;
template <class T, int D, int R>
__global__ __launch_bounds__(64 * kJoinWaves) void k_attn_kv4_join(Kv4 c, AttnArgs a, int slots, int fill, int few, int row_blocks,
                                                                   const float* parts) {
    constexpr int N = D / 64, W = kJoinWaves;
    constexpr size_t P = part_words<D, R>();
    __shared__ float lds_x[W][D], lds_sum[W], lds_top[W];
    const int lane = threadIdx.x & 63, wave = wave_of_block();
    const int g = blockIdx.x / row_blocks, G = a.Hq / c.heads;
    Kv4Work w;
    if (!kv4_work<R>(c, G, slots, fill, few, true, blockIdx.y + blockIdx.z * gridDim.y, &w) || w.chunks == 1) return;
    const int r0 = w.tile * R, n = min(R, w.rows * G - r0);
    const float* part = parts + ((size_t)g * slots + w.slot) * P;
    for (int r = blockIdx.x % row_blocks; r < n; r += row_blocks) {
        float m = -__builtin_inff(), total = 0.0f, x[N] = {};
        for (int k0 = wave; k0 < w.chunks; k0 += W * 16) {
            // lane i: the maximum and the sum of span k0 + W i, i < 16
            const int some = min(16, (w.chunks - k0 + W - 1) / W), k = k0 + W * min(lane, some - 1);
            const float top = part[k * P + R * D + r], sum = part[k * P + R * (D + 1) + r];
            float y[16][N];
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int d = 0; d < N; ++d) y[i][d] = part[(k0 + W * min(i, some - 1)) * P + r * D + lane * N + d];
            float up = fmaxf(m, top);
#pragma unroll
            for (int i = 1; i < 16; i <<= 1) up = fmaxf(up, __shfl_xor(up, i));
            up = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(up)));
            // the sum of a span that saw nothing is 0, or NaN
            const float f = top == up || top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top - up);
            const float before = total * (m == up || m == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - up));
            const float of = lane < some ? f * sum : 0.0f;
            m = up;
            total = before + __int_as_float(__builtin_amdgcn_readlane(wave_scan(__float_as_int(of), add_floats), 63));
            const float inv = reciprocal_or_0(total), share = of * inv;
#pragma unroll
            for (int d = 0; d < N; ++d) x[d] *= before * inv;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (i >= some) continue;
                const float si = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(share), i));
#pragma unroll
                for (int d = 0; d < N; ++d) x[d] = __builtin_fmaf(si, y[i][d], x[d]);
            }
        }
#pragma unroll
        for (int d = 0; d < N; ++d) lds_x[wave][lane * N + d] = x[d];
        if (lane == 0) {
            lds_sum[wave] = total;
            lds_top[wave] = m;
        }
        __syncthreads();
        if (wave == 0) {
            float up = m;
#pragma unroll
            for (int k = 1; k < W; ++k) up = fmaxf(up, lds_top[k]);
            float of[W];
            total = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                of[k] = lds_sum[k] * (lds_top[k] == up || lds_top[k] == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(lds_top[k] - up));
                total += of[k];
            }
            const float inv = reciprocal_or_0(total);
#pragma unroll
            for (int d = 0; d < N; ++d) x[d] = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
#pragma unroll
                for (int d = 0; d < N; ++d) x[d] = __builtin_fmaf(of[k] * inv, lds_x[k][lane * N + d], x[d]);
            const int i0 = (r0 + r) / G, h = g * G + (r0 + r) % G;
            kv4_finish<T, D>(x, up, total, c.rotate, a.y + ((int64_t)(w.first + i0) * a.Hq + h) * D);
        }
        __syncthreads();
    }
}

// f(head's size, groups of a head), as constants.
template <class F>
void by_form(const Kv4& c, F f) {
    const auto groups = [&](auto d, auto n) {
        if (c.dim == d && c.dim / c.group == n) f(d, n);
    };
    const std::integral_constant<int, 64> d64;
    const std::integral_constant<int, 128> d128;
    const std::integral_constant<int, 256> d256;
    const std::integral_constant<int, 1> n1;
    const std::integral_constant<int, 2> n2;
    const std::integral_constant<int, 4> n4;
    const std::integral_constant<int, 8> n8;
    groups(d64, n1);
    groups(d64, n2);
    groups(d128, n1);
    groups(d128, n2);
    groups(d128, n4);
    groups(d256, n2);
    groups(d256, n4);
    groups(d256, n8);
}

}  // namespace

hipError_t launch_kv4_append(bool fp16, const uint16_t* k, int64_t k_row, int64_t k_head, const uint16_t* v,
                             int64_t v_row, int64_t v_head, const Kv4& c, hipStream_t st) {
    const AppendArgs a{c, {k, v}, {k_row, v_row}, {k_head, v_head}};
    // groups of 16 rows that B sequences' T tokens can lie in
    const int64_t n = ((int64_t)c.T + 30 * (int64_t)(c.B < c.T ? c.B : c.T)) / 16;
    const int y = (int)(n < 32768 ? n : 32768);
    const dim3 grid((2 * c.heads + 3) / 4, y, (unsigned)((n + y - 1) / y));
    by_form(c, [&](auto d, auto ng) {
        if (fp16) k_kv4_append<Fp16, d, ng><<<grid, 256, 0, st>>>(a);
        else k_kv4_append<Bf16, d, ng><<<grid, 256, 0, st>>>(a);
    });
    return hipGetLastError();
}

namespace {

// Rows a block takes, in tiles of 16; the tile groups that there can be; the
// blocks of a head that the chip runs at once, two a CU at most (few) or all
// (fill), and those that the grid has;
// none where no sequence is worth a second span.
// Tokens up to which one block takes a sequence, with twice the waves: two
// turns of them.
constexpr int kOneSpan = 1024;
struct Grid {
    int tiles, rows, groups, slots, fill, few;   // rows: of a tile
};
Grid attn_kv4_grid(int T, int G, int heads, int dim, int scales, int page, int width, int B) {
    Grid g;
    const int most = dim == 64 ? max_tiles<64>() : dim == 128 ? max_tiles<128>() : max_tiles<256>();
    const int64_t rows = ((int64_t)T * G + B - 1) / B;   // of a sequence, on average
    g.rows = rows <= 8 ? 8 : 16;
    g.tiles = rows > 16 * most ? most : (int)(rows + 15) / 16;
    const int R = g.rows * g.tiles;
    // a sequence's rows are a multiple of G: the last group of each lacks at most R - gcd(G, R)
    g.groups = (int)(((int64_t)T * G + (int64_t)(B < T ? B : T) * (R - std::gcd(G, R))) / R);
    g.slots = g.fill = g.few = 0;
    if ((int64_t)width * page > kOneSpan) {
        const int blocks = blocks_a_cu(dim, scales, g.rows);
        g.fill = std::max(256 * blocks / heads, 1);
        g.few = std::max(256 * std::min(blocks, 2) / heads, 1);
        g.slots = 2 * g.fill + g.groups + 1;
    }
    return g;
}
size_t part_bytes(int dim, int rows) { return (size_t)rows * (dim + 2) * 4; }

template <class T, int D, int NG, int RT, int TR, int W>
hipError_t run_attn_kv4(const AttnArgs& a, const Kv4& c, const Grid& g, float* ws, hipStream_t st) {
    const auto grid = [&](int n, int x) {
        const int y = n < 32768 ? n : 32768;
        return dim3(x, y, (n + y - 1) / y);
    };
    constexpr int R = TR * RT, lds = 4 * lds_words<D, W, TR>();
    hipError_t e = hipSuccess;
    const auto go = [&](auto kernel, std::atomic<uint64_t>& done) {
        if (lds > 65536 && (e = opt_in_lds(reinterpret_cast<const void*>(kernel), lds, done)) != hipSuccess) return;
        kernel<<<grid(g.slots ? g.slots : g.groups, c.heads), 64 * W, lds, st>>>(c, a, g.slots, g.fill, g.few, ws);
        e = hipGetLastError();
    };
    static std::atomic<uint64_t> done[2];
    if (TR == 8 || c.rotate || a.fp16) go(k_attn_kv4<T, D, NG, RT, TR, true, W>, done[0]);
    else if constexpr (TR == 16) go(k_attn_kv4<T, D, NG, RT, TR, false, W>, done[1]);
    if (e != hipSuccess || g.slots == 0) return e;
    // as many blocks as a group has rows on average, while there are few groups: some 1024 in all.  us a call, a block
    // a row / 1024 / 512: 64 sequences of 4000 tokens (joins nothing) 82 / 79.5 / 78.7, 4 of 8 new tokens 35 / 35 /
    // 37.6, 2 of 200 145 / 126 / 125
    const int64_t rows = ((int64_t)c.T * (a.Hq / c.heads) + g.groups - 1) / g.groups;
    const int64_t most = 1024 / ((int64_t)g.groups * c.heads) + 1;
    const int row_blocks = (int)(rows < R ? (rows < most ? rows : most) : (R < most ? R : most));
    k_attn_kv4_join<T, D, R><<<grid(g.groups, c.heads * row_blocks), 64 * kJoinWaves, 0, st>>>(c, a, g.slots, g.fill, g.few, row_blocks, ws);
    return hipGetLastError();
}

}  // namespace

size_t attn_kv4_workspace(int T, int Hq, int heads, int dim, int group, int page, int width, int B) {
    if (T == 0 || B == 0) return 0;
    const Grid g = attn_kv4_grid(T, Hq / heads, heads, dim, dim / group, page, width, B);
    return (size_t)g.slots * heads * part_bytes(dim, g.rows * g.tiles);
}

hipError_t launch_attn_kv4(const AttnArgs& a, const Kv4& c, void* ws, hipStream_t st) {
    const Grid g = attn_kv4_grid(c.T, a.Hq / c.heads, c.heads, c.dim, c.dim / c.group, 1 << c.page_log2, c.width, c.B);
    hipError_t e = hipErrorInvalidValue;
    by_form(c, [&](auto d, auto ng) {
        const auto tiles = [&](auto rt, auto rows) {
            if constexpr (rt <= max_tiles<d>()) {
                if (g.tiles != rt || g.rows != rows) return;
                const auto run = [&](auto waves) {
                    e = a.fp16 ? run_attn_kv4<Fp16, d, ng, rt, rows, waves>(a, c, g, (float*)ws, st)
                               : run_attn_kv4<Bf16, d, ng, rt, rows, waves>(a, c, g, (float*)ws, st);
                };
                // (a head of 256 takes the registers of two waves)
                if constexpr (d < 256 && rt == 1) {
                    if (g.slots == 0) return run(std::integral_constant<int, 8>());
                }
                run(std::integral_constant<int, 4>());
            }
        };
        const std::integral_constant<int, 16> sixteen;
        tiles(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
        tiles(std::integral_constant<int, 1>(), sixteen);
        tiles(std::integral_constant<int, 2>(), sixteen);
        tiles(std::integral_constant<int, 3>(), sixteen);
    });
    return e;
}

}  // namespace cr
