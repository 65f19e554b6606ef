// Attention over whole prompts: packed sequences, grouped heads, causal or
// both ways.
//
//   y[i, h] = T(sum_j p[i, j] v[j, h / G] / sum_j p[i, j]),
//   p[i, j] = exp(scale q[i, h] . k[j, h / G]),
// j over the tokens of i's sequence, up to i if causal.
#include <type_traits>

#include "cr_w4g.h"

namespace cr {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ f32x16 mfma32(Bf16, u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(Fp16, u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(Bf16, float a, float b) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t pack2(Fp16, float a, float b) {
    f32x2_t f;
    f.x = a; f.y = b;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
}

// sum + the two values of p
__device__ __forceinline__ float add2(Bf16, uint32_t p, float sum) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, p), __builtin_bit_cast(bf16x2_t, 0x3F803F80u), sum, false);
}
__device__ __forceinline__ float add2(Fp16, uint32_t p, float sum) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, p), __builtin_bit_cast(f16x2, 0x3C003C00u), sum, false);
}

// Two values of 0 times: a scale of 0 goes to q, whose infinities and NaN it turns into NaN.
template <class T>
__device__ __forceinline__ uint32_t none_of(uint32_t v) {
    constexpr uint32_t top = std::is_same_v<T, Fp16> ? 0x7C00u : 0x7F80u;
    return ((v & top) == top ? 0x7FFFu : 0u) | ((v >> 16 & top) == top ? 0x7FFF0000u : 0u);
}

// One row by one wave, without matrix cores: only what the row sees is touched.
// A lane takes a key of 64, then d = l D / 64 and on.  o holds the average so
// far, which is no larger than v is.  Ends when every value is NaN.
template <class T, int D>
__device__ __forceinline__ void attn_row(const uint16_t* q, const uint16_t* k, int64_t k_row, const uint16_t* v, int64_t v_row,
                              int keys, float scale, uint16_t* y) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63;
    float top = -__builtin_inff(), sum = 0.0f, o[N] = {};
    for (int j0 = 0; j0 < keys; j0 += 64) {
        const int n = min(64, keys - j0);
        const uint16_t* kr = k + (int64_t)(j0 + min(lane, n - 1)) * k_row;
        float s = 0.0f;
        for (int d = 0; d < D; d += 8) {
            float x[8], w[8];
            w4g_values<T>(q + d, x);
            w4g_values<T>(kr + d, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __builtin_fmaf(scale == 0.0f ? x[i] * 0.0f : x[i], w[i], s);
        }
        s = lane < n ? s * scale : -__builtin_inff();
        float m = s;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
        const float up = fmaxf(top, m), f = top == up ? 1.0f : expf(top - up);
        // keys of a score of -infinity weigh nothing, also where there has been no other yet
        const float p = up > -__builtin_inff() ? (lane < n ? expf(s - up) : 0.0f) : s == s ? 0.0f : s;
        float all = p;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) all += __shfl_xor(all, x);
        const float total = sum * f + all, inv = total == 0.0f ? 0.0f : 1.0f / total, keep = sum * f * inv;
        sum = total;
        top = up;
        bool open = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!(fabsf(o[i]) == __builtin_inff())) o[i] *= keep;
            open |= o[i] == o[i];
        }
        if (!__any(open)) break;
        // what an infinity is multiplied with: a weight that is 0 in float32 alone is none of the definition's
        const float share = p * inv, some = s > -__builtin_inff() ? fmaxf(share, 1e-30f) : share;
        for (int j = 0; j < n; ++j) {
            const float w = __shfl(share, j), w_inf = __shfl(some, j);
            const uint16_t* vr = v + (int64_t)(j0 + j) * v_row + lane * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = T::to_f32(vr[i]);
                o[i] = __builtin_fmaf(fabsf(x) == __builtin_inff() ? w_inf : w, x, o[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) y[lane * N + i] = T::from_f32(sum == 0.0f ? __builtin_nanf("") : o[i]);
}

// The sequence and the tile of BM rows in it that tile `t` from the end is:
// sequences' tiles counted one after the other.  Every wave counts for itself.
struct Tile {
    int first, len, row;   // the sequence's first row and its length; the tile's first row in it
};
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* cu, int B, int T, int t, Tile* out) {
    const int lane = threadIdx.x & 63;
    auto rows_of = [&](int b0, int* first) {
        const int b = min(b0 + lane, B - 1);
        *first = min(max(cu[b], 0), T);
        return b0 + lane < B ? min(max(cu[b + 1], *first), T) - *first : 0;
    };
    int first0;
    const int len0 = rows_of(0, &first0);
    int total = __builtin_amdgcn_readlane(wave_scan((len0 + BM - 1) / BM, add_ints), 63);
    for (int b0 = 64; b0 < B; b0 += 64) {
        int first;
        const int len = rows_of(b0, &first);
        total += __builtin_amdgcn_readlane(wave_scan((len + BM - 1) / BM, add_ints), 63);
    }
    int left = total - 1 - t;   // tiles before this one
    if (left < 0) return false;
    for (int b0 = 0; b0 < B; b0 += 64) {
        int first = first0, len = len0;
        if (b0 > 0) len = rows_of(b0, &first);
        const int n = (len + BM - 1) / BM, upto = wave_scan(n, add_ints);
        const uint64_t after = __ballot(upto > left);
        if (after) {
            const int l = __builtin_ctzll(after);
            out->first = __builtin_amdgcn_readlane(first, l);
            out->len = __builtin_amdgcn_readlane(len, l);
            out->row = (left - __builtin_amdgcn_readlane(upto - n, l)) * BM;
            return true;
        }
        left -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Rows of K or V in LDS: 16-byte chunk c of row r at chunk c ^ swizzle(r).
// K is read 16 rows at one chunk, V 4 rows at four chunks (64 bytes): either
// way all banks are hit alike.
template <int D, bool V>
__device__ __forceinline__ int swizzle(int r) {
    constexpr int rows = D >= 128 ? 1 : 128 / D;   // rows in 256 bytes
    return V ? ((r / rows) & (rows > 1 ? 1 : 3)) * 4 : (r / rows) & (rows > 1 ? 7 : 15);
}

// Bytes of an output row in LDS; of a block: two buffers of K and V for each
// half of the waves, later its rows.
template <int D>
constexpr int out_row() { return 2 * D + 16; }
template <int D, int NW, int BN, int KG>
constexpr int lds_bytes() {
    constexpr int tiles = KG * 4 * BN * D * 2, rows = NW * 32 * out_row<D>();
    return tiles > rows ? tiles : rows;
}

// One block: BM = 32 NW rows of one head, a wave 32 of them, over tiles of BN
// keys that NW waves share in LDS, the next tile's on their way meanwhile.
// KG = 2: twice the waves, the second half on the odd tiles, its sums joined to
// the first half's at the end.
//   S^T = K Q^T   MFMA 32x32x16: a lane holds 16 keys' scores of one row
//   O^T = V^T P^T the same lane's weights are the second operand as they lie:
//                 step s takes its scores 8 s + 0..7, keys 16 s + 8 (i / 4) + 4 (lane / 32) + i % 4;
//                 V's operand comes transposed from LDS, 4 keys a read
// The weights go to the second product in T's 16 bits, as q, k and v are (a
// second part would double that product): largest error on standard normal
// values, bf16, 0.0018 to 0.0023, with float32 weights 0.0016.  Their sum is of
// the rounded weights.  fp16 weights carry 2^6.
//   Long prompts: the matrix units' time and the chip's power.  16384 tokens, 32
// heads of 128, causal: 2.2 TF, 1.95 to 2.07 ms (1.06 to 1.13 PF; a large product
// reaches 1.43); the products alone took 1.29 ms, and the clock holds 1.8 GHz; of
// some 1600 cycles a 128 x 64 tile and CU the units work 1024.  Short ones: the
// longest row block, one tile after the other (1220 tokens: 20 tiles of 0.8 us,
// 8 us before and behind them).  Not faster: halves of the waves that alternate
// products and weights (1220 tokens 26.8 -> 28.9 us), reads of LDS sent 4 to 8
// products ahead, wave priorities, 8 waves of rows (16384 tokens -3 %, 2500 +12 %).
template <class T, int D, int NW, int BN, int KG>
__global__ __launch_bounds__(64 * NW * KG, D == 256 ? 1 : 2) void k_attn_prompt(AttnArgs a) {
    constexpr int BM = 32 * NW, KS = D / 16, DT = D / 32, MT = BN / 32, PS = BN / 16;
    constexpr int kTile = BN * D * 2, kLoads = kTile / 1024 / NW;   // bytes of a K or V tile; 1 KiB loads of a wave
    constexpr bool MEET = KG == 2 && NW == 2, BETWEEN = NW == 4;
    constexpr float kMove = 8.0f;   // the maximum follows when weights would pass 2^8
    // fp16 weights: 2^6 at the maximum, so that fewer fall below its normal range
    constexpr float kBias = std::is_same_v<T, Fp16> ? 6.0f : 0.0f;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, wave = wave_of_block() % NW, kg = wave_of_block() / NW;
    Tile t;
    if (!find_tile<BM>(a.cu, a.B, a.T, blockIdx.y + blockIdx.z * gridDim.y, &t)) return;
    // blocks go to the 8 XCDs in turn: heads of one key head to the same one
    int h = blockIdx.x;
    if ((a.Hq & 7) == 0) h = (h & 7) * (a.Hq >> 3) + (h >> 3);
    const int g = h / (a.Hq / a.Hkv);
    const uint16_t* q = a.q + t.first * a.q_row + h * a.q_head;
    const uint16_t* k = a.k + t.first * a.k_row + g * a.k_head;
    const uint16_t* v = a.v + t.first * a.v_row + g * a.v_head;
    const int row0 = t.row + wave * 32, row = row0 + (lane & 31);
    const int keys = a.causal ? min(t.len, t.row + BM) : t.len;
    const int tiles = (keys + BN - 1) / BN;
    const int mine = row0 >= t.len ? 0 : a.causal ? min(row0 + 32, t.len) : t.len;   // keys this wave's rows see

    // the wave's part of a tile's loads: load i fills 1 KiB of K or V, lane by lane
    uint32_t k_off[kLoads], v_off[kLoads];
    auto offsets = [&](int rows) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = (wave * kLoads + i) * 64 + lane, r = at / (D / 8), c = at % (D / 8), rr = min(r, rows - 1);
            k_off[i] = (uint32_t)rr * (uint32_t)a.k_row * 2 + (c ^ swizzle<D, false>(r)) * 16;
            v_off[i] = (uint32_t)rr * (uint32_t)a.v_row * 2 + (c ^ swizzle<D, true>(r)) * 16;
        }
    };
    auto rows_at = [&](const uint16_t* p, int64_t stride, int j) {
        const uint64_t at = (uint64_t)(uintptr_t)(p + (int64_t)j * stride);
        v4i r;
        r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)at);
        r.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xFFFFu));
        r.z = -1;   // every offset lies inside (rows past the last bring the last)
        r.w = 0x00020000;
        return r;
    };
    char* mem = lds + kg * 4 * kTile;   // of this half of the waves: two buffers of K and V
    const uint32_t lds0 = lds_address(mem);
    auto load = [&](int tile, int buffer) {
        const int j = tile * BN;
        if (keys - j < BN) offsets(t.len - j < BN ? t.len - j : BN);
        const v4i kr = rows_at(k, a.k_row, j), vr = rows_at(v, a.v_row, j);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds0 + buffer * 2 * kTile + wave * kLoads * 1024);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) w4g_x_to_lds(kr, k_off[i], to + i * 1024);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) w4g_x_to_lds(vr, v_off[i], to + kTile + i * 1024);
    };
    offsets(min(t.len, BN));
    if (kg < tiles) load(kg, 0);

    u32x4 qv[KS];
    {
        const uint16_t* p = q + (int64_t)min(row, t.len - 1) * a.q_row + 8 * (lane >> 5);
#pragma unroll
        for (int s = 0; s < KS; ++s) qv[s] = *reinterpret_cast<const u32x4*>(p + 16 * s);
        if (!(a.scale > 0.0f)) {   // the sign goes to q, and 0
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) qv[s][j] = a.scale < 0.0f ? qv[s][j] ^ 0x80008000u : none_of<T>(qv[s][j]);
        }
    }
    // Halves of two waves do not wait for each other: each has a count of its waves that have come to a turn (a
    // barrier of the whole block: 600 tokens of 32 heads 16.9 us, this 15.7; D = 256 ragged 59.7 and 56.6; with halves
    // of four waves it is the slower one, 1220 tokens 24.6 and 25.5).
    __shared__ uint32_t came[2];
    if constexpr (MEET) {
        if (threadIdx.x < 2) came[threadIdx.x] = 0;
        __syncthreads();
    }
    auto meet = [&](int turn) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what this wave asked LDS for has been read
        if (lane == 0) __hip_atomic_fetch_add(&came[kg], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        const uint32_t all = (uint32_t)(turn + 1) * NW;
        while (__builtin_amdgcn_readfirstlane(__hip_atomic_load(&came[kg], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)) < all) {}
        asm volatile("" ::: "memory");
    };
    f32x16 o[DT] = {};
    // (a scale of 0 is in q, and would make NaN of the scores that are masked)
    const float c = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.4426950408889634f;
    float top = -__builtin_inff(), sum = 0.0f;   // of the scores times c; this lane's keys

    for (int turn = 0; turn * KG < tiles; ++turn) {
        const int j = turn * KG + kg;
        w4g_wait();
        if constexpr (MEET) meet(turn);
        else w4g_barrier();
        // The next tile's loads.  Blocks of four waves of rows send them between the products, where the wait of one
        // load for another (64 bytes a clock) is hidden: two pictures 225.6 -> 219.1 us, 2500 tokens 64.5 -> 62.5; the
        // others (ragged D = 256 56.7 and 57.4, 20 fp16 prompts 17.4 and 17.7 so) at once.  (Between the products
        // there is no question whether there is a next tile: past the last it comes once more, to where nothing is read.)
        const int next = min(j + KG, tiles - 1) * BN;
        if (keys - next < BN) offsets(t.len - next < BN ? t.len - next : BN);
        const v4i k_next = rows_at(k, a.k_row, next), v_next = rows_at(v, a.v_row, next);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds0 + ((turn + 1) & 1) * 2 * kTile + wave * kLoads * 1024);
        auto piece = [&](int i) {
            if (i < kLoads) w4g_x_to_lds(k_next, k_off[i], to + i * 1024);
            else w4g_x_to_lds(v_next, v_off[i - kLoads], to + kTile + (i - kLoads) * 1024);
        };
        const bool sees = j * BN < mine;
        if ((!BETWEEN || !sees) && j + KG < tiles) {
#pragma unroll
            for (int i = 0; i < 2 * kLoads; ++i) piece(i);
        }
        if (!sees) continue;
        const char* kt = mem + (turn & 1) * 2 * kTile;
        const char* vt = kt + kTile;
        f32x16 s[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[mt] = f32x16{};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int r = 32 * mt + (lane & 31);
                s[mt] = mfma32(T(), *reinterpret_cast<const u32x4*>(kt + r * (2 * D) + ((2 * ks + (lane >> 5)) ^ swizzle<D, false>(r)) * 16),
                               qv[ks], s[mt]);
                if (BETWEEN && mt == MT - 1) {
#pragma unroll
                    for (int i = ks * 2 * kLoads / KS; i < (ks + 1) * 2 * kLoads / KS; ++i) piece(i);
                }
            }
        // this lane's score i of part mt: key j BN + 32 mt + 8 (i / 4) + 4 (lane / 32) + i % 4
        if (j * BN + BN > (a.causal ? min(row0 + 1, t.len) : t.len)) {
            const int last = (a.causal ? min(row, t.len - 1) : t.len - 1) - j * BN - 4 * (lane >> 5);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (32 * mt + 8 * (i / 4) + i % 4 > last) s[mt][i] = -__builtin_inff();
        }
        float m = s[0][0];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, s[mt][i]);
        m *= c;
        if (__any(m > top + kMove)) {
            m = fmaxf(m, __shfl_xor(m, 32));
            const float up = fmaxf(top, m), f = top == up ? 1.0f : __builtin_amdgcn_exp2f(top - up);
            top = up;
            sum *= f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[dt][i] *= f;
        }
        u32x4 p[PS];
        const float off = top == -__builtin_inff() ? 0.0f : kBias - top;   // a row whose keys have all scored -infinity
#pragma unroll
        for (int ps = 0; ps < PS; ++ps) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[ps / 2][8 * (ps % 2) + i], c, off));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[ps][i] = pack2(T(), e[2 * i], e[2 * i + 1]);
                sum = add2(T(), p[ps][i], sum);
            }
        }
        // V^T: the 16 lanes of a group take 4 keys x 16 d, lane i the keys' d = i
        const int vr = 4 * (lane >> 5) + ((lane & 15) >> 2), vc = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
        for (int ps = 0; ps < PS; ++ps) {
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                u32x4 b;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 16 * ps + 8 * x + vr;
                    const char* at = vt + r * (2 * D) + ((4 * dt + vc) ^ swizzle<D, true>(r)) * 16 + (lane & 1) * 8;
                    const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_s16x4*)(__attribute__((address_space(3))) char*)at);
                    const uint2 u = __builtin_bit_cast(uint2, w);
                    b[2 * x] = u.x;
                    b[2 * x + 1] = u.y;
                }
                o[dt] = mfma32(T(), b, p[ps], o[dt]);
            }
        }
    }

    w4g_wait();   // the last loads are in before LDS is used for something else
    sum += __shfl_xor(sum, 32);
    if constexpr (KG == 2) {
        // sums as they lie in the registers: lane by lane, 16 bytes each
        f32x4* to = reinterpret_cast<f32x4*>(lds) + wave * (DT * 4 * 64) + lane;
        float* stat = reinterpret_cast<float*>(lds + NW * DT * 4096) + wave * 128 + lane;
        __syncthreads();   // the last tiles were read
        if (kg == 1) {
#pragma unroll
            for (int i = 0; i < DT * 4; ++i)
                to[i * 64] = f32x4{o[i / 4][i % 4 * 4], o[i / 4][i % 4 * 4 + 1], o[i / 4][i % 4 * 4 + 2], o[i / 4][i % 4 * 4 + 3]};
            stat[0] = top;
            stat[64] = sum;
        }
        __syncthreads();
        if (kg == 0) {
        const float other = stat[0], up = fmaxf(top, other);
        // a half that has seen no key has sums of 0, or NaN
        const float f0 = top == up || top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top - up);
        const float f1 = other == up || other == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(other - up);
        sum = sum * f0 + stat[64] * f1;
#pragma unroll
        for (int i = 0; i < DT * 4; ++i) {
            const f32x4 v = to[i * 64];
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i / 4][i % 4 * 4 + x] = o[i / 4][i % 4 * 4 + x] * f0 + v[x] * f1;
        }
        }
    }
    __syncthreads();   // where the rows go, the last tiles or the other half's sums were read
    if (kg == 1 || row0 >= t.len) return;
    const float inv = 1.0f / sum;
    bool bad = false;
    float y[DT][16];
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            y[dt][i] = o[dt][i] * inv;
            bad |= !w4g_finite(y[dt][i]);
        }
    const uint64_t wrong = __ballot(bad);
    const uint32_t again = (uint32_t)(wrong | wrong >> 32);   // rows that are infinite or NaN somewhere
    // whole rows to memory: by way of LDS, each wave in a place of its own, 16 bytes between its rows (stored as
    // they lie, 8 bytes a lane, 32 rows a store, they took 2 us)
    constexpr int kRow = out_row<D>();
    char* mine_out = lds + wave * 32 * kRow;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            uint2 w;
            w.x = pack2(T(), y[dt][i], y[dt][i + 1]);
            w.y = pack2(T(), y[dt][i + 2], y[dt][i + 3]);
            *reinterpret_cast<uint2*>(mine_out + (lane & 31) * kRow + 8 * (lane >> 5) + 64 * dt + 4 * i) = w;
        }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    uint16_t* out = a.y + ((int64_t)(t.first + row0) * a.Hq + h) * D;
    const int rows = min(32, t.len - row0);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const int r = (i * 64 + lane) / (D / 8), ch = (i * 64 + lane) % (D / 8);
        if (r < rows && !(again >> r & 1))
            *reinterpret_cast<u32x4*>(out + (int64_t)r * a.Hq * D + 8 * ch) =
                *reinterpret_cast<const u32x4*>(mine_out + r * kRow + 16 * ch);
    }
    // A weight of 0 times an infinity or a NaN of a key that the row does not see
    // made some of these: once more, without that key.
    for (uint32_t r = __builtin_amdgcn_readfirstlane(again); r != 0; r &= r - 1) {
        const int i = row0 + __builtin_ctz(r);
        if (i >= t.len) break;
        attn_row<T, D>(q + i * a.q_row, k, a.k_row, v, a.v_row, a.causal ? i + 1 : t.len, a.scale,
                               a.y + ((int64_t)(t.first + i) * a.Hq + h) * D);
    }
}

template <class T, int D, int NW, int BN, int KG>
hipError_t launch(const AttnArgs& a, hipStream_t st) {
    constexpr int BM = 32 * NW, lds = lds_bytes<D, NW, BN, KG>();
    static_assert(KG == 1 || NW * (D / 32 * 4096 + 512) <= lds, "the second half's sums fit");
    static std::atomic<uint64_t> done{0};
    if (lds > 65536) {
        const hipError_t e = opt_in_lds(reinterpret_cast<const void*>(&k_attn_prompt<T, D, NW, BN, KG>), lds, done);
        if (e != hipSuccess) return e;
    }
    // tiles that B sequences of T rows can have
    const int64_t tiles = a.B == 1 ? (a.T + BM - 1) / BM : ((int64_t)a.T + (int64_t)a.B * (BM - 1)) / BM;
    const int y = (int)(tiles < 32768 ? tiles : 32768);
    k_attn_prompt<T, D, NW, BN, KG><<<dim3(a.Hq, y, (unsigned)((tiles + y - 1) / y)), 64 * NW * KG, lds, st>>>(a);
    return hipGetLastError();
}
// What a block takes, by the number of blocks of 128 rows and the sequences'
// mean length (rows of a block / keys of a tile / halves of the waves on the
// keys).  Few blocks: what a block takes is what the call takes, so that 64 rows
// and two halves are best, then 128 and two halves; many: 128 rows load each
// key half as often; sequences shorter than a block leave most of it empty.
// us a call, causal, one sequence or as said:
//                                             128/64/1  128/64/2  64/64/2  64/32/2  64/32/1
//   D = 128, 32 heads: 300 tokens  (96 blocks)    10.7      11.0     10.1     10.2     12.0
//     600 (160)                                   17.1      15.6     15.7     15.2     18.4
//     1220 (320)                                  30.1      24.4     35.9     26.6     34.5
//     2500 (640)                                  63.9      73.0     95.5     77.9     73.7
//     20 of 220 (1408)                            32.5      48.0     73.2     44.9     31.1
//     40 of 60 (1216)                             19.0      37.5     37.1     21.4     16.1
//   D = 64, 16 heads: 600 (80)                    11.9      10.3      9.2      9.8     12.9
//     1220 (160)                                  19.7      15.7     14.6     16.0     23.2
//     2500 (320)                                  36.2      28.6     25.9     29.5     43.7
//     5000 (640)                                  75.9      67.7     78.6     70.9     87.7
//   D = 64, 14 heads: 20 from 0 to 903 (616)      20.9      20.4     21.6     17.6     20.9
//     20 of 220 (616)                             12.9      14.5     17.5     13.2     11.1
//     8 of 1000 (924)                             31.8      33.3     39.1     35.0     32.2
//   D = 64, 32 heads: 64 of 60 (1984)             13.4      23.0     23.4     14.8     11.0
// The host knows T and B, not the lengths.  Where short sequences of heads of 64
// leave some blocks (up to 704), 64/32/2 loses less on like lengths than it
// gains on unlike ones, 14 heads, 64/32/2 and 64/32/1: 30 of 100 9.4 and 8.7, 30
// from 0 to 200 9.6 and 9.2; 20 of 220 13.1 and 11.2, from 0 to 440 12.5 and
// 13.4, from 0 to 900 17.5 and 20.6; 10 of 400 13.7 and 13.5, from 0 to 800 17.1
// and 18.9; 12 from 0 to 600 15.1 and 16.5.
// D = 256 (one wave a SIMD), 128/32/1 and 64/32/2: 16 heads, 300 tokens (48
// blocks) 21.2 / 17.5; 8 heads, 2741 (192) 91 / 57, 16384 (1024) 1410 / 1660.
template <class T, int D>
hipError_t launch_by_size(const AttnArgs& a, hipStream_t st) {
    const int64_t blocks = ((int64_t)a.T / 128 + (a.B + 1) / 2) * a.Hq;   // half a tile lost a sequence
    const int mean = a.T / a.B;
    if constexpr (D == 256) {
        return blocks <= 448 ? launch<T, D, 2, 32, 2>(a, st) : launch<T, D, 4, 32, 1>(a, st);
    } else {
        if (blocks <= (D == 64 ? 352 : 192)) return launch<T, D, 2, 64, 2>(a, st);
        if constexpr (D == 64) {
            if (blocks <= 704 && mean < 512) return launch<T, D, 2, 32, 2>(a, st);
        }
        if (blocks <= (D == 64 ? 704 : 448)) return launch<T, D, 4, 64, 2>(a, st);
        return mean <= 128 ? launch<T, D, 2, 32, 1>(a, st) : launch<T, D, 4, 64, 1>(a, st);
    }
}
template <class T>
hipError_t launch_by_dim(const AttnArgs& a, hipStream_t st) {
    return a.D == 64 ? launch_by_size<T, 64>(a, st) : a.D == 128 ? launch_by_size<T, 128>(a, st) : launch_by_size<T, 256>(a, st);
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t st) {
    return a.fp16 ? launch_by_dim<Fp16>(a, st) : launch_by_dim<Bf16>(a, st);
}

}  // namespace cr
