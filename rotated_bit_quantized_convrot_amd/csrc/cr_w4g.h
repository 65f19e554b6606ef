// 4-bit weights with group scales (W4G): packed layout and the device core
// shared by the linear (cr_w4g.hip) and the mixture-of-experts layer
// (cr_moe.hip).
//
// W[n,k] = s[n, k/g] (q[n,k] - z[n, k/g]),  q in 0..15, z in 0..15 (8 for a
// weight without zero points), s and the activations of one 16-bit type T.
//
// Packed weight, Np = N rounded up to 16, U = ceil(K / 128) units of 128 k:
//   codes   1 KiB tiles (16 rows x 128 k), tile (t, u) at (t U + u) * 1024;
//           lane l of the wave that reads it owns the 16 bytes at 16 l: row
//           16 t + l % 16, dword d holding k = 128 u + 32 d + 8 (l / 16) + 0..7,
//           the B operand of one MFMA 16x16x32: q ^ 8 of k + 2 j in bits 4 j,
//           of k + 2 j + 1 in bits 16 + 4 j (below, the 16-bit types)
//   scales  16-bit, [t][u][row % 16][128 / g]
//   zeros   (weights with zero points) [t][u][row % 16][max(1, 64 / g)]
//           bytes, group i of the unit in bits 4 (i % 2) of byte i / 2
// Rows past N and k past K hold zeros.
#pragma once
#include "cr_device.h"

namespace cr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The 16-bit types: the MFMA, conversions, and an MFMA operand of 8 codes.
// The operand holds (q - z) / 16, exact in both types; the accumulators hold
// a sixteenth of the sums, and the factor 16 is left to who takes them (in the
// scales it would make infinities of those from 2^124 up).
//   fp16  (1 + q / 16) is the code put into the top mantissa bits of 1.0, and
//         one packed add takes 1 + z / 16 off.
//   bf16  has no packed add; v_cvt_off_f32_i4 turns a two's-complement nibble
//         c into c / 16 as float32, whose upper half is that value in bf16.
//         The packed codes are therefore stored as q ^ 8 = q - 8; where a
//         weight has zero points the operand stays (q - 8) / 16 and the
//         sums start from (8 - z) / 16 sum x.
struct Bf16 {
    static constexpr uint32_t kMinusOne = 0xBF80BF80u;
    static constexpr bool kZeroInOperand = false;
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ float to_f32(uint32_t v) { return __uint_as_float(v << 16); }
    static __device__ __forceinline__ uint16_t from_f32(float v) { return (uint16_t)f32_to_bf16_rne(v); }
    static __device__ __forceinline__ u32x4 operand(uint32_t c, uint32_t) {
        // the low nibbles of c's bytes are k 0, 4, 1, 5, those of c >> 4 are k 2, 6, 3, 7
        uint32_t h = c >> 4;
        asm("" : "+v"(h));   // kept as it is: the conversions then take its bytes with no shift of their own
        u32x4 b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = (j & 1) ? h : c;
            const float lo = __builtin_amdgcn_cvt_off_f32_i4((v >> (4 * (j & 2))) & 0xFFu);
            const float hi = __builtin_amdgcn_cvt_off_f32_i4((v >> (16 + 4 * (j & 2))) & 0xFFu);
            b[j] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        }
        return b;
    }
};
struct Fp16 {
    static constexpr uint32_t kMinusOne = 0xBC00BC00u;
    static constexpr bool kZeroInOperand = true;
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ float to_f32(uint32_t v) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
    }
    static __device__ __forceinline__ uint16_t from_f32(float v) {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
    // `off`: -(1 + z / 16) twice; the XOR sets 1.0 and flips the code's top bit back
    static __device__ __forceinline__ u32x4 operand(uint32_t c, uint32_t off) {
        u32x4 b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int sh = 6 - 4 * j;
            const uint32_t v = sh >= 0 ? c << (sh >= 0 ? sh : 0) : c >> (sh < 0 ? -sh : 0);
            const uint32_t p = (v & 0x03C003C0u) ^ 0x3E003E00u;
            b[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p) + __builtin_bit_cast(f16x2, off));
        }
        return b;
    }
};

// bf16 operands against a weight whose scales are of type T.
template <class T>
struct DownT : Bf16 {
    static __device__ __forceinline__ float to_f32(uint32_t v) { return T::to_f32(v); }
};

// Layout of a packed weight (byte offsets); `gpu` is 128 / g, the groups of
// a unit.
struct W4gLayout {
    int tiles, units, gpu;
    size_t scales, zeros, total;
};
__host__ __device__ constexpr int w4g_zero_bytes(int gpu) { return gpu == 4 ? 2 : 1; }
__host__ __device__ inline W4gLayout w4g_layout(int group, bool zeros, int N, int K) {
    W4gLayout l;
    l.tiles = (N + 15) / 16;
    l.units = (K + 127) / 128;
    l.gpu = 128 / group;
    const size_t tu = (size_t)l.tiles * l.units;
    l.scales = tu * 1024;
    l.zeros = l.scales + tu * 32 * l.gpu;
    // whole 256-byte blocks, so that stacked weights stay aligned
    l.total = (l.zeros + (zeros ? tu * 16 * w4g_zero_bytes(l.gpu) : 0) + 255) / 256 * 256;
    return l;
}

// A unit's weights of one lane: 4 operand dwords, its row's scales and zero
// points.  Where those are narrower than a dword, the whole dword is loaded
// and the row's part taken at use: the compiler widens a narrower load's
// result next to the load, which would make loads ahead wait there.
template <int GPU>
struct W4gUnit {
    u32x4 codes;
    uint32_t scale[(GPU + 1) / 2];   // 16-bit scales, low half first (one: two rows')
    uint32_t zero;                   // nibbles (4 rows', one group to 2; two rows', 4 groups)
};

template <int GPU, bool ZP>
__device__ __forceinline__ W4gUnit<GPU> w4g_load(const uint8_t* w, const W4gLayout& l, size_t tile_unit, int lane) {
    W4gUnit<GPU> r;
    r.codes = *reinterpret_cast<const u32x4*>(w + tile_unit * 1024 + lane * 16);
    const uint8_t* s = w + l.scales + tile_unit * (32 * GPU);
    if constexpr (GPU == 1) {
        r.scale[0] = *reinterpret_cast<const uint32_t*>(s + (lane & 14) * 2);
    } else if constexpr (GPU == 2) {
        r.scale[0] = *reinterpret_cast<const uint32_t*>(s + (lane & 15) * 4);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(s + (lane & 15) * 8);
        r.scale[0] = v.x;
        r.scale[1] = v.y;
    }
    r.zero = 0;
    if constexpr (ZP) {
        constexpr int b = w4g_zero_bytes(GPU);
        r.zero = *reinterpret_cast<const uint32_t*>(w + l.zeros + tile_unit * (16 * b) + ((lane & 15) * b & ~3));
    }
    return r;
}
// The scale and the zero point of group g.
template <class T, int GPU>
__device__ __forceinline__ float w4g_scale(const W4gUnit<GPU>& w, int g, int lane) {
    const uint32_t v = GPU == 1 ? w.scale[0] >> (16 * (lane & 1)) : w.scale[g / 2] >> (16 * (g % 2));
    return T::to_f32(v & 0xFFFFu);
}
template <int GPU>
__device__ __forceinline__ uint32_t w4g_zero(const W4gUnit<GPU>& w, int g, int lane) {
    const int row = GPU == 4 ? 16 * (lane & 1) : 8 * (lane & 3);
    return (w.zero >> (row + 4 * g)) & 15u;
}

// acc[mt][nt] += x W^T / 16 over group g of a unit.  a[mt][s]: x rows
// 16 mt + lane % 16 at k = 32 (g SPG + s) + 8 (lane / 16) + 0..7 of the unit
// (zero where there is no such k; rows do not mix, so what a row that does
// not exist holds is no matter); acc in the MFMA's C layout: column
// n = lane % 16, rows m = 4 (lane / 16) + i.  The group's sum is held in
// float32 and scaled there.  P: x is the sum of P values in T, part p of step
// s in a[mt][p SPG + s]; their products meet in one sum.
template <class T, int GPU, bool ZP, int MT, int NT, int P = 1>
__device__ __forceinline__ void w4g_mac(int g, const W4gUnit<GPU> (&w)[NT], const u32x4 (&a)[MT][P * (4 / GPU)],
                                        f32x4 (&acc)[MT][NT]) {
    constexpr int SPG = 4 / GPU;   // MFMA steps per group
    const int lane = threadIdx.x & 63;
    u32x4 b[NT][SPG];
    float scale[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) scale[nt] = w4g_scale<T, GPU>(w[nt], g, lane);
    if constexpr (ZP && !T::kZeroInOperand) {
        // -sum x of the group comes from one more MFMA, against -1, in the lanes that need it; the
        // operands are made first, so that one row tile's sums are alive at a time
        const u32x4 minus = {T::kMinusOne, T::kMinusOne, T::kMinusOne, T::kMinusOne};
        float z[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int s = 0; s < SPG; ++s) b[nt][s] = T::operand(w[nt].codes[g * SPG + s], 0);
            z[nt] = 0.0625f * (float)((int)w4g_zero<GPU>(w[nt], g, lane) - 8);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            f32x4 xs = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < P * SPG; ++s) xs = T::mfma(a[mt][s], minus, xs);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                f32x4 t = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < P * SPG; ++s) t = T::mfma(a[mt][s], b[nt][s % SPG], t);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[mt][nt][i] = __builtin_fmaf(scale[nt], __builtin_fmaf(xs[i], z[nt], t[i]), acc[mt][nt][i]);
            }
        }
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint32_t z = ZP ? w4g_zero<GPU>(w[nt], g, lane) : 8u;
            f32x4 t[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) t[mt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < SPG; ++s) {
                b[nt][s] = T::operand(w[nt].codes[g * SPG + s], 0xBC00BC00u + z * 0x00400040u);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int p = 0; p < P; ++p) t[mt] = T::mfma(a[mt][p * SPG + s], b[nt][s], t[mt]);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = __builtin_fmaf(scale[nt], t[mt][i], acc[mt][nt][i]);
        }
    }
}

// This wave's number in its block, in a scalar register: what follows from it
// (loop bounds, addresses) is then known to be the same in all lanes.
__device__ __forceinline__ int wave_of_block() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Sums over the lanes up to each, by DPP (row_shr 1, 2, 4, 8, row_bcast 15, 31).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false); }
template <class F>
__device__ __forceinline__ int wave_scan(int v, F add) {
    v = add(v, dpp_or_zero<0x111, 0xF>(v));
    v = add(v, dpp_or_zero<0x112, 0xF>(v));
    v = add(v, dpp_or_zero<0x114, 0xF>(v));
    v = add(v, dpp_or_zero<0x118, 0xF>(v));
    v = add(v, dpp_or_zero<0x142, 0xA>(v));
    return add(v, dpp_or_zero<0x143, 0xC>(v));
}
__device__ __forceinline__ int add_ints(int a, int b) { return a + b; }
__device__ __forceinline__ int add_floats(int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }

// 8 values of T.
template <class T>
__device__ __forceinline__ void w4g_values(const uint16_t* p, float (&v)[8]) {
    const u32x4 raw = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = T::to_f32(raw[i] & 0xFFFFu);
        v[2 * i + 1] = T::to_f32(raw[i] >> 16);
    }
}

// sum_k x[k] W[n,k] by the definition, in float64; x8(k, v) gives x[k..k + 7].
// For the sums that w4g_mac leaves infinite or NaN, and only for those: a
// group's own sum, taken before its scale, can overflow where the result does
// not; an infinity times (q - 8) / 16 and times (8 - z) / 16 can cancel; and
// the chunks past K meet the row's last values with a scale of 0.  Ends at the
// first NaN.  1220 rows of K = 9728 against N = 2560, ms a call: 0.08 where all
// are finite, 0.09 where all hold NaN, 0.45 with an infinity in one row, 12.5
// with one in each.
template <class T, int GPU, bool ZP, class X>
__device__ __forceinline__ double w4g_defined(const uint8_t* w, const W4gLayout& l, int n, int K, X x8) {
    const int row = n & 15;
    double sum = 0.0;
    for (int k = 0; k < K && sum == sum; k += 8) {
        const size_t tu = (size_t)(n >> 4) * l.units + (k >> 7);
        const int g = (k & 127) / (128 / GPU);
        const uint32_t c =
            *reinterpret_cast<const uint32_t*>(w + tu * 1024 + (row + 2 * (k & 24)) * 16 + ((k >> 5) & 3) * 4) ^ 0x88888888u;
        const double s = T::to_f32(*reinterpret_cast<const uint16_t*>(w + l.scales + ((tu * 16 + row) * GPU + g) * 2));
        int z = 8;
        if constexpr (ZP) z = (w[l.zeros + (tu * 16 + row) * w4g_zero_bytes(GPU) + (g >> 1)] >> (4 * (g & 1))) & 15;
        float v[8];
        x8(k, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum = fma((double)v[2 * j], s * ((int)(c >> (4 * j) & 15u) - z), sum);
            sum = fma((double)v[2 * j + 1], s * ((int)(c >> (16 + 4 * j) & 15u) - z), sum);
        }
    }
    return sum;
}
__device__ __forceinline__ bool w4g_finite(float v) { return fabsf(v) < __builtin_inff(); }
// The same with x a row of T.
template <class T, int GPU, bool ZP>
__device__ __forceinline__ float w4g_defined_row(const uint16_t* x, int K, const uint8_t* w, const W4gLayout& l, int n) {
    return (float)w4g_defined<T, GPU, ZP>(w, l, n, K, [&](int k, float (&v)[8]) { w4g_values<T>(x + k, v); });
}

// Rows of x behind a buffer descriptor.  One tile's rows, or one pass's: the
// offsets stay in 32 bits whatever the matrix.
__device__ __forceinline__ v4i w4g_rows(const uint16_t* x, int rows, int K) {
    const uint64_t a = (uint64_t)(uintptr_t)x;
    v4i r;
    r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
    r.z = __builtin_amdgcn_readfirstlane(rows * K * 2);
    r.w = 0x00020000;
    return r;
}
// Lane i's 16 bytes at byte offset `off` of the rows go to LDS address
// lds + 16 i (wave-uniform); the caller waits (w4g_wait) before they are
// read.  Every offset has to lie inside the rows.
__device__ __forceinline__ void w4g_x_to_lds(v4i x, uint32_t off, uint32_t lds) {
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(off), "s"(x), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
// Every load of this wave has arrived / has been read from LDS.  The builtin,
// not assembly: the compiler then knows that the loads it counts itself are
// there.  Otherwise it waits for them at their first use, by a count that
// leaves out the loads to LDS issued meanwhile, so that it would wait for the
// next unit's as well.
__device__ __forceinline__ void w4g_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void w4g_wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// After it every wave of the block has read what it asked LDS for: loads that
// go there may follow.
__device__ __forceinline__ void w4g_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Operand rows through LDS: rows of 256 bytes (the 128 k of a unit), 16-byte
// chunk c of row r at slot c ^ (r % 16), so that the 16 rows of an operand
// read hit 16 different slots.  w4g_chunk: the byte, from the row's start,
// that lane i of an instruction filling rows r0..r0 + 3 brings for unit u; a
// chunk past K (its weights' scales are 0) brings the row's last one.
__device__ __forceinline__ uint32_t w4g_chunk(int r0, int u, int K, int lane) {
    const uint32_t row = (uint32_t)(r0 + (lane >> 4));
    const uint32_t b = u * 256u + (((uint32_t)lane & 15u) ^ (row & 15u)) * 16u;
    return b < 2u * K ? b : 2u * K - 16u;
}
// Step d's operand of this lane's row r of those at `rows`; of the first 16.
__device__ __forceinline__ u32x4 w4g_operand_row(const char* rows, int r, int d, int lane) {
    return *reinterpret_cast<const u32x4*>(rows + r * 256 + (((d * 4 + (lane >> 4)) ^ (r & 15)) * 16));
}
__device__ __forceinline__ u32x4 w4g_operand_rows(const char* rows, int d, int lane) {
    return w4g_operand_row(rows, lane & 15, d, lane);
}

}  // namespace cr
