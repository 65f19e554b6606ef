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
//           k + 2 j in bits 4 j and k + 2 j + 1 in bits 16 + 4 j: the order in
//           which one shift and one AND-OR make an operand register of two
//           codes, and 4 dwords are the B operands of 4 MFMA 16x16x32.
//   scales  16-bit, [t][u][row % 16][128 / g]
//   zeros   (weights with zero points) [t][u][row % 16][max(1, 64 / g)]
//           bytes, group i of the unit in bits 4 (i % 2) of byte i / 2
// Rows past N and k past K hold code 0 and scale 0.
#pragma once
#include "cr_device.h"

namespace cr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// The 16-bit types.  An operand register of two codes is (1 + q / 16) twice:
// the code in the top mantissa bits of 1.0, so making it takes no
// conversion, and 16 sum x (1 + q/16) - (16 + z) sum x = sum x (q - z).
// 1 + q/16 is exact in both types; the offset costs the float32 sums ~2 bits
// against sums of x (q - z), of which a 16-bit result keeps 8 or 11.
struct Bf16 {
    static constexpr uint32_t kMask = 0x00780078u, kOne = 0x3F803F80u;
    static constexpr int kShift = 3;
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ float to_f32(uint32_t v) { return __uint_as_float(v << 16); }
    static __device__ __forceinline__ uint16_t from_f32(float v) { return (uint16_t)f32_to_bf16_rne(v); }
};
struct Fp16 {
    static constexpr uint32_t kMask = 0x03C003C0u, kOne = 0x3C003C00u;
    static constexpr int kShift = 6;
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
};

// Layout of a packed weight (byte offsets); `gpu` is 128 / g, the groups of
// a unit.
struct W4gLayout {
    int tiles, units, gpu;
    size_t scales, zeros, total;
};
__host__ __device__ inline int w4g_zero_bytes(int gpu) { return gpu == 4 ? 2 : 1; }
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
// points.
template <int GPU>
struct W4gUnit {
    u32x4 codes;
    uint32_t scale[(GPU + 1) / 2];   // 16-bit scales, low half first
    uint32_t zero;                   // nibbles
};

template <int GPU, bool ZP>
__device__ __forceinline__ W4gUnit<GPU> w4g_load(const uint8_t* w, const W4gLayout& l, size_t tile_unit, int lane) {
    W4gUnit<GPU> r;
    r.codes = *reinterpret_cast<const u32x4*>(w + tile_unit * 1024 + lane * 16);
    const uint8_t* s = w + l.scales + tile_unit * (32 * GPU) + (lane & 15) * (2 * GPU);
    if constexpr (GPU == 1) {
        r.scale[0] = *reinterpret_cast<const uint16_t*>(s);
    } else if constexpr (GPU == 2) {
        r.scale[0] = *reinterpret_cast<const uint32_t*>(s);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(s);
        r.scale[0] = v.x;
        r.scale[1] = v.y;
    }
    r.zero = 0;
    if constexpr (ZP) {
        const uint8_t* z = w + l.zeros + tile_unit * (16 * w4g_zero_bytes(GPU)) + (lane & 15) * w4g_zero_bytes(GPU);
        if constexpr (GPU == 4) r.zero = *reinterpret_cast<const uint16_t*>(z);
        else r.zero = *z;
    }
    return r;
}

// Eight codes -> the MFMA operand (1 + q / 16) x 8.
template <class T>
__device__ __forceinline__ u32x4 w4g_operand(uint32_t c) {
    u32x4 b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int sh = T::kShift - 4 * j;
        const uint32_t v = sh >= 0 ? c << (sh >= 0 ? sh : 0) : c >> (sh < 0 ? -sh : 0);
        b[j] = (v & T::kMask) | T::kOne;
    }
    return b;
}

// acc[mt][nt] += x W^T over one unit.  a[mt][d]: x rows 16 mt + lane % 16 at
// k = 32 d + 8 (lane / 16) + 0..7 of the unit (zero where there is no such
// row or k); acc in the MFMA's C layout: column n = lane % 16, rows
// m = 4 (lane / 16) + i.  Every group's sum is held in float32 and scaled
// there; sum x comes from one more MFMA against ones, which leaves it in the
// lanes that need it and is shared by the NT weight tiles.
template <class T, int GPU, bool ZP, int MT, int NT>
__device__ __forceinline__ void w4g_mac(const W4gUnit<GPU> (&w)[NT], const u32x4 (&a)[MT][4], f32x4 (&acc)[MT][NT]) {
    constexpr int SPG = 4 / GPU;   // MFMA steps per group
    const u32x4 ones = {T::kOne, T::kOne, T::kOne, T::kOne};
#pragma unroll
    for (int g = 0; g < GPU; ++g) {
        f32x4 xs[MT], t[MT][NT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            xs[mt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) t[mt][nt] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < SPG; ++s) {
            const int d = g * SPG + s;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) xs[mt] = T::mfma(a[mt][d], ones, xs[mt]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const u32x4 b = w4g_operand<T>(w[nt].codes[d]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) t[mt][nt] = T::mfma(a[mt][d], b, t[mt][nt]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float s = T::to_f32((w[nt].scale[g / 2] >> (16 * (g % 2))) & 0xFFFFu);
            const float z = ZP ? (float)((w[nt].zero >> (4 * g)) & 15u) : 8.0f;
            const float s16 = 16.0f * s, sz = -s * (16.0f + z);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[mt][nt][i] = __builtin_fmaf(s16, t[mt][nt][i], __builtin_fmaf(sz, xs[mt][i], acc[mt][nt][i]));
        }
    }
}

// 8 values of x row `row` (nullptr: none) at k, zero past K.
__device__ __forceinline__ u32x4 w4g_x(const uint16_t* row, int k, int K) {
    if (row == nullptr || k >= K) return u32x4{0, 0, 0, 0};
    return *reinterpret_cast<const u32x4*>(row + k);
}

}  // namespace cr
