// 4-bit weights with group scales: encoder, packing and the linear.
#include "cr_w4g.h"

namespace cr {
namespace {

// ---------------------------------------------------------------------------
// Encoder.  Groups never cross a row (g divides K), so the weight is one
// flat run of groups; g / 8 neighbouring lanes hold a group, 8 values each.
// Bound by HBM: 2 B in, 0.5 B of codes and 2/g (3/g) B of scales out per value.
// ---------------------------------------------------------------------------
template <class T, int G, bool ZP>
__global__ __launch_bounds__(256) void k_w4g_encode(const uint16_t* __restrict__ w, size_t chunks,
                                                    uint32_t* __restrict__ codes, uint16_t* __restrict__ scales,
                                                    uint8_t* __restrict__ zeros) {
    const size_t c = (size_t)blockIdx.x * 256 + threadIdx.x;
    const bool in = c < chunks;   // whole groups are in or out: G / 8 divides the chunk count
    u32x4 raw = {0, 0, 0, 0};
    if (in) raw = *reinterpret_cast<const u32x4*>(w + c * 8);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = T::to_f32(raw[i] & 0xFFFFu);
        v[2 * i + 1] = T::to_f32(raw[i] >> 16);
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int m = 1; m < G / 8; m *= 2) {
        lo = fminf(lo, __shfl_xor(lo, m));
        hi = fmaxf(hi, __shfl_xor(hi, m));
    }
    const uint16_t s16 = T::from_f32(ZP ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    const float s = T::to_f32(s16);
    const float z = ZP && s > 0.0f ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 0.0f;
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q;
        if constexpr (ZP) q = s > 0.0f ? fminf(fmaxf(rintf(v[i] / s) + z, 0.0f), 15.0f) : 0.0f;
        else q = s > 0.0f ? fminf(fmaxf(rintf(v[i] / s), -8.0f), 7.0f) + 8.0f : 8.0f;
        out |= (uint32_t)q << (4 * i);
    }
    if (!in) return;
    codes[c] = out;
    if (c % (G / 8) == 0) {
        scales[c / (G / 8)] = s16;
        if constexpr (ZP) zeros[c / (G / 8)] = (uint8_t)z;
    }
}

// ---------------------------------------------------------------------------
// Packing (once per weight): one thread per 16 bytes of a code tile; the
// lanes of rows 0..15 also place the unit's scales and zero points.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_w4g_pack(const uint8_t* __restrict__ codes,
                                                  const uint16_t* __restrict__ scales,
                                                  const uint8_t* __restrict__ zeros, int N, int K, int group,
                                                  size_t threads, uint8_t* __restrict__ out) {
    const size_t t = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= threads) return;
    const W4gLayout l = w4g_layout(group, zeros != nullptr, N, K);
    const int lane = (int)(t & 63);
    const size_t tu_all = t >> 6, per = (size_t)l.tiles * l.units;
    const size_t which = tu_all / per, tu = tu_all % per;   // weight of the stack, tile and unit in it
    const int u = (int)(tu % l.units);
    const int n = (int)(tu / l.units) * 16 + (lane & 15);
    codes += which * (size_t)N * (K / 2);
    scales += which * (size_t)N * (K / group);
    if (zeros) zeros += which * (size_t)N * (K / group);
    out += which * l.total;
    u32x4 v = {0, 0, 0, 0};
    if (n < N) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int k = u * 128 + d * 32 + (lane >> 4) * 8;
            if (k >= K) continue;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (size_t)n * (K / 2) + k / 2);
            uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
            e = (e | (e >> 4)) & 0x00FF00FFu;
            o = (o | (o >> 4)) & 0x00FF00FFu;
            v[d] = ((e | (e >> 8)) & 0xFFFFu) | ((o | (o >> 8)) << 16);
        }
    }
    *reinterpret_cast<u32x4*>(out + tu * 1024 + lane * 16) = v;
    if (lane < 16) {
        uint32_t z = 0;
        for (int i = 0; i < l.gpu; ++i) {
            const int k = u * 128 + i * group;
            const bool in = n < N && k < K;
            const size_t at = (size_t)n * (K / group) + k / group;
            reinterpret_cast<uint16_t*>(out + l.scales)[(tu * 16 + lane) * l.gpu + i] = in ? scales[at] : (uint16_t)0;
            if (zeros && in) z |= (uint32_t)(zeros[at] & 15u) << (4 * i);
        }
        if (zeros) {
            uint8_t* p = out + l.zeros + (tu * 16 + lane) * w4g_zero_bytes(l.gpu);
            p[0] = (uint8_t)z;
            if (l.gpu == 4) p[1] = (uint8_t)(z >> 8);
        }
    }
}

// ---------------------------------------------------------------------------
// Linear.  A block owns 16 weight rows and 16 MT rows of x; its waves take
// the units of K in turn and their sums meet in LDS, added in the order of
// the waves (no atomics: results do not change between runs).
// ---------------------------------------------------------------------------
constexpr int kWaves = 4;

template <class T, int GPU, bool ZP, int MT>
__global__ __launch_bounds__(64 * kWaves) void k_w4g_linear(const uint16_t* __restrict__ x, int M, int K,
                                                            const uint8_t* __restrict__ w, int N,
                                                            const uint16_t* __restrict__ bias,
                                                            uint16_t* __restrict__ y) {
    __shared__ f32x4 part[kWaves][MT][64];
    const W4gLayout l = w4g_layout(128 / GPU, ZP, N, K);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t tile = blockIdx.x;
    const int m0 = blockIdx.y * (16 * MT);
    const uint16_t* rows[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = m0 + mt * 16 + (lane & 15);
        rows[mt] = m < M ? x + (size_t)m * K : nullptr;
    }
    f32x4 acc[MT][1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][0] = f32x4{0, 0, 0, 0};
    for (int u = wave; u < l.units; u += kWaves) {
        W4gUnit<GPU> wu[1] = {w4g_load<GPU, ZP>(w, l, tile * l.units + u, lane)};
        u32x4 a[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int d = 0; d < 4; ++d) a[mt][d] = w4g_x(rows[mt], u * 128 + d * 32 + (lane >> 4) * 8, K);
        w4g_mac<T, GPU, ZP, MT, 1>(wu, a, acc);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[wave][mt][lane] = acc[mt][0];
    __syncthreads();
    // thread -> (row m of the tile, column n): 16 neighbours write 32 bytes
    for (int i = threadIdx.x; i < 256 * MT; i += 64 * kWaves) {
        const int m = i >> 4, n = i & 15;
        const int gm = m0 + m;
        const size_t gn = tile * 16 + n;
        if (gm >= M || gn >= (size_t)N) continue;
        float v = 0.0f;
#pragma unroll
        for (int wv = 0; wv < kWaves; ++wv) v += part[wv][m >> 4][((m & 15) >> 2) * 16 + n][m & 3];
        if (bias != nullptr) v += T::to_f32(bias[gn]);
        y[(size_t)gm * N + gn] = T::from_f32(v);
    }
}

template <class T, int GPU, bool ZP>
hipError_t linear_t(const uint16_t* x, int M, int K, const uint8_t* w, int N, const uint16_t* bias, uint16_t* y,
                    hipStream_t st) {
    const dim3 block(64 * kWaves);
    const unsigned tiles = (unsigned)((N + 15) / 16);
    if (M <= 16)
        k_w4g_linear<T, GPU, ZP, 1><<<dim3(tiles, 1), block, 0, st>>>(x, M, K, w, N, bias, y);
    else
        k_w4g_linear<T, GPU, ZP, 4><<<dim3(tiles, (M + 63) / 64), block, 0, st>>>(x, M, K, w, N, bias, y);
    return hipGetLastError();
}

template <class T>
hipError_t linear_g(const uint16_t* x, int M, int K, const uint8_t* w, int group, bool zeros, int N,
                    const uint16_t* bias, uint16_t* y, hipStream_t st) {
    switch (group) {
        case 32: return zeros ? linear_t<T, 4, true>(x, M, K, w, N, bias, y, st) : linear_t<T, 4, false>(x, M, K, w, N, bias, y, st);
        case 64: return zeros ? linear_t<T, 2, true>(x, M, K, w, N, bias, y, st) : linear_t<T, 2, false>(x, M, K, w, N, bias, y, st);
        default: return zeros ? linear_t<T, 1, true>(x, M, K, w, N, bias, y, st) : linear_t<T, 1, false>(x, M, K, w, N, bias, y, st);
    }
}

template <class T, int G>
void encode_t(const uint16_t* w, size_t chunks, uint32_t* codes, uint16_t* scales, uint8_t* zeros, hipStream_t st) {
    const unsigned blocks = (unsigned)((chunks + 255) / 256);
    if (zeros) k_w4g_encode<T, G, true><<<blocks, 256, 0, st>>>(w, chunks, codes, scales, zeros);
    else k_w4g_encode<T, G, false><<<blocks, 256, 0, st>>>(w, chunks, codes, scales, zeros);
}

template <class T>
void encode_g(int group, const uint16_t* w, size_t chunks, uint32_t* codes, uint16_t* scales, uint8_t* zeros,
              hipStream_t st) {
    switch (group) {
        case 32: return encode_t<T, 32>(w, chunks, codes, scales, zeros, st);
        case 64: return encode_t<T, 64>(w, chunks, codes, scales, zeros, st);
        default: return encode_t<T, 128>(w, chunks, codes, scales, zeros, st);
    }
}

}  // namespace

size_t w4g_packed_bytes(int group, bool zeros, int N, int K) { return w4g_layout(group, zeros, N, K).total; }

hipError_t launch_w4g_encode(bool fp16, const uint16_t* w, int N, int K, int group, uint8_t* codes, uint16_t* scales,
                             uint8_t* zeros, hipStream_t st) {
    const size_t chunks = (size_t)N * K / 8;
    uint32_t* c = reinterpret_cast<uint32_t*>(codes);
    if (fp16) encode_g<Fp16>(group, w, chunks, c, scales, zeros, st);
    else encode_g<Bf16>(group, w, chunks, c, scales, zeros, st);
    return hipGetLastError();
}

hipError_t launch_w4g_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int count, int N,
                           int K, int group, uint8_t* out, hipStream_t st) {
    const W4gLayout l = w4g_layout(group, zeros != nullptr, N, K);
    const size_t threads = (size_t)count * l.tiles * l.units * 64;
    k_w4g_pack<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(codes, scales, zeros, N, K, group, threads, out);
    return hipGetLastError();
}

hipError_t launch_w4g_linear(bool fp16, const uint16_t* x, int M, int K, const uint8_t* w, int group, bool zeros,
                             int N, const uint16_t* bias, uint16_t* y, hipStream_t st) {
    if (fp16) return linear_g<Fp16>(x, M, K, w, group, zeros, N, bias, y, st);
    return linear_g<Bf16>(x, M, K, w, group, zeros, N, bias, y, st);
}

}  // namespace cr
