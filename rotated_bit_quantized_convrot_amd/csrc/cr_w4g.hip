// 4-bit weights with group scales: encoder, packing and the linear.
#include "cr_w4g.h"

namespace cr {
namespace {

// ---------------------------------------------------------------------------
// Encoder.  Groups never cross a row (g divides K), so the weight is one
// flat run of groups; g / 8 neighbouring lanes hold a group, 8 values each.
// Bound by HBM: 2 B in, 0.5 B of codes and 2/g (3/g) B of scales out per value,
// once the divisions are cheap: an IEEE division for each value took 66 us
// for 100 M values in groups of 32 with zero points, this 51 to 57 (261 MB:
// 4.6 to 5.1 TB/s).
//
// rint(fl(v / s)) without the division: r = v fl(1/s) is within 2 steps of
// v / s, and r + (v - r s) fl(1/s), the residue exact in an fma, is v / s
// wherever that is a float32 (so ties stay ties) and within a step of it
// otherwise.  That cannot pass a tie: v and s have at most 11 bits and a tie
// k + 1/2 at most 5, so v and s (k + 1/2), where they differ, do so by more
// than 2^-18 of themselves.  Scales whose reciprocal leaves float32's normal
// range take the division.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float r = v * inv;
    return __builtin_fmaf(__builtin_fmaf(-r, s, v), inv, r);
}

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
    lo = fminf(lo, lane_xor<1>(lo));
    hi = fmaxf(hi, lane_xor<1>(hi));
    lo = fminf(lo, lane_xor<2>(lo));
    hi = fmaxf(hi, lane_xor<2>(hi));
    if constexpr (G >= 64) {
        lo = fminf(lo, lane_xor<4>(lo));
        hi = fmaxf(hi, lane_xor<4>(hi));
    }
    if constexpr (G >= 128) {
        lo = fminf(lo, lane_xor<8>(lo));
        hi = fmaxf(hi, lane_xor<8>(hi));
    }
    float step = fmaxf(hi, -lo) / 7.0f;
    if constexpr (ZP) {
        // bf16 values can lie further apart than float32 reaches: then in halves
        const bool far = hi - lo == __builtin_inff();
        step = (far ? 0.5f * hi - 0.5f * lo : hi - lo) / 15.0f;
        step = far ? 2.0f * step : step;
    }
    const uint16_t s16 = T::from_f32(step);
    const float s = T::to_f32(s16);
    float z = 0.0f, q[8];
    if (s > 0x1p-100f && s < 0x1p100f) {
        const float inv = 1.0f / s;
        if constexpr (ZP) z = fminf(fmaxf(rintf(quotient(-lo, s, inv)), 0.0f), 15.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = rintf(quotient(v[i], s, inv));
    } else if (s > 0.0f) {
        if constexpr (ZP) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = rintf(v[i] / s);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = 0.0f;
    }
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (ZP) q[i] = fminf(fmaxf(q[i] + z, 0.0f), 15.0f);
        else q[i] = fminf(fmaxf(q[i], -8.0f), 7.0f) + 8.0f;
        out |= (uint32_t)q[i] << (4 * i);
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
            v[d] = (((e | (e >> 8)) & 0xFFFFu) | ((o | (o >> 8)) << 16)) ^ 0x88888888u;
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
// Linear.  Block tile BM = 16 MT WM rows of x by BN = 16 NT WN weight rows,
// by WM x WN waves for each of KG groups of waves that take the units of K
// in turn; the groups' sums meet in LDS and are added in their order (no
// atomics: results do not change between runs).  A group's x tile (BM rows
// x 128 k) goes straight to LDS, one unit ahead; weights go straight to
// registers, one unit ahead, and are made operands there.  A group of one
// wave needs no barrier: it waits for its own loads.
// LDS rows of 256 bytes, 16-byte chunk c of row r at slot c ^ (r % 16): the
// 16 rows of an operand read hit 16 different slots.
// ---------------------------------------------------------------------------
template <int MT, int NT, int WM, int WN, int KG>
struct Tile {
    static constexpr int kThreads = 64 * WM * WN * KG;
    static constexpr int kBM = 16 * MT * WM, kBN = 16 * NT * WN;
    static constexpr int kTile = kBM * 256, kStage = KG * kTile;
    static constexpr int kSums = KG * kBM * kBN * 4;
    static constexpr int kLds = 2 * kStage > kSums ? 2 * kStage : kSums;
    static_assert(kLds <= 160 * 1024 && kThreads <= 1024, "a block fits a CU");
    static_assert(kBM / 4 % (WM * WN) == 0, "the group's waves share the staging evenly");
};

template <class T, int GPU, bool ZP, int MT, int NT, int WM, int WN, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG) void k_w4g_linear(const uint16_t* __restrict__ x, int M, int K,
                                                                  const uint8_t* __restrict__ w, int N,
                                                                  const uint16_t* __restrict__ bias,
                                                                  uint16_t* __restrict__ y) {
    using C = Tile<MT, NT, WM, WN, KG>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const uint32_t lds0 = lds_address(lds);
    const W4gLayout l = w4g_layout(128 / GPU, ZP, N, K);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / (WM * WN), r = wave % (WM * WN), wm = r % WM, wn = r / WM;
    const int m0 = blockIdx.y * C::kBM, rows = M - m0 < C::kBM ? M - m0 : C::kBM;
    const int tile0 = blockIdx.x * (NT * WN) + wn * NT;
    const v4i xb = w4g_rows(x + (size_t)m0 * K, rows, K);

    // x of unit u into stage s: 4 rows an instruction.  Rows and k that do
    // not exist read ones that do: their results are not stored, their
    // weights' scales are 0.
    auto stage = [&](int u, int s) {
        u = u < l.units ? u : l.units - 1;
#pragma unroll
        for (int i = 0; i < C::kBM / 4 / (WM * WN); ++i) {
            const int row4 = (i * (WM * WN) + r) * 4, row = row4 + (lane >> 4);
            const uint32_t rb = (uint32_t)(row < rows ? row : rows - 1) * (2u * K);
            w4g_x_to_lds(xb, rb + w4g_chunk(row4, u, K, lane), lds0 + s * C::kStage + kg * C::kTile + row4 * 256);
        }
    };
    auto weights = [&](int u, W4gUnit<GPU> (&wu)[NT]) {
        u = u < l.units ? u : l.units - 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int t = tile0 + nt < l.tiles ? tile0 + nt : l.tiles - 1;
            wu[nt] = w4g_load<GPU, ZP>(w, l, (size_t)t * l.units + u, lane);
        }
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0, 0, 0, 0};
    const int iters = (l.units + KG - 1) / KG;
    W4gUnit<GPU> wu[NT];
    weights(kg, wu);
    stage(kg, 0);
    for (int it = 0; it < iters; ++it) {
        const int u = it * KG + kg;
        w4g_wait();
        // this unit's x is there, and the other stage has been read by all
        if constexpr (WM * WN > 1) w4g_barrier();
        else w4g_wait_lds();
        W4gUnit<GPU> next[NT];
        if (it + 1 < iters) {
            weights(u + KG, next);
            stage(u + KG, (it + 1) & 1);
        }
        const char* xt = lds + (it & 1) * C::kStage + kg * C::kTile + wm * MT * 4096;
        if (u < l.units) {
#pragma unroll
            for (int g = 0; g < GPU; ++g) {
                u32x4 a[MT][4 / GPU];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int s = 0; s < 4 / GPU; ++s)
                        a[mt][s] = w4g_operand_rows(xt + mt * 4096, g * (4 / GPU) + s, lane);
                w4g_mac<T, GPU, ZP, MT, NT>(g, wu, a, acc);
            }
        }
        if (it + 1 < iters) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) wu[nt] = next[nt];
        }
    }
    __syncthreads();
    f32x4* part = reinterpret_cast<f32x4*>(lds);   // [KG][WN NT][WM MT][64]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            part[((kg * (WN * NT) + wn * NT + nt) * (WM * MT) + wm * MT + mt) * 64 + lane] = acc[mt][nt];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * C::kBN; i += C::kThreads) {
        const int m = i / C::kBN, n = i % C::kBN;
        const size_t gn = (size_t)blockIdx.x * C::kBN + n;
        if (gn >= (size_t)N) continue;
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < KG; ++g)
            v += part[((g * (WN * NT) + (n >> 4)) * (WM * MT) + (m >> 4)) * 64 + ((m & 15) >> 2) * 16 + (n & 15)][m & 3];
        v *= 16.0f;
        if (!w4g_finite(v)) v = w4g_defined_row<T, GPU, ZP>(x + (size_t)(m0 + m) * K, K, w, l, (int)gn);
        if (bias != nullptr) v += T::to_f32(bias[gn]);
        y[(size_t)(m0 + m) * N + gn] = T::from_f32(v);
    }
}

struct LinearArgs {
    const uint16_t* x;
    int M, K;
    const uint8_t* w;
    int N;
    const uint16_t* bias;
    uint16_t* y;
};

template <class T, int GPU, bool ZP, int MT, int NT, int WM, int WN, int KG>
hipError_t tile(const LinearArgs& a, hipStream_t st) {
    using C = Tile<MT, NT, WM, WN, KG>;
    static std::atomic<uint64_t> done{0};
    const auto kernel = k_w4g_linear<T, GPU, ZP, MT, NT, WM, WN, KG>;
    const hipError_t e = opt_in_lds(reinterpret_cast<const void*>(kernel), C::kLds, done);
    if (e != hipSuccess) return e;
    kernel<<<dim3((a.N + C::kBN - 1) / C::kBN, (a.M + C::kBM - 1) / C::kBM), C::kThreads, C::kLds, st>>>(
        a.x, a.M, a.K, a.w, a.N, a.bias, a.y);
    return hipGetLastError();
}

// Tile choice.  Fewer, wider blocks read x less often and share its operand
// reads; narrow ones put more CUs to work.  Measured, us, bf16, groups of 128,
// K x N = 2560 x 9728 / 9728 x 2560 / 2560 x 2560 (weights cold):
//   M = 8     one tile, 4 K groups 6.4 / 11.3 / 4.2, 10 groups 6.7 / 7.6 / 3.9,
//             16 groups 9.0 / 7.0 / 4.1
//   M = 32    32 columns 9.4 / 16.2 / 6.0, 16 columns 11.8 / 10.1 / 4.6
//   M = 48    64 columns 9.9 / 22.5 / 8.6, with two tiles a wave and half the
//             waves 10.9 / 25.4 / 9.4, 16 columns 15.1 / 13.3 / 5.6
// Up to 48 rows the wide tile is taken where its blocks fill half the chip
// (256 CUs).  Above that the time is that of the rounds of 256 blocks (one
// fits a CU) times a block's, which go as 2 : 3 : 7 : 8 for 80 x 16, 80 x 64,
// 112 x 128 and 128 x 128 (M = 76 at 2560 x 9728: 21.0 / 12.1 for the first
// two); us, in that order, K x N x M:
//   2560 x 9728 x 100    33 / 20 / 24 / 25       2560 x 2560 x 200   15 / 12 / 23 / 25
//   2560 x 9728 x 300    66 / 32 / 27 / 28       4096 x 4096 x 300   39 / 18 / 33 / 36
//   9728 x 2560 x 1220  190 / 98 / 77 / 82       4096 x 4096 x 1000 121 / 61 / 68 / 41
//   2560 x 9728 x 1220  239 / 105 / 97 / 82
template <class T, int GPU, bool ZP>
hipError_t linear_t(const LinearArgs& a, hipStream_t st) {
    constexpr long kHalf = 128;
    const long tiles = (a.N + 15) / 16;
    const int units = (a.K + 127) / 128;
    if (a.M <= 16) {
        if (tiles > 2 * 256) return tile<T, GPU, ZP, 1, 1, 1, 1, 4>(a, st);
        if (units > 40) return tile<T, GPU, ZP, 1, 1, 1, 1, 16>(a, st);
        return tile<T, GPU, ZP, 1, 1, 1, 1, 10>(a, st);
    }
    if (a.M <= 32) {
        if ((tiles + 1) / 2 >= kHalf) return tile<T, GPU, ZP, 2, 1, 1, 2, 4>(a, st);
        return tile<T, GPU, ZP, 2, 1, 1, 1, 8>(a, st);
    }
    if (a.M <= 48) {
        if ((tiles + 3) / 4 >= kHalf) return tile<T, GPU, ZP, 3, 1, 1, 4, 4>(a, st);
        return tile<T, GPU, ZP, 3, 1, 1, 1, 6>(a, st);
    }
    // the least time: rounds of 256 blocks (one fits a CU) times a block's
    auto rounds = [&](long m, long n) { return ((a.M + m - 1) / m * ((a.N + n - 1) / n) + 255) / 256; };
    const long c16 = 2 * rounds(80, 16), c64 = 3 * rounds(80, 64), c7 = 7 * rounds(112, 128), c8 = 8 * rounds(128, 128);
    if (c8 < c7 && c8 < c64 && c8 < c16) return tile<T, GPU, ZP, 8, 2, 1, 4, 2>(a, st);
    if (c7 < c64 && c7 < c16) return tile<T, GPU, ZP, 7, 2, 1, 4, 2>(a, st);
    if (c64 < c16) return tile<T, GPU, ZP, 5, 1, 1, 4, 4>(a, st);
    return tile<T, GPU, ZP, 5, 1, 1, 1, 4>(a, st);
}

template <class T>
hipError_t linear_g(const LinearArgs& a, int group, bool zeros, hipStream_t st) {
    switch (group) {
        case 32: return zeros ? linear_t<T, 4, true>(a, st) : linear_t<T, 4, false>(a, st);
        case 64: return zeros ? linear_t<T, 2, true>(a, st) : linear_t<T, 2, false>(a, st);
        default: return zeros ? linear_t<T, 1, true>(a, st) : linear_t<T, 1, false>(a, st);
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
    const LinearArgs a = {x, M, K, w, N, bias, y};
    return fp16 ? linear_g<Fp16>(a, group, zeros, st) : linear_g<Bf16>(a, group, zeros, st);
}

}  // namespace cr
