// A paged cache of keys and values held in 4 bits (layout in cr_kv4.h): the
// writer, and attention over it.
//
//   x' = H x / sqrt D (rotate: H the Sylvester Hadamard matrix of the head, by
//   float32 butterflies of strides 1, 2, .. D / 2, a, b -> a + b, a - b, then
//   times float32(1 / sqrt D)) or x; for each group of g along the head
//   lo = min(0, min x'), hi = max(0, max x'), s = hi / 15 - lo / 15 to the
//   nearest float32 whose low four bits are 0, z = clamp(rint(-lo / s), 0, 15),
//   c = clamp(rint(x' / s) + z, 0, 15); both 0 where s = 0.
#include "cr_w4g.h"
#include "cr_kv4.h"

namespace cr {
namespace {

template <int D>
constexpr float kv4_norm() { return D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f; }

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
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float p = __shfl_xor(x[i], m);
            x[i] = (lane & m) ? p - x[i] : x[i] + p;
        }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= kv4_norm<D>();
}

struct AppendArgs {
    Kv4 c;
    const uint16_t* x[2];        // K, V
    int64_t row[2], head[2];     // their strides in values
};

// One wave a token, head and K or V.
template <class T, int D>
__global__ void k_kv4_append(AppendArgs a) {
    constexpr int N = D / 64;
    __shared__ uint8_t code[D];
    const int t = blockIdx.x, h = blockIdx.y, which = blockIdx.z, lane = threadIdx.x, d = lane * N;
    int b = 0;
    Kv4Seq s = {};
    for (; b < a.c.B; ++b) {
        s = kv4_seq(a.c, b);
        if (t >= s.first && t < s.first + s.rows) break;
    }
    if (b == a.c.B) return;
    const int pos = s.tokens - s.rows + (t - s.first);
    if (pos < 0) return;
    const int page = kv4_page(a.c, b, pos);
    if (page < 0) return;
    const uint16_t* p = a.x[which] + t * a.row[which] + h * a.head[which];
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = T::to_f32(p[d + i]);
    if (a.c.rotate) rotate_head<D>(x);
    float lo = 0.0f, hi = 0.0f;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad |= !w4g_finite(x[i]);
    }
    for (int m = 1; m < a.c.group / N; m <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, m));
        hi = fmaxf(hi, __shfl_xor(hi, m));
        bad |= __shfl_xor(bad, m);
    }
    const uint32_t sb = bad ? kKv4Nan : (__float_as_uint(hi / 15.0f - lo / 15.0f) + 8) & ~15u;
    const float sc = __uint_as_float(sb);
    const float z = sc > 0.0f ? fminf(fmaxf(rintf(-lo / sc), 0.0f), 15.0f) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        code[d + i] = sc > 0.0f ? (uint8_t)fminf(fmaxf(rintf(x[i] / sc) + z, 0.0f), 15.0f) : 0;
    __syncthreads();
    const int row = pos & ((1 << a.c.page_log2) - 1);
    uint8_t* out = a.c.codes + kv4_codes_at(a.c, page, which, h);
    for (int k = lane; k < D / 2; k += 64) {
        if (which == 0) {
            const int dw = k >> 2, at = 32 * (dw % (D / 32)) + 8 * (dw / (D / 32)), half = (k >> 1) & 1, j = 2 * (k & 1);
            out[kv4_k_byte(D, row, 0) + k] = code[at + 2 * j + half] | code[at + 2 * j + 2 + half] << 4;
        } else {
            const int at = 32 * (k >> 4) + (k & 15);
            out[kv4_v_byte(D, row, k)] = code[at] | code[at + 16] << 4;
        }
    }
    if (d % a.c.group == 0)
        a.c.scales[kv4_scales_at(a.c, page, which, h) + row * (D / a.c.group) + d / a.c.group] = sb | (uint32_t)z;
}

// x'[d], a value of the cache.
template <int D>
__device__ __forceinline__ double kv4_value(const Kv4& c, int page, int which, int h, int row, int d) {
    const uint8_t* codes = c.codes + kv4_codes_at(c, page, which, h);
    const uint32_t w = c.scales[kv4_scales_at(c, page, which, h) + row * (D / c.group) + d / c.group];
    int q;
    if (which == 0) {
        const uint32_t dw = *reinterpret_cast<const uint32_t*>(
            codes + kv4_k_byte(D, row, (d / 8 % 4) * (D / 32) + d / 32));
        q = dw >> (4 * (d % 8 / 2) + 16 * (d % 2)) & 15;
    } else {
        q = codes[kv4_v_byte(D, row, 16 * (d / 32) + d % 16)] >> (d % 32 >= 16 ? 4 : 0) & 15;
    }
    return (double)__uint_as_float(w & ~15u) * (q - (int)(w & 15u));
}

// One wave a row and head.
template <class T, int D>
__global__ void k_attn_kv4(Kv4 c, AttnArgs a) {
    constexpr int N = D / 64;
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, d = lane * N, g = h / (a.Hq / c.heads);
    int b = 0;
    Kv4Seq s = {};
    for (; b < c.B; ++b) {
        s = kv4_seq(c, b);
        if (t >= s.first && t < s.first + s.rows) break;
    }
    if (b == c.B) return;
    const int pos = s.tokens - s.rows + (t - s.first);
    float q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = T::to_f32(a.q[t * a.q_row + h * a.q_head + d + i]);
    if (c.rotate) rotate_head<D>(q);
    double top = -__builtin_inf(), sum = 0.0, acc[N] = {};
    for (int pass = 0; pass < 2; ++pass)
        for (int j = 0; j <= pos; ++j) {
            const int page = kv4_page(c, b, j), row = j & ((1 << c.page_log2) - 1);
            if (page < 0) continue;
            double v = 0.0;
#pragma unroll
            for (int i = 0; i < N; ++i) v = fma((double)q[i], kv4_value<D>(c, page, 0, g, row, d + i), v);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
            v *= a.scale;
            if (pass == 0) {
                top = v > top || v != v ? v : top;
                if (top != top) break;
            } else {
                const double p = exp(v - top);
                sum += p;
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = fma(p, kv4_value<D>(c, page, 1, g, row, d + i), acc[i]);
            }
        }
    float o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = sum > 0.0 || sum != sum ? (float)(acc[i] / sum) : 0.0f;
    if (c.rotate) rotate_head<D>(o);
#pragma unroll
    for (int i = 0; i < N; ++i) a.y[((int64_t)t * a.Hq + h) * D + d + i] = T::from_f32(o[i]);
}

template <class F>
void by_dim(int D, F f) {
    if (D == 64) f(std::integral_constant<int, 64>());
    if (D == 128) f(std::integral_constant<int, 128>());
    if (D == 256) f(std::integral_constant<int, 256>());
}

}  // namespace

hipError_t launch_kv4_append(bool fp16, const uint16_t* k, int64_t k_row, int64_t k_head, const uint16_t* v,
                             int64_t v_row, int64_t v_head, const Kv4& c, hipStream_t st) {
    const AppendArgs a{c, {k, v}, {k_row, v_row}, {k_head, v_head}};
    const dim3 grid(c.T, c.heads, 2);
    by_dim(c.dim, [&](auto d) {
        if (fp16) k_kv4_append<Fp16, d><<<grid, 64, 0, st>>>(a);
        else k_kv4_append<Bf16, d><<<grid, 64, 0, st>>>(a);
    });
    return hipGetLastError();
}

size_t attn_kv4_workspace(int, int, int, int, int, int, int) { return 0; }

hipError_t launch_attn_kv4(const AttnArgs& a, const Kv4& c, void*, hipStream_t st) {
    const dim3 grid(c.T, a.Hq);
    by_dim(c.dim, [&](auto d) {
        if (a.fp16) k_attn_kv4<Fp16, d><<<grid, 64, 0, st>>>(c, a);
        else k_attn_kv4<Bf16, d><<<grid, 64, 0, st>>>(c, a);
    });
    return hipGetLastError();
}

}  // namespace cr
