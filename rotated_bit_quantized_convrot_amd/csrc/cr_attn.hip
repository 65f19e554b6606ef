// Attention over whole prompts: packed sequences, grouped heads, causal or
// both ways.
//
//   y[i, h] = T(sum_j p[i, j] v[j, h / G] / sum_j p[i, j]),
//   p[i, j] = exp(scale q[i, h] . k[j, h / G]),
// j over the tokens of i's sequence, up to i if causal.
#include "cr_w4g.h"

namespace cr {
namespace {

// One row by the definition, in float64, by one wave: lane l takes
// d = l D / 64 and on.  Two passes over the keys: the largest score, then the
// sums, so that infinities and NaN come out as they do in the definition.
template <class T, int D>
__device__ void attn_row_defined(const uint16_t* q, const uint16_t* k, int64_t k_row, const uint16_t* v, int64_t v_row,
                                 int keys, float scale, uint16_t* y) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63, d = lane * N;
    double top = -__builtin_inf(), sum = 0.0, o[N] = {};
    for (int pass = 0; pass < 2; ++pass) {
        for (int j = 0; j < keys; ++j) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < N; ++i) s = fma((double)T::to_f32(q[d + i]), (double)T::to_f32(k[j * k_row + d + i]), s);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
            s *= scale;
            if (pass == 0) {
                top = s > top || s != s ? s : top;
                if (top != top) break;
            } else {
                const double p = exp(s - top);
                sum += p;
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fma(p, (double)T::to_f32(v[j * v_row + d + i]), o[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) y[d + i] = keys > 0 ? T::from_f32((float)(o[i] / sum)) : 0;
}

// The sequence that row t is in, or -1.
__device__ int sequence_of(const int32_t* cu, int B, int T, int t) {
    for (int b = 0; b < B; ++b) {
        const int first = min(max(cu[b], 0), T), last = min(max(cu[b + 1], first), T);
        if (t >= first && t < last) return b;
    }
    return -1;
}

template <class T, int D>
__global__ void k_attn_prompt(AttnArgs a) {
    const int t = blockIdx.x, h = blockIdx.y;
    const int b = sequence_of(a.cu, a.B, a.T, t);
    if (b < 0) return;
    const int first = min(max(a.cu[b], 0), a.T), last = min(max(a.cu[b + 1], first), a.T);
    const int g = h / (a.Hq / a.Hkv);
    attn_row_defined<T, D>(a.q + t * a.q_row + h * a.q_head, a.k + first * a.k_row + g * a.k_head, a.k_row,
                           a.v + first * a.v_row + g * a.v_head, a.v_row, a.causal ? t - first + 1 : last - first,
                           a.scale, a.y + ((int64_t)t * a.Hq + h) * D);
}

template <class T>
void launch(const AttnArgs& a, hipStream_t st) {
    const dim3 grid(a.T, a.Hq);
    if (a.D == 64) k_attn_prompt<T, 64><<<grid, 64, 0, st>>>(a);
    if (a.D == 128) k_attn_prompt<T, 128><<<grid, 64, 0, st>>>(a);
    if (a.D == 256) k_attn_prompt<T, 256><<<grid, 64, 0, st>>>(a);
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t st) {
    if (a.fp16) launch<Fp16>(a, st);
    else launch<Bf16>(a, st);
    return hipGetLastError();
}

}  // namespace cr
