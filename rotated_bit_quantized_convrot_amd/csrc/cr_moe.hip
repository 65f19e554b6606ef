// Mixture-of-experts layer on 4-bit weights with group scales, for a few
// tokens: router logits, top-k and softmax, the chosen experts' gated MLPs
// and their weighted sum.
//
//   l[m,e] = sum_k x[m,k] r[e,k];  e_0..e_{k-1} the largest, ties to the lower e
//   p = exp(l - max l),  c[m,r] = p[e_r] / (sum over the chosen, or over all)
//   h[m,r] = T(c[m,r] silu(Wg_e x[m]) (Wu_e x[m]))        (T: the 16-bit type)
//   y[m]   = T(sum_r Wd_{e_r} h[m,r])
//
// A pass is bound by the chosen experts' weights, each read once: the gate /
// up kernel takes an expert's tokens together, and the down kernel gives
// every 16 output columns to one block, which walks all chosen experts and
// sums in a fixed order (no atomics on results).
#include "cr_w4g.h"

namespace cr {
namespace {

constexpr int kChunk = kMoeChunk;   // tokens per pass

// Workspace of one pass over `m` tokens (byte offsets, 256-byte regions).
struct MoeWs {
    size_t logits, ids, weights, lists, slot_pair, h, total;
};
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
MoeWs moe_ws(int M, int F, int E, int topk) {
    const size_t m = M < kChunk ? M : kChunk, pairs = m * topk;
    const size_t slots = pairs < (size_t)E ? pairs : (size_t)E;
    MoeWs l;
    l.logits = 0;
    l.ids = l.logits + up256(m * E * 8);
    l.weights = l.ids + up256(pairs * 4);
    l.lists = l.weights + up256(pairs * 4);
    l.slot_pair = l.lists + up256((1 + 2 * slots + 1 + pairs) * 4);
    l.h = l.slot_pair + up256(slots * kChunk * 2);
    l.total = l.h + up256(pairs * F * 2);
    return l;
}

// lists: [0] active experts A; [1 + s] expert of slot s; then offsets
// [slots + 1] into the pair list; then the pairs (m * topk + r) by slot.
struct MoeLists {
    int32_t* active;
    int32_t* expert;
    int32_t* offset;
    int32_t* pair;
};
__host__ __device__ inline MoeLists moe_lists(int32_t* base, int slots) {
    return {base, base + 1, base + 1 + slots, base + 2 + 2 * slots};
}

// ---------------------------------------------------------------------------
// Router logits in float64: which expert is chosen hangs on the order of
// values that can be close, and the sums then do not depend on their order.
// A wave per expert, tokens in turn.
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(256) void k_moe_logits(const uint16_t* __restrict__ x, int M, int K,
                                                    const uint16_t* __restrict__ r, int E,
                                                    double* __restrict__ logits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 4 + wave;
    const int m = blockIdx.y;
    if (e >= E) return;
    double s = 0.0;
    for (int k = lane * 8; k < K; k += 512) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(x + (size_t)m * K + k);
        const u32x4 b = *reinterpret_cast<const u32x4*>(r + (size_t)e * K + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fma((double)T::to_f32(a[i] & 0xFFFFu), (double)T::to_f32(b[i] & 0xFFFFu), s);
            s = fma((double)T::to_f32(a[i] >> 16), (double)T::to_f32(b[i] >> 16), s);
        }
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o);
    if (lane == 0) logits[(size_t)m * E + e] = s;
}

// Total order of float64 values as unsigned integers: -0 as +0, NaN above
// everything, so that the ranks of a row are always a permutation.
__device__ __forceinline__ unsigned long long order_key(double v) {
    if (v != v) return ~0ull;
    unsigned long long u = __builtin_bit_cast(unsigned long long, v + 0.0);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

// ---------------------------------------------------------------------------
// Top-k, softmax and the lists of the chosen experts: one block of 16 waves,
// a wave per token.
// ---------------------------------------------------------------------------
constexpr int kRouteWaves = 16;

__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(const double* __restrict__ logits, int M, int E,
                                                                int topk, int norm, int slots, int32_t* ids_ws,
                                                                float* weights_ws, int32_t* lists,
                                                                int16_t* slot_pair, int32_t* ids_out,
                                                                float* weights_out) {
    __shared__ int count[kMoeMaxExperts], slot_of[kMoeMaxExperts];
    __shared__ int wave_sum[2][kRouteWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < E; e += 64 * kRouteWaves) count[e] = 0;
    for (int i = tid; i < slots * kChunk; i += 64 * kRouteWaves) slot_pair[i] = -1;
    __syncthreads();
    for (int m = wave; m < M; m += kRouteWaves) {
        const double* row = logits + (size_t)m * E;
        double v[kMoeMaxExperts / 64];
        unsigned long long key[kMoeMaxExperts / 64];
        double top = 0.0;
#pragma unroll
        for (int i = 0; i < kMoeMaxExperts / 64; ++i) {
            const int e = i * 64 + lane;
            key[i] = 0;   // below every value's key (-inf maps to 0x000F..F)
            v[i] = 0.0;
            if (e < E) {
                v[i] = row[e];
                key[i] = order_key(v[i]);
            }
        }
        int mine_id = 0;
        float mine_p = 0.0f, chosen = 0.0f;
        for (int r = 0; r < topk; ++r) {
            unsigned long long best = 0;
            int at = kMoeMaxExperts;
#pragma unroll
            for (int i = 0; i < kMoeMaxExperts / 64; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i * 64 + lane;
                }
#pragma unroll
            for (int o = 1; o < 64; o *= 2) {
                const unsigned long long b = __shfl_xor(best, o);
                const int a = __shfl_xor(at, o);
                if (b > best || (b == best && a < at)) {
                    best = b;
                    at = a;
                }
            }
            double val = 0.0;
#pragma unroll
            for (int i = 0; i < kMoeMaxExperts / 64; ++i)
                if (at == i * 64 + lane) {
                    key[i] = 0;
                    val = v[i];
                }
            val = __shfl(val, at & 63);
            if (r == 0) top = val;
            const float p = expf((float)(val - top));
            chosen += p;
            if (lane == r) {
                mine_id = at;
                mine_p = p;
            }
        }
        float sum = chosen;
        if (!norm) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kMoeMaxExperts / 64; ++i)
                if (i * 64 + lane < E) sum += expf((float)(v[i] - top));
#pragma unroll
            for (int o = 1; o < 64; o *= 2) sum += __shfl_xor(sum, o);
        }
        if (lane < topk) {
            const int p = m * topk + lane;
            const float c = mine_p / sum;
            ids_ws[p] = mine_id;
            weights_ws[p] = c;
            if (ids_out) ids_out[p] = mine_id;
            if (weights_out) weights_out[p] = c;
            atomicAdd(&count[mine_id], 1);
        }
    }
    __syncthreads();
    // slots of the chosen experts in the order of their index, and where
    // each one's pairs begin: a scan over the experts (E <= 1024 threads)
    const MoeLists l = moe_lists(lists, slots);
    const int n = tid < E ? count[tid] : 0;
    int a = n > 0 ? 1 : 0, b = n;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int pa = __shfl_up(a, o), pb = __shfl_up(b, o);
        if (lane >= o) {
            a += pa;
            b += pb;
        }
    }
    if (lane == 63) {
        wave_sum[0][wave] = a;
        wave_sum[1][wave] = b;
    }
    __syncthreads();
    for (int i = 0; i < wave; ++i) {
        a += wave_sum[0][i];
        b += wave_sum[1][i];
    }
    if (n > 0) {
        l.expert[a - 1] = tid;
        l.offset[a - 1] = b - n;
        slot_of[tid] = a - 1;
        count[tid] = b - n;   // next free place of its pairs
    }
    if (tid == 64 * kRouteWaves - 1) {
        l.active[0] = a;
        l.offset[a] = b;
    }
    __syncthreads();
    for (int p = tid; p < M * topk; p += 64 * kRouteWaves) {
        const int e = ids_ws[p], s = slot_of[e];
        l.pair[atomicAdd(&count[e], 1)] = p;   // the order inside a slot moves columns, not sums
        slot_pair[(size_t)s * kChunk + p / topk] = (int16_t)p;
    }
}

// ---------------------------------------------------------------------------
// Gate and up: a block owns 16 rows of one chosen expert's gate and up
// weights; its waves split K, the tokens of the expert go 16 at a time.
// ---------------------------------------------------------------------------
constexpr int kWaves = 4;

template <class T, int GPU, bool ZP>
__global__ __launch_bounds__(64 * kWaves) void k_moe_gate_up(const uint16_t* __restrict__ x, int M, int K, int F,
                                                             const uint8_t* __restrict__ wg,
                                                             const uint8_t* __restrict__ wu, int topk, int slots,
                                                             int32_t* lists, const float* __restrict__ weights,
                                                             uint16_t* __restrict__ h) {
    __shared__ f32x4 part[kWaves][2][64];
    const MoeLists ml = moe_lists(lists, slots);
    const int slot = blockIdx.y;
    if (slot >= ml.active[0]) return;
    const int e = ml.expert[slot], begin = ml.offset[slot], end = ml.offset[slot + 1];
    const W4gLayout l = w4g_layout(128 / GPU, ZP, F, K);
    wg += (size_t)e * l.total;
    wu += (size_t)e * l.total;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t tile = blockIdx.x;
    const buf_t xb = w4g_buf(x, M, K);
    for (int p0 = begin; p0 < end; p0 += 16) {
        const int mine = p0 + (lane & 15);
        const uint32_t row = mine < end ? (uint32_t)(ml.pair[mine] / topk) * (2u * K) : kNoRow;
        f32x4 acc[1][2] = {{f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}};
        for (int u = wave; u < l.units; u += kWaves) {
            const W4gUnit<GPU> w[2] = {w4g_load<GPU, ZP>(wg, l, tile * l.units + u, lane),
                                       w4g_load<GPU, ZP>(wu, l, tile * l.units + u, lane)};
#pragma unroll
            for (int g = 0; g < GPU; ++g) {
                u32x4 a[1][4 / GPU];
#pragma unroll
                for (int s = 0; s < 4 / GPU; ++s)
                    a[0][s] = w4g_x(xb, row, u * 128 + (g * (4 / GPU) + s) * 32 + (lane >> 4) * 8, K);
                w4g_mac<T, GPU, ZP, 1, 2>(g, w, a, acc);
            }
        }
        part[wave][0][lane] = acc[0][0];
        part[wave][1][lane] = acc[0][1];
        __syncthreads();
        const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
        if (p0 + m < end) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int wv = 0; wv < kWaves; ++wv) {
                g += part[wv][0][(m >> 2) * 16 + n][m & 3];
                u += part[wv][1][(m >> 2) * 16 + n][m & 3];
            }
            const int p = ml.pair[p0 + m];
            h[(size_t)p * F + tile * 16 + n] = T::from_f32(g / (1.0f + expf(-g)) * u * weights[p]);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Down and combination: a block owns 16 columns of y for every token and
// walks the units of all chosen experts; h already holds the routing weight,
// so the experts' sums add up in the same accumulators.
// ---------------------------------------------------------------------------
template <class T, int GPU, bool ZP, int MT>
__global__ __launch_bounds__(64 * kWaves) void k_moe_down(const uint16_t* __restrict__ h, int M, int F, int N, int topk,
                                                          const uint8_t* __restrict__ wd, int slots, int32_t* lists,
                                                          const int16_t* __restrict__ slot_pair,
                                                          uint16_t* __restrict__ y) {
    __shared__ f32x4 part[kWaves][MT][64];
    const MoeLists ml = moe_lists(lists, slots);
    const W4gLayout l = w4g_layout(128 / GPU, ZP, N, F);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const size_t tile = blockIdx.x;
    const int total = ml.active[0] * l.units;
    const buf_t hb = w4g_buf(h, M * topk, F);
    f32x4 acc[MT][1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][0] = f32x4{0, 0, 0, 0};
    for (int i = wave; i < total; i += kWaves) {
        const int slot = i / l.units, u = i - slot * l.units;
        const W4gUnit<GPU> w[1] = {
            w4g_load<GPU, ZP>(wd + (size_t)ml.expert[slot] * l.total, l, tile * l.units + u, lane)};
        uint32_t row[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int p = slot_pair[(size_t)slot * kChunk + mt * 16 + (lane & 15)];
            row[mt] = p >= 0 ? (uint32_t)p * (2u * F) : kNoRow;
        }
#pragma unroll
        for (int g = 0; g < GPU; ++g) {
            u32x4 a[MT][4 / GPU];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int s = 0; s < 4 / GPU; ++s)
                    a[mt][s] = w4g_x(hb, row[mt], u * 128 + (g * (4 / GPU) + s) * 32 + (lane >> 4) * 8, F);
            w4g_mac<T, GPU, ZP, MT, 1>(g, w, a, acc);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[wave][mt][lane] = acc[mt][0];
    __syncthreads();
    for (int i = threadIdx.x; i < 256 * MT; i += 64 * kWaves) {
        const int m = i >> 4, n = i & 15;
        const size_t gn = tile * 16 + n;
        if (m >= M || gn >= (size_t)N) continue;
        float v = 0.0f;
#pragma unroll
        for (int wv = 0; wv < kWaves; ++wv) v += part[wv][m >> 4][((m & 15) >> 2) * 16 + n][m & 3];
        y[(size_t)m * N + gn] = T::from_f32(v);
    }
}

template <class T, int GPU, bool ZP>
hipError_t moe_t(const MoeArgs& a, const MoeWs& l, int M, const uint16_t* x, uint16_t* y, int32_t* ids,
                 float* weights, hipStream_t st) {
    char* ws = static_cast<char*>(a.ws);
    double* logits = reinterpret_cast<double*>(ws + l.logits);
    int32_t* lists = reinterpret_cast<int32_t*>(ws + l.lists);
    int32_t* ids_ws = reinterpret_cast<int32_t*>(ws + l.ids);
    float* weights_ws = reinterpret_cast<float*>(ws + l.weights);
    int16_t* slot_pair = reinterpret_cast<int16_t*>(ws + l.slot_pair);
    uint16_t* h = reinterpret_cast<uint16_t*>(ws + l.h);
    const int pairs = M * a.topk, slots = pairs < a.E ? pairs : a.E;
    k_moe_logits<T><<<dim3((a.E + 3) / 4, M), 256, 0, st>>>(x, M, a.K, a.router, a.E, logits);
    k_moe_route<<<1, 64 * kRouteWaves, 0, st>>>(logits, M, a.E, a.topk, a.norm, slots, ids_ws, weights_ws, lists,
                                                slot_pair, ids, weights);
    k_moe_gate_up<T, GPU, ZP><<<dim3(a.F / 16, slots), 64 * kWaves, 0, st>>>(x, M, a.K, a.F, a.wg, a.wu, a.topk, slots,
                                                                            lists, weights_ws, h);
    const dim3 dg((a.K + 15) / 16), db(64 * kWaves);
    if (M <= 16)
        k_moe_down<T, GPU, ZP, 1><<<dg, db, 0, st>>>(h, M, a.F, a.K, a.topk, a.wd, slots, lists, slot_pair, y);
    else if (M <= 32)
        k_moe_down<T, GPU, ZP, 2><<<dg, db, 0, st>>>(h, M, a.F, a.K, a.topk, a.wd, slots, lists, slot_pair, y);
    else
        k_moe_down<T, GPU, ZP, 4><<<dg, db, 0, st>>>(h, M, a.F, a.K, a.topk, a.wd, slots, lists, slot_pair, y);
    return hipGetLastError();
}

template <class T>
hipError_t moe_pass(const MoeArgs& a, const MoeWs& l, int M, const uint16_t* x, uint16_t* y, int32_t* ids,
                    float* weights, hipStream_t st) {
    switch (a.group) {
        case 32: return a.zeros ? moe_t<T, 4, true>(a, l, M, x, y, ids, weights, st) : moe_t<T, 4, false>(a, l, M, x, y, ids, weights, st);
        case 64: return a.zeros ? moe_t<T, 2, true>(a, l, M, x, y, ids, weights, st) : moe_t<T, 2, false>(a, l, M, x, y, ids, weights, st);
        default: return a.zeros ? moe_t<T, 1, true>(a, l, M, x, y, ids, weights, st) : moe_t<T, 1, false>(a, l, M, x, y, ids, weights, st);
    }
}

}  // namespace

size_t moe_workspace(int M, int F, int E, int topk) { return moe_ws(M, F, E, topk).total; }

hipError_t launch_moe(const MoeArgs& a, hipStream_t st) {
    const MoeWs l = moe_ws(a.M, a.F, a.E, a.topk);
    for (int m = 0; m < a.M; m += kChunk) {
        const int n = a.M - m < kChunk ? a.M - m : kChunk;
        const uint16_t* x = a.x + (size_t)m * a.K;
        uint16_t* y = a.y + (size_t)m * a.K;
        int32_t* ids = a.ids ? a.ids + (size_t)m * a.topk : nullptr;
        float* weights = a.weights ? a.weights + (size_t)m * a.topk : nullptr;
        const hipError_t e = a.fp16 ? moe_pass<Fp16>(a, l, n, x, y, ids, weights, st)
                                    : moe_pass<Bf16>(a, l, n, x, y, ids, weights, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace cr
