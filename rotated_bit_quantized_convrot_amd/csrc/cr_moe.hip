// Mixture-of-experts layer on 4-bit weights with group scales, for a few
// tokens: router logits, top-k and softmax, the chosen experts' gated MLPs
// and their weighted sum, in three launches.
//
//   l[m,e] = sum_k x[m,k] r[e,k];  e_0..e_{k-1} the largest, ties to the lower e
//   p = exp(l - max l),  c[m,r] = p[e_r] / (sum over the chosen, or over all)
//   h[m,r] = silu(Wg_e x[m]) (Wu_e x[m])
//   y[m]   = T(sum_r c[m,r] Wd_{e_r} h[m,r])       (T: the 16-bit type)
//
// A pass is bound by the chosen experts' weights, each read once, and for a
// single token by the launches and the loads that wait for each other.  So
// there is no launch for the choice: whether expert e is chosen by token m is
// a count of the logits above l[m,e], which every block of the gate / up
// kernel makes for itself; the down kernel reads the chosen ids.
// h goes to the down product as it is in float32, as the sum of three bf16
// values of 8 bits each (in bf16's range for either T): y's rounding is the
// only one to fewer bits.  The three are rows of one MFMA operand, or operands
// of MFMAs into the same sums.
// Both products bring a wave's operand rows to its own piece of LDS, by as
// many 4-row instructions as it has rows (an expert of a few tokens has 1 to
// 3, so most of a 16-row load by registers would be for nothing), and
// take them to registers before the next unit's are brought to the same place.
#include <type_traits>

#include "cr_w4g.h"

namespace cr {
namespace {

constexpr int kChunk = kMoeChunk;   // tokens per pass
constexpr int kParts = 3;           // bf16 values whose sum is h

// The down product's grid: blocks by columns, and on the same columns enough
// to fill the chip's CUs twice, each wave (or group of waves) with at least
// two (expert, unit) items.
constexpr int kDownWaves = 8, kMaxSplits = 8, kWideTiles = 4, kWideGroups = kDownWaves / kWideTiles;
constexpr int kDownTok = 5, kWideTok = 16;   // tokens of a pass, apart and in wide blocks
// Gate / up: an expert has some tokens, so that sharing their rows among tiles
// pays; us, apart / shared: 64 tokens, 8 experts (16 each) 85 / 54, 32 experts
// (12) 27 / 27, 60 experts (4.3) 45 / 52, 128 experts (4) 53 / 65; 8 experts, 32
// tokens (8) 45 / 43, 20 tokens (5) 45 / 42.  With up to 16 tokens there is little
// in it: 16 on 8 of 8 experts 51 / 46 and 17.9 / 18.8, 12 on 4 of 8 21 / 23.
bool share_rows(int M, int E, int topk) { return M > 16 && (long)M * topk >= 5L * E; }
// Down: blocks of four tiles that share the rows of h pay where an expert's
// tokens are more than a pass of a block apart takes, the more of them the
// fewer blocks the columns can give (K / 64 times kMaxSplits: 512 at K = 4096);
// us, apart / wide, by tokens an expert:
//   K = 4096   6: 76 / 70   8: 54 / 38   16: 90 / 56.5 (64 tokens, 2 of 8, F = 5632), 34 / 27 (F = 1792)
//   K = 2880   6: 26 / 24   8: 31 / 25.5, 105 / 72 (32 experts)   16: 46 / 34
//   K = 2048   8: 17 / 18, 26 / 30, 41 / 41   12: 42 / 38   16: 50 / 46, 23.5 / 22.6, 27 / 18
//   K = 1536  32: 26.3 / 25.9   K = 1024   8: 9.4 / 11   16: 23 / 31
bool wide_down(int M, int wide_columns, int E, int topk) {
    const long pairs = (long)M * topk, blocks = (long)wide_columns * kMaxSplits;
    return pairs >= 12L * E ? blocks >= 256 : pairs >= 5L * E && blocks >= 352;
}
struct DownGrid {
    bool wide;
    int columns, splits;
};
DownGrid down_grid(int M, int F, int N, int E, int topk) {
    const long pairs = (long)M * topk, items = (pairs < E ? pairs : E) * ((F + 127) / 128);
    DownGrid g;
    const int wide = (N / 16 + kWideTiles - 1) / kWideTiles;
    g.wide = wide_down(M, wide, E, topk);
    g.columns = g.wide ? wide : N / 16;
    const long most = items / (2 * (g.wide ? kWideGroups : kDownWaves));
    long s = 512 / g.columns;
    s = s < most ? s : most;
    g.splits = s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : (int)s);
    return g;
}

// Workspace of one pass (byte offsets, 256-byte regions).
struct MoeWs {
    size_t logits, ids, top, h, arrived, parts, total;
};
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
MoeWs moe_ws(int M, int K, int F, int E, int topk) {
    const size_t m = M < kChunk ? M : kChunk, pairs = m * topk;
    // neither the splits nor the tokens of a last, smaller pass are more
    const size_t splits = m ? down_grid((int)m, F, K, E, topk).splits : 1, parts = splits > 1 ? splits * m : 0;
    MoeWs l;
    l.logits = 0;                                        // double [m][E]
    l.ids = l.logits + up256(m * E * 8);                 // int32 [m][topk]
    l.top = l.ids + up256(pairs * 4);                    // double [m][topk]: the chosen logits
    l.h = l.top + up256(pairs * 8);                      // bf16 [m topk][kParts][F]
    l.arrived = l.h + up256(pairs * F * 2 * kParts);     // uint32 [K / 16]
    l.parts = l.arrived + up256((size_t)(K / 16) * 4);   // float [splits][m][K]
    l.total = l.parts + up256(parts * K * 4);
    return l;
}

// ---------------------------------------------------------------------------
// Router logits in float64: which expert is chosen hangs on the order of
// values that can be close, and the sums then do not depend on their order.
// A wave per expert and token (the router's row comes from the caches again
// for each token: 4 tokens a wave took 9.7 us at 16 tokens, 128 experts,
// K = 2048, this 4.7).
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(256) void k_moe_logits(const uint16_t* __restrict__ x, int K,
                                                    const uint16_t* __restrict__ r, int E,
                                                    double* __restrict__ logits, uint32_t* __restrict__ arrived,
                                                    int counters) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 4 + wave, m = blockIdx.y;
    // the down kernel's arrival counters start at 0
    if (m == 0)
        for (int i = blockIdx.x * 256 + threadIdx.x; i < counters; i += gridDim.x * 256) arrived[i] = 0;
    if (e >= E) return;
    double s = 0.0;
#pragma unroll 4
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
typedef unsigned long long u64;
__device__ __forceinline__ u64 order_key(double v) {
    if (v != v) return ~0ull;
    const u64 u = __builtin_bit_cast(u64, v + 0.0);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

// ---------------------------------------------------------------------------
// Gate and up.  blockIdx.y is a (token, rank) pair where there are fewer
// pairs than experts, else an expert.  The block finds its expert and the
// tokens that chose it; a block whose expert no token chose, or whose expert
// an earlier token's pair already stands for, ends.  `ks` of its waves share
// a tile of 16 rows of the expert's gate and up weights and take the units of
// K in turn, each loading one unit ahead of its products; tokens go 16 at a
// time.  With ks = 1 nothing is waited for but a wave's own loads.
// Bound by the weights' bytes, after some 3 us in which a block finds its
// expert: us, F x K = 768 x 2048, 8 of 128 experts: 9 for a token (13 MB),
// 38 for 16 (134 MB: 3.5 TB/s).
// ---------------------------------------------------------------------------
constexpr int kUpWaves = 8;

struct Choice {
    int16_t rank_of[kChunk], list[kChunk];   // of the block's expert: rank by token (-1: not chosen), tokens
    int chosen;
};
struct ByRank {
    int16_t above[kUpWaves][kMoeMaxExperts];   // by wave and expert: the logits above its own in the wave's share
    int found;
};
// The expert of rank `want` in a row of up to 64 EACH logits: each wave counts, for
// every expert, which of its share of the row lie above it; the share comes
// by uniform loads, so that a comparison takes a scalar operand and LDS only
// the counts.  (The largest taken out `want` + 1 times by wave-wide maxima
// costs 0.5 us a rank; counting by reads of LDS 3 us at 128 experts.)
template <int WAVES, int EACH>
__device__ __forceinline__ int moe_of_rank(ByRank& c, const double* __restrict__ row, int E, int want) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int share = (E + WAVES - 1) / WAVES, j0 = wave * share, j1 = j0 + share < E ? j0 + share : E;
    u64 key[EACH];
    int n[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = i * 64 + lane;
        key[i] = order_key(row[e < E ? e : E - 1]);
        n[i] = 0;
    }
#pragma unroll 2
    for (int j = j0; j < j1; ++j) {
        const u64 k = order_key(row[j]);
#pragma unroll
        for (int i = 0; i < EACH; ++i) n[i] += k > key[i] || (k == key[i] && j < i * 64 + lane);
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (i * 64 + lane < E) c.above[wave][i * 64 + lane] = (int16_t)n[i];
    __syncthreads();
    for (int e = tid; e < E; e += 64 * WAVES) {
        int all = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) all += c.above[w][e];
        if (all == want) c.found = e;   // ranks are a permutation: one thread
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(c.found);
}

// The tokens of expert e (c.list, c.rank_of); returns their number, 0 where one
// before token `first` chose it too.  Blocks of the first tile write the choice
// down: ids and logits by (token, rank).
template <int WAVES>
__device__ __forceinline__ int moe_tokens(Choice& c, int M, int E, int topk, int e, int first,
                                          const double* __restrict__ logits, int32_t* __restrict__ ids,
                                          double* __restrict__ top) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the rank of e in every row: the logits above its own, counted by a wave,
    // four rows and 128 logits under way at a time
    constexpr int kRows = 4, kCols = 2;
    for (int m0 = wave; m0 < M; m0 += WAVES * kRows) {
        u64 mine[kRows];
        int n[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int m = m0 + r * WAVES < M ? m0 + r * WAVES : m0;
            mine[r] = order_key(logits[(size_t)m * E + e]);
            n[r] = 0;
        }
        for (int j0 = 0; j0 < E; j0 += 64 * kCols) {
            double v[kRows][kCols];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    const int m = m0 + r * WAVES < M ? m0 + r * WAVES : m0, j = j0 + i * 64 + lane;
                    v[r][i] = logits[(size_t)m * E + (j < E ? j : E - 1)];
                }
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    const int j = j0 + i * 64 + lane;
                    const u64 o = order_key(v[r][i]);
                    n[r] += __popcll(__ballot(j < E && (o > mine[r] || (o == mine[r] && j < e))));
                }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (lane == 0 && m0 + r * WAVES < M) c.rank_of[m0 + r * WAVES] = (int16_t)(n[r] < topk ? n[r] : -1);
    }
    __syncthreads();
    if (wave == 0) {
        const bool mine = lane < M && c.rank_of[lane] >= 0;
        const u64 all = __ballot(mine);
        if (mine) {
            c.list[__popcll(all & ((1ull << lane) - 1))] = (int16_t)lane;
            if (blockIdx.x == 0) {
                ids[lane * topk + c.rank_of[lane]] = e;
                top[lane * topk + c.rank_of[lane]] = logits[(size_t)lane * E + e];
            }
        }
        if (lane == 0) c.chosen = (all & ((1ull << first) - 1)) ? 0 : __popcll(all);
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(c.chosen);
}

// The same where blockIdx.y is a (token, rank) pair: the expert comes out in e,
// and a block that has nothing to do gets 0.
template <int WAVES>
__device__ __forceinline__ int moe_choice_by_pair(Choice& c, ByRank& by, int M, int E, int topk,
                                                  const double* __restrict__ logits, int32_t* __restrict__ ids,
                                                  double* __restrict__ top, int& e) {
    const int first = blockIdx.y / topk, want = blockIdx.y - first * topk;
    const double* row = logits + (size_t)first * E;
    e = E <= 128 ? moe_of_rank<WAVES, 2>(by, row, E, want)
                 : E <= 256 ? moe_of_rank<WAVES, 4>(by, row, E, want)
                            : moe_of_rank<WAVES, kMoeMaxExperts / 64>(by, row, E, want);
    if (M > 1) return moe_tokens<WAVES>(c, M, E, topk, e, first, logits, ids, top);
    if (threadIdx.x == 0) {
        c.rank_of[0] = (int16_t)want;
        c.list[0] = 0;
        if (blockIdx.x == 0) {
            ids[want] = e;
            top[want] = logits[e];
        }
    }
    __syncthreads();
    return 1;
}

// silu(g) u into element n of pair p's h: the upper 8 bits of its significand, the next 8 and the last 8,
// each a bf16 value; the differences are exact (down to bf16's smallest
// number).  An infinity has no rest.
__device__ __forceinline__ void moe_store_h(uint16_t* h, int p, int F, int n, float g, float u) {
    float v = g / (1.0f + expf(-g)) * u;
    uint16_t* to = h + (size_t)p * kParts * F + n;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        const uint32_t top = __float_as_uint(v) & 0xFFFF0000u;
        to[(size_t)i * F] = (uint16_t)(top >> 16);
        v = (top & 0x7F800000u) == 0x7F800000u ? 0.0f : v - __uint_as_float(top);
    }
}

// Element f of pair p's h from the products' definition: for accumulators
// that are not finite.  Kept out of the loops that store the others, where a
// copy for each of their elements cost 8 us of 73 (64 tokens, 2 of 8 experts of
// 5632 x 4096 with zero points).
template <class T, int GPU, bool ZP>
__device__ __forceinline__ void moe_hidden_defined(const uint16_t* x, int K, int F, const uint8_t* wg, const uint8_t* wu,
                                                   const W4gLayout& l, uint16_t* h, int p, int f) {
    float v[2] = {0.0f, 0.0f};
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        v[0] = v[1];
        v[1] = w4g_defined_row<T, GPU, ZP>(x, K, i ? wu : wg, l, f);
    }
    moe_store_h(h, p, F, f, v[0], v[1]);
}

template <class T, int GPU, bool ZP>
__global__ __launch_bounds__(64 * kUpWaves, 4) void k_moe_gate_up(const uint16_t* __restrict__ x, int M, int K, int F,
                                                               const uint8_t* __restrict__ wg,
                                                               const uint8_t* __restrict__ wu, int E, int topk,
                                                               int by_pair, int ks_log2,
                                                               const double* __restrict__ logits,
                                                               int32_t* __restrict__ ids, double* __restrict__ top,
                                                               uint16_t* __restrict__ h) {
    __shared__ Choice c;
    __shared__ ByRank by_rank;
    __shared__ __attribute__((aligned(16))) char rows_lds[kUpWaves][4096];
    __shared__ f32x4 part[kUpWaves][2][64];
    constexpr int kThreads = 64 * kUpWaves;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int e = blockIdx.y;
    const int n_tok = by_pair ? moe_choice_by_pair<kUpWaves>(c, by_rank, M, E, topk, logits, ids, top, e)
                              : moe_tokens<kUpWaves>(c, M, E, topk, e, 0, logits, ids, top);
    if (n_tok == 0) return;

    const W4gLayout l = w4g_layout(128 / GPU, ZP, F, K);
    wg += (size_t)e * l.total;
    wu += (size_t)e * l.total;
    const v4i xb = w4g_rows(x, M, K);
    const int ks = 1 << ks_log2, part_k = wave & (ks - 1);
    const int tile = blockIdx.x * (kUpWaves >> ks_log2) + (wave >> ks_log2);
    const bool work = tile < l.tiles;
    const char* my_rows = rows_lds[wave];
    const uint32_t my_lds = lds_address(my_rows);
    uint32_t again = 0;   // this thread's elements to be formed from the definition: four for each 16 tokens
    static_assert(256 * (kUpWaves / 2) <= 4 * kThreads && kChunk <= 128, "its bits");
    for (int p0 = 0; p0 < n_tok; p0 += 16) {
        const int n = n_tok - p0 < 16 ? n_tok - p0 : 16, fills = (n + 3) >> 2;
        uint32_t row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = 4 * j + (lane >> 4);
            row[j] = (uint32_t)c.list[p0 + (m < n ? m : n - 1)] * (2u * K);
        }
        f32x4 acc[2][1][1] = {{{f32x4{0, 0, 0, 0}}}, {{f32x4{0, 0, 0, 0}}}};   // gate, up
        W4gUnit<GPU> next[2][1];
        auto load = [&](int u) {
            next[0][0] = w4g_load<GPU, ZP>(wg, l, (size_t)tile * l.units + u, lane);
            next[1][0] = w4g_load<GPU, ZP>(wu, l, (size_t)tile * l.units + u, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < fills) w4g_x_to_lds(xb, row[j] + w4g_chunk(4 * j, u, K, lane), my_lds + j * 1024);
        };
        if (work && part_k < l.units) {
            load(part_k);
            for (int u = part_k; u < l.units; u += ks) {
                w4g_wait();
                const W4gUnit<GPU> w[2][1] = {{next[0][0]}, {next[1][0]}};
                u32x4 a[GPU][1][4 / GPU];
#pragma unroll
                for (int d = 0; d < 4; ++d) a[d / (4 / GPU)][0][d % (4 / GPU)] = w4g_operand_rows(my_rows, d, lane);
                w4g_wait_lds();
                if (u + ks < l.units) load(u + ks);
                // one weight's products after the other's: fewer registers
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int g = 0; g < GPU; ++g) w4g_mac<T, GPU, ZP, 1, 1>(g, w[i], a[g], acc[i]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        auto store = [&](int m, int n, float g, float u) {
            const int t = c.list[p0 + m];
            moe_store_h(h, t * topk + c.rank_of[t], F, n, 16.0f * g, 16.0f * u);
            return w4g_finite(16.0f * g) && w4g_finite(16.0f * u);
        };
        if (ks == 1) {
            if (work) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = (lane >> 4) * 4 + i;
                    if (p0 + m < n_tok && !store(m, tile * 16 + (lane & 15), acc[0][0][0][i], acc[1][0][0][i]))
                        again |= 1u << (p0 / 4 + i);
                }
            }
            continue;
        }
        part[wave][0][lane] = acc[0][0][0];
        part[wave][1][lane] = acc[1][0][0];
        __syncthreads();
        for (int i = tid; i < 256 * (kUpWaves >> ks_log2); i += kThreads) {
            const int m = (i >> 4) & 15, n = i & 15, w0 = (i >> 8) << ks_log2;
            const int t = blockIdx.x * (kUpWaves >> ks_log2) + (i >> 8);
            if (p0 + m >= n_tok || t >= l.tiles) continue;
            float g = 0.0f, u = 0.0f;
            for (int wv = w0; wv < w0 + ks; ++wv) {
                g += part[wv][0][(m >> 2) * 16 + n][m & 3];
                u += part[wv][1][(m >> 2) * 16 + n][m & 3];
            }
            if (!store(m, t * 16 + n, g, u)) again |= 1u << (p0 / 4 + i / kThreads);
        }
        __syncthreads();
    }
    for (; again; again &= again - 1) {
        const int b = __builtin_ctz(again), i = tid + kThreads * (b & 3);
        const int m = b / 4 * 16 + (ks == 1 ? (lane >> 4) * 4 + (b & 3) : (i >> 4) & 15);
        const int f = ks == 1 ? tile * 16 + (lane & 15) : (blockIdx.x * (kUpWaves >> ks_log2) + (i >> 8)) * 16 + (i & 15);
        const int t = c.list[m];
        moe_hidden_defined<T, GPU, ZP>(x + (size_t)t * K, K, F, wg, wu, l, h, t * topk + c.rank_of[t], f);
    }
}

// ---------------------------------------------------------------------------
// Gate and up, more tokens: the same, but the block's waves own a tile each
// and go through K together, so that the rows of x are brought once for all
// of them; up to 32 tokens at once, in one 16-row operand or two.  52 us for
// 64 tokens, 2 of 8 experts of 5632 x 4096 (196 MB: 3.8 TB/s).
// ---------------------------------------------------------------------------
constexpr int kManyWaves = 4;
template <class T, int GPU, bool ZP>
__global__ __launch_bounds__(64 * kManyWaves, 4) void k_moe_gate_up_many(
    const uint16_t* __restrict__ x, int M, int K, int F, const uint8_t* __restrict__ wg,
    const uint8_t* __restrict__ wu, int E, int topk, const double* __restrict__ logits, int32_t* __restrict__ ids,
    double* __restrict__ top, uint16_t* __restrict__ h) {
    __shared__ Choice c;
    constexpr int kStage = 8192;
    __shared__ __attribute__((aligned(16))) char rows_lds[2 * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e = blockIdx.y;   // no fewer pairs than experts here: share_rows
    const int n_tok = moe_tokens<kManyWaves>(c, M, E, topk, e, 0, logits, ids, top);
    if (n_tok == 0) return;

    const W4gLayout l = w4g_layout(128 / GPU, ZP, F, K);
    wg += (size_t)e * l.total;
    wu += (size_t)e * l.total;
    const v4i xb = w4g_rows(x, M, K);
    const int tile = blockIdx.x * kManyWaves + wave, mine = tile < l.tiles ? tile : l.tiles - 1;
    const uint32_t lds0 = lds_address(rows_lds);
    uint32_t again = 0;   // this lane's elements to be formed from the definition: four for each 16 tokens
    auto run = [&](auto mt_count, int p0) {
        constexpr int MT = decltype(mt_count)::value;
        // wave w brings rows 4 w..4 w + 3, and 16 more than that
        const int n = n_tok - p0 < 16 * MT ? n_tok - p0 : 16 * MT, r0 = 4 * wave;
        uint32_t row[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = 16 * mt + r0 + (lane >> 4);
            row[mt] = (uint32_t)c.list[p0 + (m < n ? m : n - 1)] * (2u * K);
        }
        W4gUnit<GPU> next[2];
        auto load = [&](int u, int stage) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                if (16 * mt + r0 < n)
                    w4g_x_to_lds(xb, row[mt] + w4g_chunk(r0, u, K, lane), lds0 + stage * kStage + mt * 4096 + r0 * 256);
            next[0] = w4g_load<GPU, ZP>(wg, l, (size_t)mine * l.units + u, lane);
            next[1] = w4g_load<GPU, ZP>(wu, l, (size_t)mine * l.units + u, lane);
        };
        f32x4 acc[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = f32x4{0, 0, 0, 0};
        load(0, 0);
        for (int u = 0, stage = 0; u < l.units; ++u, stage ^= 1) {
            w4g_wait();
            w4g_barrier();   // the unit's rows are there, the other stage has been read
            const W4gUnit<GPU> w[2] = {next[0], next[1]};
            if (u + 1 < l.units) load(u + 1, stage ^ 1);
#pragma unroll
            for (int g = 0; g < GPU; ++g) {
                u32x4 a[MT][4 / GPU];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int s = 0; s < 4 / GPU; ++s)
                        a[mt][s] = w4g_operand_rows(rows_lds + stage * kStage + mt * 4096, g * (4 / GPU) + s, lane);
                w4g_mac<T, GPU, ZP, MT, 2>(g, w, a, acc);
            }
        }
        w4g_barrier();   // before the next tokens' rows come into the first stage
        if (tile >= l.tiles) return;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = mt * 16 + (lane >> 4) * 4 + i;
                if (m >= n) continue;
                const int t = c.list[p0 + m];
                const float g = 16.0f * acc[mt][0][i], v = 16.0f * acc[mt][1][i];
                moe_store_h(h, t * topk + c.rank_of[t], F, tile * 16 + (lane & 15), g, v);
                if (!w4g_finite(g) || !w4g_finite(v)) again |= 1u << (p0 / 4 + mt * 4 + i);
            }
    };
    for (int p0 = 0; p0 < n_tok; p0 += 32) {
        if (n_tok - p0 <= 16) run(std::integral_constant<int, 1>{}, p0);
        else run(std::integral_constant<int, 2>{}, p0);
    }
    for (; again; again &= again - 1) {
        const int b = __builtin_ctz(again), t = c.list[b / 4 * 16 + (lane >> 4) * 4 + (b & 3)];
        moe_hidden_defined<T, GPU, ZP>(x + (size_t)t * K, K, F, wg, wu, l, h, t * topk + c.rank_of[t],
                                       tile * 16 + (lane & 15));
    }
}

// ---------------------------------------------------------------------------
// Down and combination.  The pairs are sorted by expert and cut into passes of
// up to kDownTok tokens, whose rows of h lie in LDS with a token's three parts
// next to each other; the items (pass, unit of F) are shared out in contiguous
// runs.
// At the end of a pass a wave adds c times its sums into its own rows of LDS;
// the waves' rows are added in their order, and so are those of the gridDim.y
// blocks on the same columns, by the one that arrives last: the order of
// every sum is fixed.  The blocks' sums go through device-scope stores and
// loads, waited for before the arrival is counted; no fence of the caches is
// needed.  us: 7.2 for one token and 8 of 128 experts of 2048 x 768 (7 MB), 22
// for 16 tokens (67 MB: 3.1 TB/s).  With some tokens an expert a wave takes
// 4 KB of h for each KB of weights, and those rows' way through the L2 bounds
// it, not the weights: 64 tokens, 2 of 8 experts of 4096 x 5632 take 90 us for
// 98 MB, the wide form below 56.5.  (With h rounded to two bf16 values, 16 bits,
// the three sizes took 7, 21 and 49, and one output in 400 of the last was
// rounded otherwise than by the plain float32 form; now one in 900 is.)
// An operand holds a token's parts in three of its 16 rows, five tokens in
// all: an operand a part took 25 us where this takes 22, three times the reads
// of LDS.
// ---------------------------------------------------------------------------
struct Passes {
    static constexpr int kPairs = kChunk * kMoeMaxTopk;
    int16_t pair_of[kPairs];                               // pairs by expert, then by token
    int16_t expert[kPairs], at[kPairs], n[kPairs];         // of a pass
    float c[kPairs], total[kChunk];                        // of a pair, of a token
    int scan[2][16];
    uint32_t before;
};
// While those are made, in the LDS that the rows take later.
struct ByExpert {
    u64 tokens[kMoeMaxExperts];         // bit m: token m chose the expert
    double top[Passes::kPairs];         // the pairs' logits
    int16_t pairs_at[kMoeMaxExperts];   // where an expert's pairs begin
    int16_t expert[Passes::kPairs];     // of a pair
};

// Fills the passes and the pairs' weights (the softmax's numerators over the
// tokens' denominators); returns the number of passes.  One block writes the
// choice out.  The choice is read once, everything else happens in LDS.  ONE:
// the call can be of a single token.
template <int WAVES, int TOK, bool ONE>
__device__ __forceinline__ int moe_passes(Passes& s, ByExpert& by, int M, int E, int topk, int norm,
                                          const double* __restrict__ logits, const int32_t* __restrict__ ids,
                                          const double* __restrict__ top, bool write, int32_t* __restrict__ ids_out,
                                          float* __restrict__ weights_out) {
    constexpr int kThreads = 64 * WAVES, kEach = (kMoeMaxExperts + kThreads - 1) / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = M * topk;
    for (int p = tid; p < pairs; p += kThreads) {
        by.expert[p] = (int16_t)ids[p];
        by.top[p] = top[p];
    }
    const bool more = !ONE || M > 1;
    if (more)
        for (int e = tid; e < E; e += kThreads) by.tokens[e] = 0;
    if (!norm) {
        for (int m = wave; m < M; m += WAVES) {
            const double* of = logits + (size_t)m * E;
            const double most = top[m * topk];
            float v = 0.0f;
#pragma unroll 4
            for (int j = lane; j < E; j += 64) v += expf((float)(of[j] - most));
#pragma unroll
            for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
            if (lane == 0) s.total[m] = v;
        }
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int m = p / topk;
        s.c[p] = expf((float)(by.top[p] - by.top[m * topk]));
        if (more) {
            atomicOr(&by.tokens[by.expert[p]], 1ull << m);
        } else {
            s.pair_of[p] = s.at[p] = (int16_t)p;
            s.expert[p] = by.expert[p];
            s.n[p] = 1;
        }
    }
    __syncthreads();
    if (norm && tid < M) {
        float v = 0.0f;
        for (int r = 0; r < topk; ++r) v += s.c[tid * topk + r];
        s.total[tid] = v;
    }
    int passes = topk;
    if (more) {
        // a thread's kEach experts: their pairs and passes, and those before them
        int n[kEach], a = 0, b = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = tid * kEach + i;
            n[i] = e < E ? __popcll(by.tokens[e]) : 0;
            a += n[i];
            b += (n[i] + TOK - 1) / TOK;
        }
        const int own_a = a, own_b = b;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const int pa = __shfl_up(a, o), pb = __shfl_up(b, o);
            if (lane >= o) {
                a += pa;
                b += pb;
            }
        }
        if (lane == 63) {
            s.scan[0][wave] = a;
            s.scan[1][wave] = b;
        }
        __syncthreads();
        a -= own_a;
        b -= own_b;
        passes = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            if (i < wave) {
                a += s.scan[0][i];
                b += s.scan[1][i];
            }
            passes += s.scan[1][i];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (n[i] > 0) by.pairs_at[tid * kEach + i] = (int16_t)a;
            for (int q = 0; q < n[i]; q += TOK) {
                s.expert[b] = (int16_t)(tid * kEach + i);
                s.at[b] = (int16_t)(a + q);
                s.n[b] = (int16_t)(n[i] - q < TOK ? n[i] - q : TOK);
                ++b;
            }
            a += n[i];
        }
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int m = p / topk, e = by.expert[p];
        const float c = s.c[p] / s.total[m];
        s.c[p] = c;
        if (write) {
            if (ids_out) ids_out[p] = e;
            if (weights_out) weights_out[p] = c;
        }
        if (more) s.pair_of[by.pairs_at[e] + __popcll(by.tokens[e] & ((1ull << m) - 1))] = (int16_t)p;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(passes);
}

// c times token t's sum v of a pass into the wave's rows [M][16].
__device__ __forceinline__ void moe_add(const Passes& s, int n, int at, int t, int topk, float v, float* sums) {
    if (t >= n) return;
    const int p = s.pair_of[at + t];
    float& to = sums[p / topk * 16 + (threadIdx.x & 15)];
    to = __builtin_fmaf(s.c[p], v, to);
}

// y[m,n] by the definition, for what is not finite otherwise.
template <class T, int GPU, bool ZP>
__device__ __forceinline__ float moe_defined(const Passes& s, const uint16_t* h, int F, const uint8_t* wd,
                                             const W4gLayout& l, const int32_t* ids, int topk, int m, int n) {
    double y = 0.0;
    for (int p = m * topk; p < (m + 1) * topk && y == y; ++p) {
        const double c = s.c[p];
        if (c == c)   // a NaN of the softmax needs no sum
            y += c * w4g_defined<T, GPU, ZP>(wd + (size_t)ids[p] * l.total, l, n, F, [&](int k, float (&v)[8]) {
                const uint16_t* hp = h + (size_t)p * kParts * F + k;
                w4g_values<Bf16>(hp, v);
#pragma unroll
                for (int i = 1; i < kParts; ++i) {
                    float part[8];
                    w4g_values<Bf16>(hp + (size_t)i * F, part);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += part[j];
                }
            });
        else
            y = c;
    }
    return (float)y;
}

// Columns C blockIdx.x.. of y: 16 times this block's sums value(m, column) and,
// where more blocks share the columns, theirs; defined(m, n) where that is not
// finite.
template <class T, int WAVES, int C, class V, class D>
__device__ __forceinline__ void moe_finish(Passes& s, int M, int N, uint32_t* arrived, float* parts, uint16_t* y,
                                           V value, D defined) {
    constexpr int kThreads = 64 * WAVES;
    const int tid = threadIdx.x, splits = gridDim.y;
    for (int i = tid; i < M * C; i += kThreads) {
        const int m = i / C;
        const size_t n = (size_t)blockIdx.x * C + i % C;
        if (n >= (size_t)N) continue;
        const float v = value(m, i % C);
        if (splits == 1)
            y[(size_t)m * N + n] = T::from_f32(w4g_finite(16.0f * v) ? 16.0f * v : defined(m, (int)n));
        else
            __hip_atomic_store(&parts[((size_t)blockIdx.y * M + m) * N + n], v, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (splits == 1) return;
    w4g_wait();   // this wave's sums are where every block reads them
    __syncthreads();
    if (tid == 0)
        s.before = __hip_atomic_fetch_add(&arrived[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (s.before + 1 != (uint32_t)splits) return;
    for (int i = tid; i < M * C; i += kThreads) {
        const int m = i / C;
        const size_t n = (size_t)blockIdx.x * C + i % C;
        if (n >= (size_t)N) continue;
        // all under way at once: each comes from beyond the L2
        float part[kMaxSplits], v = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxSplits; ++j)
            part[j] = __hip_atomic_load(&parts[((size_t)(j < splits ? j : 0) * M + m) * N + n], __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int j = 0; j < kMaxSplits; ++j) v += j < splits ? part[j] : 0.0f;
        y[(size_t)m * N + n] = T::from_f32(w4g_finite(16.0f * v) ? 16.0f * v : defined(m, (int)n));
    }
}

template <class T, int GPU, bool ZP>
__global__ __launch_bounds__(64 * kDownWaves, 4) void k_moe_down(
    const uint16_t* __restrict__ h, int M, int F, int N, const uint8_t* __restrict__ wd, int E, int topk, int norm,
    const double* __restrict__ logits, const int32_t* __restrict__ ids, const double* __restrict__ top,
    uint32_t* __restrict__ arrived,
    float* __restrict__ parts, uint16_t* __restrict__ y, int32_t* __restrict__ ids_out,
    float* __restrict__ weights_out) {
    // one tile of 16 columns a block, the items shared out to its waves, each
    // with rows of its own
    constexpr int kThreads = 64 * kDownWaves;
    extern __shared__ __attribute__((aligned(16))) float sums[];   // [waves][M][16]
    __shared__ Passes s;
    constexpr int kFills = 4;
    static_assert(kParts * kDownTok == 4 * kFills - 1, "one operand, a row left over");
    __shared__ __attribute__((aligned(16))) char rows_lds[kDownWaves][kFills * 1024];
    static_assert(sizeof(ByExpert) <= sizeof(rows_lds), "the rows' place holds it");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int i = tid; i < kDownWaves * M * 16; i += kThreads) sums[i] = 0.0f;
    const int passes = moe_passes<kDownWaves, kDownTok, true>(s, *reinterpret_cast<ByExpert*>(rows_lds), M, E, topk, norm,
                                                        logits, ids, top, blockIdx.x == 0 && blockIdx.y == 0, ids_out,
                                                        weights_out);

    const W4gLayout l = w4g_layout(128 / GPU, ZP, N, F);
    const int tile = blockIdx.x, split = blockIdx.y, splits = gridDim.y;
    const v4i hb = w4g_rows(h, kParts * M * topk, F);
    const int items = passes * l.units, run = (items + kDownWaves * splits - 1) / (kDownWaves * splits);
    const int begin = (split * kDownWaves + wave) * run, end = begin + run < items ? begin + run : items;
    const char* my_rows = rows_lds[wave];
    const uint32_t my_lds = lds_address(my_rows);
    // operand rows 4 t..4 t + 2 are the parts of token t < 4, so that their sums
    // lie in one lane, rows 3, 7 and 11 those of token 4
    const int quad = (lane >> 2) & 3, my_row = (lane & 3) < 3 ? 3 * quad + (lane & 3) : 12 + quad;
    // the next item to load: its pass, its unit, and what changes with the pass
    int pass = begin / l.units, u = begin % l.units, fills = 0;
    const uint8_t* we = wd;
    uint32_t row[kFills];
    W4gUnit<GPU> next[1];
    auto turn = [&]() {
        const int n = __builtin_amdgcn_readfirstlane(s.n[pass]), at = s.at[pass];
        we = wd + (size_t)__builtin_amdgcn_readfirstlane(s.expert[pass]) * l.total;
        fills = (kParts * n + 3) >> 2;
#pragma unroll
        for (int j = 0; j < kFills; ++j) {
            const int r = 4 * j + (lane >> 4), t = r / kParts < n ? r / kParts : n - 1;
            row[j] = (uint32_t)(kParts * s.pair_of[at + t] + r % kParts) * (2u * F);
        }
    };
    auto load = [&]() {
        next[0] = w4g_load<GPU, ZP>(we, l, (size_t)tile * l.units + u, lane);
#pragma unroll
        for (int j = 0; j < kFills; ++j)
            if (j < fills) w4g_x_to_lds(hb, row[j] + w4g_chunk(4 * j, u, F, lane), my_lds + j * 1024);
    };
    if (begin < end) {
        turn();
        load();
    }

    f32x4 acc[1][1] = {{f32x4{0, 0, 0, 0}}};
    for (int i = begin; i < end; ++i) {
        w4g_wait();
        const W4gUnit<GPU> w[1] = {next[0]};
        u32x4 a[GPU][1][4 / GPU];
#pragma unroll
        for (int d = 0; d < 4; ++d) a[d / (4 / GPU)][0][d % (4 / GPU)] = w4g_operand_row(my_rows, my_row, d, lane);
        w4g_wait_lds();
        const int done = pass;
        if (++u == l.units) {
            u = 0;
            ++pass;
        }
        if (i + 1 < end) {
            if (pass != done) turn();
            load();
        }
#pragma unroll
        for (int g = 0; g < GPU; ++g) w4g_mac<DownT<T>, GPU, ZP, 1, 1>(g, w, a[g], acc);
        if (i + 1 == end || pass != done) {
            f32x4& v = acc[0][0];
            const int n = s.n[done], at = s.at[done];
            const float last = v[3] + __shfl_down(v[3], 16) + __shfl_down(v[3], 32);
            moe_add(s, n, at, lane >> 4, topk, v[0] + v[1] + v[2], sums + wave * M * 16);
            if (lane < 16) moe_add(s, n, at, 4, topk, last, sums + wave * M * 16);
            v = f32x4{0, 0, 0, 0};
        }
    }
    __syncthreads();
    moe_finish<T, kDownWaves, 16>(s, M, N, arrived, parts, y, [&](int m, int n) {
        float v = 0.0f;
#pragma unroll
        for (int wv = 0; wv < kDownWaves; ++wv) v += sums[(wv * M + m) * 16 + n];
        return v;
    }, [&](int m, int n) { return moe_defined<T, GPU, ZP>(s, h, F, wd, l, ids, topk, m, n); });
}

// The same with kWideTiles tiles of 16 columns a block, whose waves go through
// the same items together, so that the rows of h are brought once for all of
// them; kWideGroups such groups of waves a block, each with its share of the
// items; passes of up to kWideTok tokens, an operand of 16 rows for each part.
// The rows are taken to registers before the next item's are brought to the
// same place, which leaves room for two blocks on a CU: with two places and
// one block 73 us where this takes 56.5.
template <class T, int GPU, bool ZP>
__global__ __launch_bounds__(64 * kDownWaves, 4) void k_moe_down_wide(
    const uint16_t* __restrict__ h, int M, int F, int N, const uint8_t* __restrict__ wd, int E, int topk, int norm,
    const double* __restrict__ logits, const int32_t* __restrict__ ids, const double* __restrict__ top,
    uint32_t* __restrict__ arrived,
    float* __restrict__ parts, uint16_t* __restrict__ y, int32_t* __restrict__ ids_out,
    float* __restrict__ weights_out) {
    constexpr int kThreads = 64 * kDownWaves, kFills = kParts * kWideTok / 4, kRows = kFills * 1024,
                  kMine = kFills / kWideTiles;
    static_assert(kWideTok == 16 && kFills % kWideTiles == 0, "an operand a part, the waves share the fills evenly");
    extern __shared__ __attribute__((aligned(16))) float sums[];   // [waves][M][16]
    __shared__ Passes s;
    __shared__ __attribute__((aligned(16))) char rows_lds[kWideGroups * kRows];
    static_assert(sizeof(ByExpert) <= sizeof(rows_lds), "the rows' place holds it");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = wave / kWideTiles, wn = wave % kWideTiles;
    for (int i = tid; i < kDownWaves * M * 16; i += kThreads) sums[i] = 0.0f;
    const int passes = moe_passes<kDownWaves, kWideTok, false>(s, *reinterpret_cast<ByExpert*>(rows_lds), M, E, topk, norm,
                                                        logits, ids, top, blockIdx.x == 0 && blockIdx.y == 0, ids_out,
                                                        weights_out);

    const W4gLayout l = w4g_layout(128 / GPU, ZP, N, F);
    const int tile = blockIdx.x * kWideTiles + wn, mine = tile < l.tiles ? tile : l.tiles - 1;
    const int split = blockIdx.y, splits = gridDim.y;
    const v4i hb = w4g_rows(h, kParts * M * topk, F);
    const int items = passes * l.units, run = (items + kWideGroups * splits - 1) / (kWideGroups * splits);
    const int begin = (split * kWideGroups + group) * run, end = begin + run < items ? begin + run : items;
    const char* my_rows = rows_lds + group * kRows;
    const uint32_t my_lds = lds_address(my_rows);
    int pass = begin / l.units, u = begin % l.units, n = 0;
    const uint8_t* we = wd;
    uint32_t row[kMine];   // of this wave's instructions wn, wn + kWideTiles..
    W4gUnit<GPU> next[1];
    auto turn = [&]() {
        n = __builtin_amdgcn_readfirstlane(s.n[pass]);
        const int at = s.at[pass];
        we = wd + (size_t)__builtin_amdgcn_readfirstlane(s.expert[pass]) * l.total;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int r = 4 * (i * kWideTiles + wn) + (lane >> 4), p = r / kWideTok, t = r % kWideTok;
            row[i] = (uint32_t)(kParts * s.pair_of[at + (t < n ? t : n - 1)] + p) * (2u * F);
        }
    };
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int j = i * kWideTiles + wn;
            if (4 * j % kWideTok < n) w4g_x_to_lds(hb, row[i] + w4g_chunk(4 * j, u, F, lane), my_lds + j * 1024);
        }
        next[0] = w4g_load<GPU, ZP>(we, l, (size_t)mine * l.units + u, lane);
    };
    if (begin < end) {
        turn();
        load();
    }

    f32x4 acc[1][1] = {{f32x4{0, 0, 0, 0}}};
    for (int i = begin; i < begin + run; ++i) {   // as many turns for every wave: they meet in each
        w4g_wait();
        w4g_barrier();   // the item's rows are there
        const W4gUnit<GPU> w[1] = {next[0]};
        u32x4 a[GPU][1][kParts * (4 / GPU)];
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                a[d / (4 / GPU)][0][p * (4 / GPU) + d % (4 / GPU)] = w4g_operand_rows(my_rows + p * 4096, d, lane);
        w4g_barrier();   // and have been read
        if (i >= end) continue;
        const int done = pass;
        if (++u == l.units) {
            u = 0;
            ++pass;
        }
        if (i + 1 < end) {
            if (pass != done) turn();
            load();
        }
#pragma unroll
        for (int g = 0; g < GPU; ++g) w4g_mac<DownT<T>, GPU, ZP, 1, 1, kParts>(g, w, a[g], acc);
        if (i + 1 == end || pass != done) {
            f32x4& v = acc[0][0];
            const int n_done = s.n[done], at = s.at[done];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                moe_add(s, n_done, at, (lane >> 4) * 4 + t, topk, v[t], sums + wave * M * 16);
            v = f32x4{0, 0, 0, 0};
        }
    }
    __syncthreads();
    moe_finish<T, kDownWaves, 16 * kWideTiles>(s, M, N, arrived, parts, y, [&](int m, int c) {
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < kWideGroups; ++g) v += sums[((g * kWideTiles + (c >> 4)) * M + m) * 16 + (c & 15)];
        return v;
    }, [&](int m, int n) { return moe_defined<T, GPU, ZP>(s, h, F, wd, l, ids, topk, m, n); });
}

template <class T, int GPU, bool ZP>
hipError_t moe_t(const MoeArgs& a, const MoeWs& l, int M, const uint16_t* x, uint16_t* y, int32_t* ids,
                 float* weights, hipStream_t st) {
    char* ws = static_cast<char*>(a.ws);
    double* logits = reinterpret_cast<double*>(ws + l.logits);
    int32_t* ids_ws = reinterpret_cast<int32_t*>(ws + l.ids);
    uint16_t* h = reinterpret_cast<uint16_t*>(ws + l.h);
    double* top = reinterpret_cast<double*>(ws + l.top);
    const DownGrid grid = down_grid(M, a.F, a.K, a.E, a.topk);
    static std::atomic<uint64_t> done[2];
    const auto down = grid.wide ? k_moe_down_wide<T, GPU, ZP> : k_moe_down<T, GPU, ZP>;
    const hipError_t err =
        opt_in_lds(reinterpret_cast<const void*>(down), kDownWaves * kChunk * 64, done[grid.wide]);
    if (err != hipSuccess) return err;
    uint32_t* arrived = reinterpret_cast<uint32_t*>(ws + l.arrived);
    float* parts = reinterpret_cast<float*>(ws + l.parts);
    k_moe_logits<T><<<dim3((a.E + 3) / 4, M), 256, 0, st>>>(x, a.K, a.router, a.E, logits, arrived,
                                                            grid.splits > 1 ? grid.columns : 0);
    const int pairs = M * a.topk, by_pair = pairs < a.E, rows = by_pair ? pairs : a.E;
    // waves that share a tile's K: as many as give the chip's 1024 SIMDs one
    // each, and further up to its 4096 wave slots while each keeps 8 units; us,
    // by waves a tile (units of a wave): 8 x 48 tiles 4 (4) 9.9, 8 (2) 10.5;
    // 16 x 48 tiles 2 (8) 13.3, 4 (4) 13.8, 8 (2) 17.3; 20 x 88 tiles 1 (11)
    // 15.4, 4 (2.8) 20; 8 x 352 tiles 1 (32) 48, 2 (16) 42.7
    const int tiles = a.F / 16, units = (a.K + 127) / 128;
    int ks_log2 = 0;
    for (; (1 << ks_log2) < kUpWaves; ++ks_log2) {
        const long waves = (long)rows * tiles << ks_log2;
        if (waves >= 1024 && (waves >= 4096 || units >> (ks_log2 + 1) < 8)) break;
    }
    const int per = kUpWaves >> ks_log2;
    // its blocks of kManyWaves tiles take K whole: every CU has to have one (us,
    // apart / shared: 256 blocks 20.5 / 19.6, 224 blocks 28 / 31)
    if (share_rows(M, a.E, a.topk) && (long)rows * ((tiles + kManyWaves - 1) / kManyWaves) >= 256)
        k_moe_gate_up_many<T, GPU, ZP><<<dim3((tiles + kManyWaves - 1) / kManyWaves, rows), 64 * kManyWaves, 0, st>>>(
            x, M, a.K, a.F, a.wg, a.wu, a.E, a.topk, logits, ids_ws, top, h);
    else
        k_moe_gate_up<T, GPU, ZP><<<dim3((tiles + per - 1) / per, rows), 64 * kUpWaves, 0, st>>>(
            x, M, a.K, a.F, a.wg, a.wu, a.E, a.topk, by_pair, ks_log2, logits, ids_ws, top, h);
    down<<<dim3(grid.columns, grid.splits), 64 * kDownWaves, kDownWaves * M * 64, st>>>(
        h, M, a.F, a.K, a.wd, a.E, a.topk, a.norm, logits, ids_ws, top, arrived, parts, y, ids, weights);
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

size_t moe_workspace(int M, int K, int F, int E, int topk) { return moe_ws(M, K, F, E, topk).total; }

hipError_t launch_moe(const MoeArgs& a, hipStream_t st) {
    const MoeWs l = moe_ws(a.M, a.K, a.F, a.E, a.topk);
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
