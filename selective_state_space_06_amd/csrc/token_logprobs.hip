// token_logprobs.hip -- log probabilities of given tokens under the softmax of their logits, the rows' entropies and most
// probable tokens, and the gradient to the logits, for gfx950.
//
// Forward: with m the greatest logit, s = sum e^(x - m) and t = sum e^(x - m) (x - m), the log probability of a token
// is (x_token - m) - log s and the entropy log s - t / s.  One pass: every lane keeps its own m, s and t, rescaled
// when its m rises, and a wave its list of the k greatest logits (top_lists.hpp); lanes, waves and, where a row is
// cut into slices, blocks are joined in 64 bits.  Backward: with p = e^(x - m) / s,
//     dx_v = g (1[v = token] - p_v) - h p_v (log p_v + entropy),
// one pass over the logits from the row's m, 1 / s and entropy - log s.  Both are bound by memory.
#include <algorithm>

#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"
#include "top_lists.hpp"

namespace mss {
namespace {

struct LArgs {
    const void* logits;     // (R, V)
    const int32_t* tokens;  // (R)
    float* logprobs;        // (R)
    float* entropy;         // (R), nullable
    float* top_logprobs;    // (R, K)
    int32_t* top_tokens;
    float* saved;           // (R, 3), nullable
    double* part_s;         // (R, slices)
    double* part_t;
    uint64_t* cand;         // (R, slices, K)
    float* part_m;          // (R, slices)
    int64_t R, V;
    int64_t tiles;          // per slice
    int K, slices;
};

// (x - m) where it stands in a product with e^(x - m): bounded, so that a masked logit adds 0 and no NaN.  e^-200 is
// far under fp32's range.
constexpr float kFar = -200.0f;

struct Sums {  // of some logits: the greatest (-inf: none), sum of e^(x - m), sum of e^(x - m) (x - m)
    float m;
    double s, t;
    // the same in terms of a greater m
    __device__ __forceinline__ void lift(float top) {
        if (s == s && !(m > -INFINITY)) {
            s = t = 0.0;
        } else {
            const float d = fmaxf(m - top, kFar);
            const double f = fast_exp2(d * kLog2e);
            t = f * (t + s * d);
            s *= f;
        }
        m = top;
    }
};

// Joins the sums of the first `count` lanes (a power of two), into every lane.
__device__ __forceinline__ void join_lanes(Sums& v, int count) {
    v.lift(value_of(wave_max(order_of(v.m))));
    for (int x = count / 2; x > 0; x >>= 1) {
        v.s += __shfl_xor(v.s, x);
        v.t += __shfl_xor(v.t, x);
    }
    v.s = __shfl(v.s, 0);
    v.t = __shfl(v.t, 0);
}

// A row's outputs by one wave; `key`: lane j's alternative.
template <class E>
__device__ __forceinline__ void finish_row(const LArgs& a, int64_t row, const Sums& v, uint64_t key, int lane) {
    const bool dead = v.s == 0.0;  // every logit is -inf
    const double ls = dead ? 0.0 : log(v.s);
    const float entropy = dead ? 0.0f : static_cast<float>(ls - v.t / v.s);
    if (lane == 0) {
        const int64_t token = a.tokens[row];
        float lp = 0.0f;
        if (token >= 0 && token < a.V) {
            const float x = E::load1(a.logits, row * a.V + token);
            lp = dead ? -INFINITY : static_cast<float>((static_cast<double>(x) - v.m) - ls);
        }
        a.logprobs[row] = lp;
        if (a.entropy) a.entropy[row] = entropy;
        if (a.saved) {
            float* o = a.saved + row * 3;
            o[0] = dead ? 0.0f : v.m;
            o[1] = dead ? 0.0f : static_cast<float>(1.0 / v.s);
            o[2] = dead ? 0.0f : static_cast<float>(static_cast<double>(entropy) - ls);
        }
    }
    if (lane < a.K) {
        const bool some = key > kNone;
        a.top_logprobs[row * a.K + lane] =
            some ? static_cast<float>((static_cast<double>(value_of(key >> 32)) - v.m) - ls) : -INFINITY;
        a.top_tokens[row * a.K + lane] = some ? token_of(key) : -1;
    }
}

// One block per (row, slice of the vocabulary), its waves on successive parts of the slice, each with two tiles on
// their way.  VEC: rows are whole aligned 16-byte vectors.
constexpr int kWaves = 8;

template <class E, bool VEC, bool TOP>
__global__ __launch_bounds__(64 * kWaves) void logprob_kernel(LArgs a) {
    using S = typename E::storage;
    __shared__ uint64_t all[TOP ? kWaves * kBeamMost : 1];
    __shared__ double all_s[kWaves], all_t[kWaves];
    __shared__ float all_m[kWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int64_t works = a.R * a.slices, tiles = (a.V + kTile - 1) / kTile;
    for (int64_t g = blockIdx.x; g < works; g += gridDim.x) {
        const int64_t row = g / a.slices, from = g % a.slices * a.tiles;
        const int64_t to = from + a.tiles < tiles ? from + a.tiles : tiles;
        const int64_t per = (to - from + kWaves - 1) / kWaves;
        const int64_t lo = from + wave * per, hi = lo + per < to ? lo + per : to;  // this wave's tiles
        const S* p = static_cast<const S*>(a.logits) + row * a.V;
        List list;
        float m = -INFINITY, s = 0.0f, t = 0.0f;
        Raw<E> raw[2] = {};
        const auto load = [&](int64_t k, Raw<E>& r) MSS_INLINED {
            load8<E, VEC>(p + k * kTile, a.V, clamp_tile(a.V - k * kTile), lane, r);
        };
        const auto tile = [&](int64_t k, Raw<E>& r, auto first) MSS_INLINED {
            const int rem = clamp_tile(a.V - k * kTile);
            settle8<E, VEC>(a.V, rem, lane, r);
            float v[kE];
            r.unpack(v);
            if (k + 2 < hi) load(k + 2, r);
            if (rem < kTile) {
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if (lane * kE + e >= rem) v[e] = -INFINITY;
            }
            float best = v[0];
#pragma unroll
            for (int e = 1; e < kE; ++e) best = fmaxf(best, v[e]);
            if (best > m) {
                const float d = fmaxf(m - best, kFar), f = fast_exp2(d * kLog2e);
                t = f * fmaf(s, d, t);
                s *= f;
                m = best;
            }
            const float ref = m > -INFINITY ? m : 0.0f;
            float ss = 0.0f, tt = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float d = v[e] - ref, x = fast_exp2(d * kLog2e);
                ss += x;
                tt = fmaf(x, fmaxf(d, kFar), tt);
            }
            s += ss;
            t += tt;
            if constexpr (TOP) {
                if (ss != ss) {  // a NaN logit, which is no alternative (or one of +inf)
#pragma unroll
                    for (int e = 0; e < kE; ++e) v[e] = v[e] == v[e] ? v[e] : -INFINITY;
                }
                const uint32_t most = order_of(best == best ? best : -INFINITY);
                uint32_t bar = static_cast<uint32_t>(list.last >> 32);  // nothing below it is among the k best
                if (decltype(first)::value) {
                    uint32_t cut = 0;
#pragma unroll
                    for (int bit = 31; bit >= 16; --bit) {
                        const uint32_t c = cut | 1u << bit;
                        if (__popcll(ballot(most >= c)) >= a.K) cut = c;
                    }
                    bar = cut > bar ? cut : bar;
                }
                if (ballot(most >= bar) == 0) return;
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const uint32_t o = order_of(v[e]);
                    const uint64_t key = key_of(o, static_cast<int>(k * kTile) + lane * kE + e);
                    uint64_t left = ballot((o >= bar) & (key > list.last));
                    while (left) {
                        list.insert(lane_of(key, first_of(left)), a.K, lane);
                        left &= left - 1;
                        left &= ballot(key > list.last);
                    }
                }
            }
        };
        if (lo < hi) {
            load(lo, raw[0]);
            if (lo + 1 < hi) load(lo + 1, raw[1]);
            tile(lo, raw[0], True{});
            for (int64_t k = lo + 1; k < hi; k += 2) {
                tile(k, raw[1], False{});
                if (k + 1 < hi) tile(k + 1, raw[0], False{});
            }
        }
        Sums v{m, s, t};
        join_lanes(v, 64);
        if (lane == 0) {
            all_m[wave] = v.m;
            all_s[wave] = v.s;
            all_t[wave] = v.t;
        }
        if (TOP && lane < a.K) all[wave * a.K + lane] = list.key;
        __syncthreads();
        if (wave == 0) {
            v = lane < kWaves ? Sums{all_m[lane], all_s[lane], all_t[lane]} : Sums{-INFINITY, 0.0, 0.0};
            join_lanes(v, kWaves);
            uint64_t got = kNone;
            if constexpr (TOP) got = merge_lists(all, kWaves, a.K, lane);
            if (a.slices == 1) {
                finish_row<E>(a, row, v, got, lane);
            } else {
                if (lane == 0) {
                    a.part_m[g] = v.m;
                    a.part_s[g] = v.s;
                    a.part_t[g] = v.t;
                }
                if (lane < a.K) a.cand[g * a.K + lane] = got;
            }
        }
        __syncthreads();
    }
}

// Joins the slices of a row, a wave each.  Shared memory: the lists.
template <class E>
__global__ __launch_bounds__(64) void logprob_join_kernel(LArgs a) {
    extern __shared__ uint64_t lists[];  // (slices, K)
    const int lane = threadIdx.x;
    for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
        for (int e = lane; e < a.slices * a.K; e += 64) lists[e] = a.cand[row * a.slices * a.K + e];
        Sums v{-INFINITY, 0.0, 0.0};
        if (lane < a.slices) v = Sums{a.part_m[row * a.slices + lane], a.part_s[row * a.slices + lane],
                                      a.part_t[row * a.slices + lane]};
        __syncthreads();
        join_lanes(v, 64);
        uint64_t got = kNone;
        if (a.K > 0) got = merge_lists(lists, a.slices, a.K, lane);
        finish_row<E>(a, row, v, got, lane);
        __syncthreads();
    }
}

// Blocks for every CU twice over, each wave with a tile; at most 64 slices.
void plan_logprob(int64_t R, int64_t V, int64_t* per, int* slices) {
    const int64_t tiles = (V + kTile - 1) / kTile;
    int64_t n = (512 + R - 1) / R;
    n = std::max<int64_t>(1, std::min({n, (tiles + kWaves - 1) / kWaves, int64_t{64}}));
    *per = (tiles + n - 1) / n;
    *slices = static_cast<int>((tiles + *per - 1) / *per);
}

struct LBArgs {
    const void* logits;
    const int32_t* tokens;
    const float* saved;
    const float* g;
    const float* h;    // nullable
    void* dlogits;
    int64_t R, V;
    int64_t tiles;     // per slice
    int slices;
};

constexpr int kBwdWaves = 4;

template <class E, bool VEC>
__global__ __launch_bounds__(64 * kBwdWaves) void logprob_bwd_kernel(LBArgs a) {
    using S = typename E::storage;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int64_t works = a.R * a.slices, tiles = (a.V + kTile - 1) / kTile;
    for (int64_t w = blockIdx.x; w < works; w += gridDim.x) {
        const int64_t row = w / a.slices, from = w % a.slices * a.tiles;
        const int64_t to = from + a.tiles < tiles ? from + a.tiles : tiles;
        const S* p = static_cast<const S*>(a.logits) + row * a.V;
        S* o = static_cast<S*>(a.dlogits) + row * a.V;
        const float m = a.saved[row * 3], inv = a.saved[row * 3 + 1], c = a.saved[row * 3 + 2];
        const int64_t token = a.tokens[row];
        // a token out of range has no log probability; a row without a finite logit no gradient
        const float g = token >= 0 && token < a.V && inv != 0.0f ? a.g[row] : 0.0f;
        const float h = a.h && inv != 0.0f ? a.h[row] : 0.0f;
        Raw<E> raw[2] = {};
        const auto load = [&](int64_t k, Raw<E>& r) MSS_INLINED {
            load8<E, VEC>(p + k * kTile, a.V, clamp_tile(a.V - k * kTile), lane, r);
        };
        const auto tile = [&](int64_t k, Raw<E>& r) MSS_INLINED {
            const int rem = clamp_tile(a.V - k * kTile);
            settle8<E, VEC>(a.V, rem, lane, r);
            float v[kE];
            r.unpack(v);
            if (k + 2 * kBwdWaves < to) load(k + 2 * kBwdWaves, r);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float d = v[e] - m, q = fast_exp2(d * kLog2e) * inv;
                v[e] = -q * fmaf(h, fmaxf(d, kFar) + c, g);
            }
            const int64_t mine = token - k * kTile - lane * kE;
            if (mine >= 0 && mine < kE) {
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if (e == mine) v[e] += g;
            }
            store8<E, VEC>(o + k * kTile, rem, lane, v);
        };
        const int64_t lo = from + wave;
        if (lo < to) load(lo, raw[0]);
        if (lo + kBwdWaves < to) load(lo + kBwdWaves, raw[1]);
        for (int64_t k = lo; k < to; k += 2 * kBwdWaves) {
            tile(k, raw[0]);
            if (k + kBwdWaves < to) tile(k + kBwdWaves, raw[1]);
        }
    }
}

}  // namespace

int64_t logprob_scratch(int64_t R, int64_t V, int64_t K) {
    if (R == 0) return 0;
    int64_t per;
    int slices;
    plan_logprob(R, V, &per, &slices);
    return slices == 1 ? 0 : R * slices * (5 + 2 * K);
}

hipError_t launch_logprob_fwd(const LogprobLaunch& l, hipStream_t s) {
    LArgs a{};
    a.logits = l.logits; a.tokens = l.tokens; a.logprobs = l.logprobs; a.entropy = l.entropy;
    a.top_logprobs = l.top_logprobs; a.top_tokens = l.top_tokens; a.saved = l.saved;
    a.R = l.R; a.V = l.V; a.K = l.K;
    plan_logprob(l.R, l.V, &a.tiles, &a.slices);
    const int64_t works = l.R * a.slices;
    a.part_s = reinterpret_cast<double*>(l.scratch);
    a.part_t = a.part_s + works;
    a.cand = reinterpret_cast<uint64_t*>(a.part_t + works);
    a.part_m = reinterpret_cast<float*>(a.cand + works * l.K);
    const dim3 grid(blocks_for(works, 1)), block(64 * kWaves);
#define MSS_FWD(E, VEC)                                                     \
    if (l.K) logprob_kernel<E, VEC, true><<<grid, block, 0, s>>>(a);        \
    else logprob_kernel<E, VEC, false><<<grid, block, 0, s>>>(a)
    if (l.bf16) {
        if (l.vec_ok) { MSS_FWD(BF16, true); } else { MSS_FWD(BF16, false); }
    } else {
        if (l.vec_ok) { MSS_FWD(F32, true); } else { MSS_FWD(F32, false); }
    }
#undef MSS_FWD
    if (a.slices > 1) {
        const size_t lds = static_cast<size_t>(a.slices) * a.K * 8;
        const dim3 rows(blocks_for(l.R, 1));
        if (l.bf16) logprob_join_kernel<BF16><<<rows, dim3(64), lds, s>>>(a);
        else logprob_join_kernel<F32><<<rows, dim3(64), lds, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_logprob_bwd(const LogprobBwdLaunch& l, hipStream_t s) {
    LBArgs a{};
    a.logits = l.logits; a.tokens = l.tokens; a.saved = l.saved; a.g = l.dlogprobs; a.h = l.dentropy;
    a.dlogits = l.dlogits; a.R = l.R; a.V = l.V;
    const int64_t tiles = (l.V + kTile - 1) / kTile;
    int64_t n = (2048 + l.R - 1) / l.R;  // blocks for every CU eight times over
    n = std::max<int64_t>(1, std::min(n, (tiles + kBwdWaves - 1) / kBwdWaves));
    a.tiles = (tiles + n - 1) / n;
    a.slices = static_cast<int>((tiles + a.tiles - 1) / a.tiles);
    const dim3 grid(blocks_for(l.R * a.slices, 1)), block(64 * kBwdWaves);
    if (l.bf16) {
        if (l.vec_ok) logprob_bwd_kernel<BF16, true><<<grid, block, 0, s>>>(a);
        else logprob_bwd_kernel<BF16, false><<<grid, block, 0, s>>>(a);
    } else {
        if (l.vec_ok) logprob_bwd_kernel<F32, true><<<grid, block, 0, s>>>(a);
        else logprob_bwd_kernel<F32, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mss
