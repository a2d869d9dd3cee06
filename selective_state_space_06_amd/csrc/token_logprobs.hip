// token_logprobs.hip -- log probabilities of given tokens under the softmax of their logits, the rows' entropies and most
// probable tokens, and the gradient to the logits, for gfx950.
//
// Forward: with m the greatest logit, s = sum e^(x - m) and t = sum e^(x - m) (x - m), the log probability of a token
// is (x_token - m) - log s and the entropy log s - t / s.  One pass: every lane keeps its own m, s and t, rescaled
// when its m rises; lanes, waves and, where a row is cut into slices, blocks are joined in 64 bits.  The alternatives come
// from the lanes' greatest logits: they bound the k-th greatest of the block from below, so that only the few lanes whose
// own greatest is not under the bound have their tiles read again (from the L2 cache).  Lists of 64-bit keys are merged
// pairwise.  Backward: with p = e^(x - m) / s,
//     dx_v = g (1[v = token] - p_v) - h p_v (log p_v + entropy),
// one pass over the logits from the row's m, 1 / s and entropy - log s.
//
// e^d is exp2 of d log2 e as it is rounded, about |d| roundings off, where nothing sees that: in the sums, whose terms e^d / s
// weigh it (it comes to 1.5 times the entropy in units of 2^-24 at most), and in gradients that are rounded to bf16.  An f32
// gradient of an improbable token is such a term alone, and has it corrected (exact_exp; the time is the same).
//
// Both are bound by memory where there is enough of it: 4096 x 50280 bf16 80 to 88 us forward (4.7 to 5.2 TB/s), 230 with the gradient
// (5.4 TB/s).  A batch of 128 x 128007 bf16 takes 14 us without alternatives (2.4 TB/s; 6.4 at the rate of a copy, the rest is
// the ends of two launches), 19 with 5 of them and 23 with 20; as lists kept by every wave along its way 14, 23 and 39.  One row
// of 50277 f32 with 20 alternatives takes 14 us, mostly latencies in a row: launches, loads, merges.
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

// The k greatest of two sorted lists, `other` held the other way round (entry j in lane size - 1 - j): the greater of each
// pair of entries, which rises and falls, sorted by comparing lanes ever closer to each other.  size: list_size(k).
__device__ __forceinline__ int list_size(int k) { return k > 1 ? 1 << (32 - __builtin_clz(k - 1)) : 1; }
template <int X>
__device__ __forceinline__ uint32_t across(uint32_t v) {  // v of the lane X away
    const int i = static_cast<int>(v);
    if (X == 1) return __builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, true);   // quad_perm 1 0 3 2
    if (X == 2) return __builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, true);   // quad_perm 2 3 0 1
    if (X == 4)                                                                   // row_half_mirror, quad_perm 3 2 1 0
        return __builtin_amdgcn_update_dpp(0, __builtin_amdgcn_update_dpp(0, i, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true);
    if (X == 8) return __builtin_amdgcn_update_dpp(0, i, 0x128, 0xF, 0xF, true);  // row_ror 8
    if (X == 16) return __builtin_amdgcn_ds_swizzle(i, 16 << 10 | 0x1F);
    return __shfl_xor(i, X);
}
template <int X>
__device__ __forceinline__ void compare_across(uint64_t& key, int size, int lane) {
    if (X >= size) return;
    const uint64_t o = join64(across<X>(static_cast<uint32_t>(key >> 32)), across<X>(static_cast<uint32_t>(key)));
    key = (o > key) == ((lane & X) == 0) ? o : key;
}
__device__ __forceinline__ uint64_t merge_two(uint64_t key, uint64_t other, int size, int lane) {
    key = other > key ? other : key;
    compare_across<32>(key, size, lane);
    compare_across<16>(key, size, lane);
    compare_across<8>(key, size, lane);
    compare_across<4>(key, size, lane);
    compare_across<2>(key, size, lane);
    compare_across<1>(key, size, lane);
    return key;
}
// Joins the lists of W waves into wave 0's (lanes from k on hold kNone).  Every wave comes here.
template <int W>
__device__ __forceinline__ void join_lists(uint64_t* all, uint64_t& key, int k, int wave, int lane) {
    const int size = list_size(k);
    for (int w = W / 2; w > 0; w >>= 1) {
        if (wave >= w && wave < 2 * w && lane < size) all[wave * 64 + size - 1 - lane] = key;
        __syncthreads();
        if (wave < w) key = merge_two(key, lane < size ? all[(wave + w) * 64 + lane] : kNone, size, lane);
        if (lane >= k) key = kNone;
    }
}

// The logit of the row's token, read long before it is used.
template <class E>
__device__ __forceinline__ float logit_of_token(const LArgs& a, int64_t row) {
    const int64_t token = a.tokens[row];
    return E::load1(a.logits, row * a.V + (token >= 0 && token < a.V ? token : 0));
}

// A row's outputs by one wave; `given`: its token's logit; `key`: lane j's alternative.
__device__ __forceinline__ void finish_row(const LArgs& a, int64_t row, float given, const Sums& v, uint64_t key, int lane) {
    const bool dead = v.s == 0.0;  // every logit is -inf
    const double ls = dead ? 0.0 : log(v.s);
    const float entropy = dead ? 0.0f : static_cast<float>(ls - v.t / v.s);
    if (lane == 0) {
        const int64_t token = a.tokens[row];
        const bool in = token >= 0 && token < a.V;
        a.logprobs[row] = !in ? 0.0f : dead ? -INFINITY : static_cast<float>((static_cast<double>(given) - v.m) - ls);
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

// One block of W waves per (row, slice of the vocabulary), its waves on successive tiles in turn, kAhead of them on their way, by
// loads that are not branched around (past the end they give 0).  Which lane takes which logit does not depend on where the
// row lies, so that equal rows have equal results: rows of any alignment are loaded as they are (4096 x 50277 bf16: 101 us
// with branches, 92 without).
constexpr int kWaves = 4, kMostWaves = 16, kAhead = 2;

template <class E, bool TOP, int W>
__global__ __launch_bounds__(64 * W) void logprob_kernel(LArgs a) {
    using S = typename E::storage;
    constexpr int ES = sizeof(S);
    __shared__ uint64_t all[TOP ? W * 64 : 1];
    __shared__ double all_s[W], all_t[W];
    __shared__ float all_m[W];
    __shared__ uint32_t bars[2][W];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int64_t works = a.R * a.slices;
    for (int64_t g = blockIdx.x; g < works; g += gridDim.x) {
        const int64_t row = g / a.slices;
        const int slice = static_cast<int>(g % a.slices);
        const S* p = static_cast<const S*>(a.logits) + row * a.V;
        const int64_t tiles = (a.V + kTile - 1) / kTile, from = slice * a.tiles;
        const int64_t to = from + a.tiles < tiles ? from + a.tiles : tiles;
        float m = -INFINITY, s = 0.0f, t = 0.0f;
        Raw<E> raw[kAhead];
        const auto load = [&](int64_t k, Raw<E>& r) MSS_INLINED {
            const int rem = k < to ? clamp_tile(a.V - k * kTile) : 0;
            const bool half = ES == 2 && rem & 1;  // the last logit is half of a word, which a buffer does not hold
            const auto buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<S*>(p + k * kTile), 0, half ? 0 : rem * ES, 0x00027000);
#pragma unroll
            for (int i = 0; i < kE / E::kPerVec; ++i)
                r.q[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(buffer, lane * kE * ES + 16 * i, 0, 0));
            if (half) load8<E, false>(p + k * kTile, a.V, rem, lane, r);
        };
        const auto take = [&](const float* v) MSS_INLINED {
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
        };
        const auto tile = [&](int64_t k, Raw<E>& r) MSS_INLINED {
            const int rem = clamp_tile(a.V - k * kTile);
            if (ES == 2 && rem & 1) settle8<E, false>(a.V, rem, lane, r);
            float v[kE];
            r.unpack(v);
            load(k + kAhead * W, r);
            if (k >= to) return;
            if (rem < kTile) {
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if (lane * kE + e >= rem) v[e] = -INFINITY;
            }
            take(v);
        };
        const int64_t lo = from + wave;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(lo + i * W, raw[i]);
        const float given = a.slices == 1 && wave == 0 ? logit_of_token<E>(a, row) : 0.0f;
        for (int64_t k = lo; k < to; k += kAhead * W) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) tile(k + i * W, raw[i]);
        }
        uint64_t key = kNone;
        if constexpr (TOP) {
            // the alternatives are at least as great as the k-th greatest of any wave's lanes, and as the least of the
            // waves' (k / W)-th greatest
            const uint32_t most = order_of(m);
            const int share = (a.K + W - 1) / W;
            uint32_t kth = 0, part = 0;
#pragma unroll
            for (int bit = 31; bit >= 16; --bit) {
                const uint32_t c = kth | 1u << bit, d = part | 1u << bit;
                if (__popcll(ballot(most >= c)) >= a.K) kth = c;
                if (__popcll(ballot(most >= d)) >= share) part = d;
            }
            if (lane == 0) bars[0][wave] = kth, bars[1][wave] = part;
            __syncthreads();
            uint32_t bar = kLeast;
            {
                uint32_t least = ~0u;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    bar = bars[0][w] > bar ? bars[0][w] : bar;
                    least = bars[1][w] < least ? bars[1][w] : least;
                }
                bar = least > bar ? least : bar;
            }
            List list;
            const auto offer = [&](uint32_t o, int token) MSS_INLINED {
                const uint64_t k = key_of(o, token);
                uint64_t left = ballot((o >= bar) & (k > list.last));
                while (left) {
                    list.insert(lane_of(k, first_of(left)), a.K, lane);
                    left &= left - 1;
                    left &= ballot(k > list.last);
                }
            };
            // the tiles of the lanes that have such logits again, 64 vectors of them at a time
            const int mine = lo < to ? static_cast<int>((to - lo + W - 1) / W) : 0;
            int lg = 0;
            while (lg < 6 && 1 << lg < mine) ++lg;
            const int first_token = static_cast<int>(lo * kTile);
            uint64_t hot = ballot(mine > 0 && most >= bar);
            while (hot) {
                const int rank = __popcll(hot & ((1ull << lane) - 1)), count = __popcll(hot);
                const int order = __builtin_amdgcn_ds_permute(4 * (hot >> lane & 1 ? rank : count + lane - rank), lane);
                const int src = __shfl(order, lane >> lg);
                for (int base = 0; base < mine; base += 64) {
                    const int i = base + (lane & ((1 << lg) - 1));
                    const int64_t at = (lo + static_cast<int64_t>(i) * W) * kTile + src * kE;
                    const bool in = lane >> lg < count && i < mine;
                    const int n = !in || at >= a.V ? 0 : a.V - at < kE ? static_cast<int>(a.V - at) : kE;  // of this lane's
                    float v[kE];
                    if (n == kE) {
                        Raw<E> r;
                        __builtin_memcpy(r.q, p + at, sizeof(r.q));
                        r.unpack(v);
                    } else {
#pragma unroll
                        for (int e = 0; e < kE; ++e) v[e] = e < n ? E::load1(p, at + e) : 0.0f;
                    }
#pragma unroll
                    for (int e = 0; e < kE; ++e) v[e] = e < n && v[e] == v[e] ? v[e] : -INFINITY;
#pragma unroll
                    for (int e = 0; e < kE; ++e) offer(order_of(v[e]), static_cast<int>(at) + e);
                }
                // those that were not taken, if they still can be among the k best
                for (int i = 0; i < 64 >> lg && hot; ++i) hot &= hot - 1;
                hot &= ballot(key_of(most, first_token + lane * kE) > list.last);
            }
            if (lane < a.K) key = list.key;
        }
        Sums v{m, s, t};
        join_lanes(v, 64);
        if (lane == 0) {
            all_m[wave] = v.m;
            all_s[wave] = v.s;
            all_t[wave] = v.t;
        }
        if (TOP) join_lists<W>(all, key, a.K, wave, lane);
        else __syncthreads();
        if (wave == 0) {
            v = lane < W ? Sums{all_m[lane], all_s[lane], all_t[lane]} : Sums{-INFINITY, 0.0, 0.0};
            join_lanes(v, W);
            if (a.slices == 1) {
                finish_row(a, row, given, v, key, lane);
            } else {
                if (lane == 0) {
                    a.part_m[g] = v.m;
                    a.part_s[g] = v.s;
                    a.part_t[g] = v.t;
                }
                if (lane < a.K) a.cand[g * a.K + lane] = key;
            }
        }
        __syncthreads();
    }
}

// Joins the slices of a row: a block of kWaves waves, of which each takes every kWaves-th list.
template <class E>
__global__ __launch_bounds__(64 * kWaves) void logprob_join_kernel(LArgs a) {
    __shared__ uint64_t all[kWaves * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
        Sums v{-INFINITY, 0.0, 0.0};
        float given = 0.0f;
        if (wave == 0) {
            given = logit_of_token<E>(a, row);
            if (lane < a.slices) v = Sums{a.part_m[row * a.slices + lane], a.part_s[row * a.slices + lane],
                                          a.part_t[row * a.slices + lane]};
        }
        uint64_t key = kNone;
        if (a.K > 0) {
            const int size = list_size(a.K), j = size - 1 - lane;
            const uint64_t* lists = a.cand + row * a.slices * a.K + j;
            constexpr int G = 4;  // lists on their way
            for (int i0 = wave; i0 < a.slices; i0 += G * kWaves) {
                uint64_t other[G];
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const int l = i0 + i * kWaves;
                    other[i] = l < a.slices && j >= 0 && j < a.K ? lists[l * a.K] : kNone;
                }
#pragma unroll
                for (int i = 0; i < G; ++i)
                    if (i0 + i * kWaves < a.slices) key = merge_two(key, other[i], size, lane);
            }
            join_lists<kWaves>(all, key, a.K, wave, lane);
        }
        if (wave == 0) {
            join_lanes(v, 64);
            finish_row(a, row, given, v, key, lane);
        }
        __syncthreads();
    }
}

// A row to a block of 16 waves where rows are no more than CUs and a wave has at most eight tiles: one launch, without scratch
// (128 x 32000 f32 with 20 alternatives: 14.4 us, 16.5 in slices; 16 x 32000 13.8 and 13.1, 1 x 50277 13.8 and 13.0, where the
// second launch, 5 us of the caller's time, costs more; 400 x 5000 23 and 16).
// Otherwise four blocks of four waves for every CU, each wave with two tiles or more (one row of 50277 f32 with 20
// alternatives: one tile 13.5 us, two 12.9); at most 64 slices.  (128 x 128007 bf16 with 5 alternatives: two blocks for every
// CU 19 us, four 18, eight 22; blocks of eight waves 19.)
void plan_logprob(int64_t R, int64_t V, int64_t* per, int* slices, int* waves) {
    const int64_t tiles = (V + kTile - 1) / kTile;
    *waves = kWaves;
    if (R <= 256 && tiles > 2 * kWaves && tiles <= 8 * kMostWaves) {
        *per = tiles;
        *slices = 1;
        *waves = kMostWaves;
        return;
    }
    int64_t n = (1024 + R - 1) / R;
    n = std::max<int64_t>(1, std::min({n, (tiles + 2 * kWaves - 1) / (2 * kWaves), int64_t{64}}));
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
// From so many bytes of logits on, theirs and their gradients' fill the 256 MB Infinity Cache: both pass it by, and what the
// forward left of the logits there is found (forward and gradients of 4096 x 50280 bf16 273 -> 232 us, 8192 x 8192 85 -> 78).
// Smaller gradients stay for who reads them next.
constexpr int64_t kPassBy = int64_t{1} << 27;

// VEC: rows are whole aligned 16-byte vectors.  PASS: kPassBy, with VEC.
template <class E, bool VEC, bool PASS>
__global__ __launch_bounds__(64 * kBwdWaves) void logprob_bwd_kernel(LBArgs a) {
    using S = typename E::storage;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
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
            const int rem = clamp_tile(a.V - k * kTile);
            if constexpr (PASS) {
                const auto buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<S*>(p + k * kTile), 0,
                                                                      rem * static_cast<int>(sizeof(S)), 0x00027000);
#pragma unroll
                for (int i = 0; i < kE / E::kPerVec; ++i)
                    r.q[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                           buffer, lane * kE * static_cast<int>(sizeof(S)) + 16 * i, 0, 2));
            } else {
                load8<E, VEC>(p + k * kTile, a.V, rem, lane, r);
            }
        };
        const auto tile = [&](int64_t k, Raw<E>& r) MSS_INLINED {
            const int rem = clamp_tile(a.V - k * kTile);
            settle8<E, VEC>(a.V, rem, lane, r);
            float v[kE];
            r.unpack(v);
            if (k + 2 * kBwdWaves < to) load(k + 2 * kBwdWaves, r);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                float d = v[e] - m, q;
                if constexpr (sizeof(S) == 4) {
                    d = d < kFar ? kFar : d;  // (a NaN stays one)
                    q = exact_exp(d) * inv;
                } else {
                    q = fast_exp2(d * kLog2e) * inv;
                    d = fmaxf(d, kFar);
                }
                v[e] = -q * fmaf(h, d + c, g);
            }
            const int64_t mine = token - k * kTile - lane * kE;
            if (mine >= 0 && mine < kE) {
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if (e == mine) v[e] += g;
            }
            if constexpr (PASS) {
#pragma unroll
                for (int j = 0; j < kE / E::kPerVec; ++j) {
                    const int at = lane * kE + j * E::kPerVec;
                    const uint4 w = E::pack(v + j * E::kPerVec);
                    if (at < rem) __builtin_nontemporal_store(u32x4{w.x, w.y, w.z, w.w}, reinterpret_cast<u32x4*>(o + k * kTile + at));
                }
            } else {
                store8<E, VEC>(o + k * kTile, rem, lane, v);
            }
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
    int slices, waves;
    plan_logprob(R, V, &per, &slices, &waves);
    return slices == 1 ? 0 : R * slices * (5 + 2 * K);
}

hipError_t launch_logprob_fwd(const LogprobLaunch& l, hipStream_t s) {
    LArgs a{};
    a.logits = l.logits; a.tokens = l.tokens; a.logprobs = l.logprobs; a.entropy = l.entropy;
    a.top_logprobs = l.top_logprobs; a.top_tokens = l.top_tokens; a.saved = l.saved;
    a.R = l.R; a.V = l.V; a.K = l.K;
    int waves;
    plan_logprob(l.R, l.V, &a.tiles, &a.slices, &waves);
    const int64_t works = l.R * a.slices;
    a.part_s = reinterpret_cast<double*>(l.scratch);
    a.part_t = a.part_s + works;
    a.cand = reinterpret_cast<uint64_t*>(a.part_t + works);
    a.part_m = reinterpret_cast<float*>(a.cand + works * l.K);
    const dim3 grid(blocks_for(works, 1)), block(64 * kWaves);
    const auto go = [&](auto e) {
        using E = decltype(e);
        const dim3 wide(64 * kMostWaves);
        if (l.K) {
            if (waves == kWaves) logprob_kernel<E, true, kWaves><<<grid, block, 0, s>>>(a);
            else logprob_kernel<E, true, kMostWaves><<<grid, wide, 0, s>>>(a);
        } else {
            if (waves == kWaves) logprob_kernel<E, false, kWaves><<<grid, block, 0, s>>>(a);
            else logprob_kernel<E, false, kMostWaves><<<grid, wide, 0, s>>>(a);
        }
    };
    if (l.bf16) go(BF16{});
    else go(F32{});
    if (a.slices > 1) {
        const dim3 rows(blocks_for(l.R, 1));
        if (l.bf16) logprob_join_kernel<BF16><<<rows, block, 0, s>>>(a);
        else logprob_join_kernel<F32><<<rows, block, 0, s>>>(a);
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
    const bool pass = l.vec_ok && l.R * l.V * (l.bf16 ? 2 : 4) >= kPassBy;
    if (l.bf16) {
        if (pass) logprob_bwd_kernel<BF16, true, true><<<grid, block, 0, s>>>(a);
        else if (l.vec_ok) logprob_bwd_kernel<BF16, true, false><<<grid, block, 0, s>>>(a);
        else logprob_bwd_kernel<BF16, false, false><<<grid, block, 0, s>>>(a);
    } else {
        if (pass) logprob_bwd_kernel<F32, true, true><<<grid, block, 0, s>>>(a);
        else if (l.vec_ok) logprob_bwd_kernel<F32, true, false><<<grid, block, 0, s>>>(a);
        else logprob_bwd_kernel<F32, false, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mss
