// beam.hip -- beam search over a decode step's logits: the best continuations of every request's
// beams, and the beams' recurrent states put in their new order, for gfx950.
//
// Selection.  A live beam's continuation by token v scores score + logit_v - log sum exp(logits);
// a finished beam has one, its end token at its own score.  Per request the k best are kept.  A
// beam's continuations are ordered by their logits alone, so one pass over the logits gives both a
// slice's greatest logit and sum of exponentials and its k best (slices kernel); a second, small
// kernel forms the slices' scores and merges a request's lists.  Scores are formed and compared in 64
// bits, so that their own rounding (6e-7 at a score of -10) decides nothing; the normaliser in them is a sum of fp32
// exponentials, kept in fp32 by each lane and joined in 64 bits (measured 1.4e-8 to 1e-7 off), and decides
// between candidates of different beams that stand closer than that.
//
// Logits are compared as whole numbers of the same order (order_of), with the token behind them as one
// 64-bit key (a higher value, then a lower token), and kept in lists (top_lists.hpp).
#include <algorithm>

#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"
#include "top_lists.hpp"

namespace mss {
namespace {

struct SArgs {
    const void* logits;      // (Bt, N, V)
    const float* scores;     // (Bt, N)
    const int32_t* finished; // (Bt, N), nullable
    float* next_scores;      // (Bt, K)
    int32_t* parents;
    int32_t* tokens;
    int32_t* next_finished;  // nullable
    double* part_s;          // (rows, slices): sum of e^(logit - part_m)
    float* part_m;           // (rows, slices): greatest logit, -inf when there is none
    uint64_t* cand;          // (rows, slices, K): keys, best first; kNone: no entry
    int64_t Bt, V;
    int64_t tiles;           // per slice
    int N, K, slices, end;   // end: -1 for none
};

// A 64-bit score in the same way, 0 for a score that is -inf or not a number.  The merge compares these and
// no doubles: the compiler here encodes a scalar move of a 64-bit -inf as one of 0 (the literal's low
// half).  For the same reason -inf is told by its two halves.
__device__ __forceinline__ uint64_t order64_of(double s) {
    s += 0.0;
    const uint32_t hi = __double2hiint(s), lo = __double2loint(s);
    if (s != s || (hi == 0xFFF00000u && lo == 0u)) return 0;
    const uint32_t flip = static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31);
    return join64(hi ^ (flip | 0x80000000u), lo ^ flip);
}
__device__ __forceinline__ float score_of(uint64_t order) {  // of one that is not 0
    const uint32_t hi = static_cast<uint32_t>(order >> 32), lo = static_cast<uint32_t>(order);
    const uint32_t flip = static_cast<uint32_t>(~(static_cast<int32_t>(hi) >> 31));
    return static_cast<float>(__hiloint2double(static_cast<int>(hi ^ (flip | 0x80000000u)), static_cast<int>(lo ^ flip)));
}

// One block per (row, slice of the vocabulary), its waves on successive parts of the slice, each with two
// tiles on their way (64 x 8 x 128008 f32: 47 to 54 us by the card, 4.8 to 5.6 TB/s; one wave with one tile on its way
// and a list of values and tokens apart 57).  VEC: rows are whole aligned 16-byte vectors.
constexpr int kWaves = 8;

template <class E, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void beam_slices_kernel(SArgs a) {
    using S = typename E::storage;
    __shared__ uint64_t all[kWaves * kBeamMost];
    __shared__ double all_s[kWaves];
    __shared__ float all_m[kWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int64_t works = a.Bt * a.N * a.slices, tiles = (a.V + kTile - 1) / kTile;
    for (int64_t g = blockIdx.x; g < works; g += gridDim.x) {
        const int64_t row = g / a.slices, from = g % a.slices * a.tiles;
        const int64_t to = from + a.tiles < tiles ? from + a.tiles : tiles;
        const int64_t per = (to - from + kWaves - 1) / kWaves;
        const int64_t lo = from + wave * per, hi = lo + per < to ? lo + per : to;  // this wave's tiles
        const S* p = static_cast<const S*>(a.logits) + row * a.V;
        List list;
        float m = -INFINITY, s = 0.0f;  // of this lane's elements: the greatest, the sum of e^(v - m)
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
            const auto sums = [&]() MSS_INLINED {
                float best = v[0];
#pragma unroll
                for (int e = 1; e < kE; ++e) best = fmaxf(best, v[e]);
                const float up = fmaxf(m, best), ref = up > -INFINITY ? up : 0.0f;
                float t = 0.0f;
#pragma unroll
                for (int e = 0; e < kE; ++e) t += fast_exp2((v[e] - ref) * kLog2e);
                return make_float3(best, up, t);
            };
            float3 b = sums();
            if (b.z != b.z) {  // a NaN logit, which is masked (or one of +inf)
#pragma unroll
                for (int e = 0; e < kE; ++e) v[e] = v[e] == v[e] ? v[e] : -INFINITY;
                b = sums();
            }
            if (b.y > m) {
                s *= fast_exp2((m - b.y) * kLog2e);
                m = b.y;
            }
            s += b.z;
            const uint32_t most = order_of(b.x);
            uint32_t bar = static_cast<uint32_t>(list.last >> 32);  // nothing below it is among the k best
            if (decltype(first)::value) {
                uint32_t cut = 0;
#pragma unroll
                for (int bit = 31; bit >= 16; --bit) {
                    const uint32_t t = cut | 1u << bit;
                    if (__popcll(ballot(most >= t)) >= a.K) cut = t;
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
        };
        // a beam at its end or without a score has no continuation that needs its logits
        const float score = a.scores[row];
        if (lo < hi && !(a.finished && a.finished[row] != 0) && score > -INFINITY) {
            load(lo, raw[0]);
            if (lo + 1 < hi) load(lo + 1, raw[1]);
            tile(lo, raw[0], True{});
            for (int64_t k = lo + 1; k < hi; k += 2) {
                tile(k, raw[1], False{});
                if (k + 1 < hi) tile(k + 1, raw[0], False{});
            }
        }
        // the lanes' sums joined in 64 bits
        const float top = value_of(wave_max(order_of(m)));
        double sum = m > -INFINITY ? static_cast<double>(s) * fast_exp2((m - top) * kLog2e) : 0.0;
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
        if (lane == 0) {
            all_m[wave] = top;
            all_s[wave] = sum;
        }
        if (lane < a.K) all[wave * a.K + lane] = list.key;
        __syncthreads();
        if (wave == 0) {
            const float wm = lane < kWaves ? all_m[lane] : -INFINITY, most = value_of(wave_max(order_of(wm)));
            double ws = wm > -INFINITY ? all_s[lane] * fast_exp2((wm - most) * kLog2e) : 0.0;
#pragma unroll
            for (int x = kWaves / 2; x > 0; x >>= 1) ws += __shfl_xor(ws, x);
            if (lane == 0) {
                a.part_m[g] = most;
                a.part_s[g] = ws;
            }
            const uint64_t got = merge_lists(all, kWaves, a.K, lane);
            if (lane < a.K) a.cand[g * a.K + lane] = got;
        }
        __syncthreads();
    }
}

// One block per request: its waves merge the slices' lists of the beams in turn, then the first wave the
// beams' lists, a lane to each.  Shared memory: the lists.  A chain of rounds, one per key taken (16
// beams of 16 over 28 slices: 13.8 us; 19.7 with eight waves and each thread's keys fetched in turn).
constexpr int kMergeWaves = 16, kFetch = 7;  // keys on their way per thread: all of 56 KB at once
__global__ __launch_bounds__(64 * kMergeWaves) void beam_merge_kernel(SArgs a) {
    extern __shared__ uint64_t lists[];  // (N, slices, K); a beam's merged list ends up in its first
    __shared__ double scores[kBeamMost], norms[kBeamMost];
    __shared__ int done[kBeamMost];
    const int each = a.slices * a.K;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    for (int64_t b = blockIdx.x; b < a.Bt; b += gridDim.x) {
        const int all = a.N * each;
        for (int e = threadIdx.x; e < all; e += kFetch * 64 * kMergeWaves) {
            uint64_t v[kFetch];
#pragma unroll
            for (int j = 0; j < kFetch; ++j) {
                const int at = e + j * 64 * kMergeWaves;
                v[j] = a.cand[b * all + (at < all ? at : e)];
            }
#pragma unroll
            for (int j = 0; j < kFetch; ++j)
                if (e + j * 64 * kMergeWaves < all) lists[e + j * 64 * kMergeWaves] = v[j];
        }
        __syncthreads();
        for (int n = wave; n < a.N; n += kMergeWaves) {
            const int64_t row = b * a.N + n;
            const float m = lane < a.slices ? a.part_m[row * a.slices + lane] : -INFINITY;
            double sum = lane < a.slices ? a.part_s[row * a.slices + lane] : 0.0;
            const float top = value_of(wave_max(order_of(m)));
            if (a.slices > 1) {
                sum = m > -INFINITY ? sum * exp(static_cast<double>(m) - top) : 0.0;
#pragma unroll
                for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
                const uint64_t got = merge_lists(lists + n * each, a.slices, a.K, lane);
                if (lane < a.K) lists[n * each + lane] = got;
            }
            if (lane == 0) {
                scores[n] = a.scores[row];
                norms[n] = static_cast<double>(top) + log(sum);
                done[n] = a.finished && a.finished[row] != 0;
            }
        }
        __syncthreads();
        if (wave == 0) {
            // lane n: beam n's next continuation, its score as a whole number (0: none left)
            const int n = lane < a.N ? lane : 0;
            const bool over = done[n];
            int at = 0, token = 0;
            uint64_t order = 0;
            const auto next = [&]() MSS_INLINED {
                order = 0;
                if (over) {  // one continuation
                    if (at == 0) order = order64_of(scores[n]);
                    token = a.end;
                } else if (at < a.K) {
                    const uint64_t key = lists[n * each + at];
                    if (key > kNone)
                        order = order64_of(scores[n] + (static_cast<double>(value_of(key >> 32)) - norms[n]));
                    token = token_of(key);
                }
            };
            if (lane < a.N) next();
            for (int j = 0; j < a.K; ++j) {
                const uint32_t hi = static_cast<uint32_t>(order >> 32), lo = static_cast<uint32_t>(order);
                const uint32_t most = wave_max(hi);
                uint64_t who = ballot(hi == most);
                if (who & (who - 1)) {
                    const uint32_t low = wave_max(hi == most ? lo : 0);
                    who = ballot((hi == most) & (lo == low));
                }
                if (lane == first_of(who)) {  // of equal scores the earlier beam's
                    const bool some = order != 0;
                    const int64_t o = b * a.K + j;
                    a.next_scores[o] = some ? score_of(order) : -INFINITY;
                    a.parents[o] = some ? n : 0;
                    a.tokens[o] = some ? token : 0;
                    if (a.next_finished) a.next_finished[o] = some && (over || token == a.end);
                    if (some) {
                        ++at;
                        next();
                    }
                }
            }
        }
        __syncthreads();
    }
}

// ---- reordering.  Thread per (tensor, request, 16-, 8-, 4- or 2-byte unit of a beam's state): every
// beam's unit is read before any is written, so the states move in place; a beam that is its own
// parent is neither read for itself nor written.
struct RArgs {
    char* data[kReorderMost];
    int64_t units[kReorderMost];  // per beam
    int64_t first[kReorderMost + 1];  // first block of each tensor
    const int32_t* parents;
    int64_t Bt;
    int count, N;
    int step;  // the greatest power of two below count, or 0
};

// NU units a thread, 256 apart.
template <class U, int MOST, int NU>
__global__ __launch_bounds__(256) void beam_reorder_kernel(RArgs a) {
    for (int64_t blk = blockIdx.x; blk < a.first[a.count]; blk += gridDim.x) {
        int t = 0;  // the last tensor whose first block is not after blk
        for (int step = a.step; step > 0; step /= 2)
            if (t + step < a.count && a.first[t + step] <= blk) t += step;
        const int64_t units = a.units[t], per = (units + 256 * NU - 1) / (256 * NU);
        const int64_t b = (blk - a.first[t]) / per;
        const int64_t u = (blk - a.first[t]) % per * (256 * NU) + threadIdx.x;
        U* base = reinterpret_cast<U*>(a.data[t]) + b * a.N * units + u;
        const int32_t* par = a.parents + b * a.N;
        U v[MOST][NU];
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            const int p = j < a.N ? par[j] : j;
            if (p != j && p >= 0 && p < a.N) {
#pragma unroll
                for (int k = 0; k < NU; ++k)
                    if (u + 256 * k < units) v[j][k] = base[p * units + 256 * k];
            }
        }
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            const int p = j < a.N ? par[j] : j;
            if (p != j && p >= 0 && p < a.N) {
#pragma unroll
                for (int k = 0; k < NU; ++k)
                    if (u + 256 * k < units) base[j * units + 256 * k] = v[j][k];
            }
        }
    }
}

// A 16-byte unit as a native vector: an array of HIP's struct would not stay in registers.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <class U, int MOST, int NU>
void reorder_n(RArgs& a, hipStream_t s) {
    for (int t = 0; t < a.count; ++t) a.first[t + 1] = a.first[t] + a.Bt * ((a.units[t] + 256 * NU - 1) / (256 * NU));
    a.step = 0;
    for (int p = 1; p < a.count; p *= 2) a.step = p;
    const int64_t total = a.first[a.count];
    const dim3 grid(static_cast<unsigned>(total < (1 << 22) ? total : (1 << 22)));
    beam_reorder_kernel<U, MOST, NU><<<grid, dim3(256), 0, s>>>(a);
}
template <class U>
void reorder_u(RArgs& a, hipStream_t s) {
    if (a.N <= 4) reorder_n<U, 4, 2>(a, s);
    else if (a.N <= 8) reorder_n<U, 8, 1>(a, s);
    else if (a.N <= 16) reorder_n<U, 16, 1>(a, s);
    else if (sizeof(U) == 16 || a.N <= 32) reorder_n<U, 32, 1>(a, s);
    else if constexpr (sizeof(U) < 16) reorder_n<U, 64, 1>(a, s);
}

// Slices per row: blocks for every CU twice over, each wave with a tile, and lists that fit the merging block's shared
// memory.  More blocks mean more lists to fill, one a wave.  Microseconds a call with blocks for every CU
//                                        twice   four times   eight times
//   64 x 8 x 128008 f32                   58.0       67.8         64.4
//   64 x 8 x 128007 f32, 1/4 finished     51.5       61.4         59.0
//   64 x 8 x 128008 bf16                  49.2       52.4         57.9
//   32 x 16 x 32000 bf16                  35.3       43.0         49.0
constexpr int64_t kMergeBytes = 56 << 10;
void plan_select(int64_t rows, int64_t N, int64_t V, int64_t K, int64_t* per, int* slices) {
    const int64_t tiles = (V + kTile - 1) / kTile;
    int64_t n = (512 + rows - 1) / rows;
    n = std::min(n, (tiles + kWaves - 1) / kWaves);
    n = std::max<int64_t>(1, std::min({n, kMergeBytes / (8 * N * K), int64_t{64}}));  // 32 KB for 64 beams of 64
    *per = (tiles + n - 1) / n;
    *slices = static_cast<int>((tiles + *per - 1) / *per);
}

}  // namespace

int64_t beam_select_scratch(int64_t Bt, int64_t N, int64_t V, int64_t K) {
    if (Bt == 0) return 0;
    int64_t per;
    int slices;
    plan_select(Bt * N, N, V, K, &per, &slices);
    return Bt * N * slices * (3 + 2 * K);
}

hipError_t launch_beam_select(const BeamSelectLaunch& l, hipStream_t s) {
    SArgs a{};
    a.logits = l.logits; a.scores = l.scores; a.finished = l.finished; a.next_scores = l.next_scores;
    a.parents = l.parents; a.tokens = l.tokens; a.next_finished = l.next_finished;
    a.Bt = l.Bt; a.V = l.V; a.N = static_cast<int>(l.N); a.K = static_cast<int>(l.K); a.end = l.end;
    plan_select(l.Bt * l.N, l.N, l.V, l.K, &a.tiles, &a.slices);
    const int64_t works = l.Bt * l.N * a.slices;
    a.part_s = reinterpret_cast<double*>(l.scratch);
    a.cand = reinterpret_cast<uint64_t*>(a.part_s + works);
    a.part_m = reinterpret_cast<float*>(a.cand + works * l.K);
    const dim3 grid(blocks_for(works, 1)), block(64 * kWaves);
    if (l.bf16) {
        if (l.vec_ok) beam_slices_kernel<BF16, true><<<grid, block, 0, s>>>(a);
        else beam_slices_kernel<BF16, false><<<grid, block, 0, s>>>(a);
    } else {
        if (l.vec_ok) beam_slices_kernel<F32, true><<<grid, block, 0, s>>>(a);
        else beam_slices_kernel<F32, false><<<grid, block, 0, s>>>(a);
    }
    const size_t lds = static_cast<size_t>(a.N) * a.slices * a.K * 8;
    beam_merge_kernel<<<dim3(blocks_for(l.Bt, 1)), dim3(64 * kMergeWaves), lds, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const BeamReorderLaunch* l, int count, const int32_t* parents, int64_t Bt, int N,
                               hipStream_t s) {
    // one launch per unit size and kReorderMost tensors
    for (int unit : {16, 8, 4, 2}) {
        RArgs a{};
        a.parents = parents;
        a.Bt = Bt;
        a.N = N;
        const auto flush = [&]() {
            if (a.count == 0) return;
            if (unit == 16) reorder_u<u32x4>(a, s);
            else if (unit == 8) reorder_u<u32x2>(a, s);
            else if (unit == 4) reorder_u<uint32_t>(a, s);
            else reorder_u<uint16_t>(a, s);
            a.count = 0;
        };
        for (int t = 0; t < count; ++t) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(l[t].data);
            const auto fits = [&](int64_t u) { return l[t].bytes % u == 0 && at % u == 0; };
            // (more than 32 units of 16 bytes would not stay in registers)
            const int mine = N <= 32 && fits(16) ? 16 : fits(8) ? 8 : fits(4) ? 4 : 2;
            if (mine != unit || l[t].bytes == 0) continue;
            a.data[a.count] = static_cast<char*>(l[t].data);
            a.units[a.count] = l[t].bytes / unit;
            if (++a.count == kReorderMost) flush();
        }
        flush();
    }
    return hipGetLastError();
}

}  // namespace mss
