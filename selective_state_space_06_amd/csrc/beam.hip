// beam.hip -- beam search over a decode step's logits: the best continuations of every request's
// beams, and the beams' recurrent states put in their new order, for gfx950.
//
// Selection.  A live beam's continuation by token v scores score + logit_v - log sum exp(logits);
// a finished beam has one, its end token at its own score.  Per request the k best are kept.  A
// beam's continuations are ordered by their logits alone, so one pass over the logits gives both a
// slice's running maximum and sum of exponentials and its k best (slices kernel); a second, small
// kernel joins the slices of a beam, forms the scores and joins the beams.  Scores are compared in
// 64 bits: they differ by the beams' sums and normalisers, whose 32-bit rounding would decide
// between near candidates.
//
// The k best are a list spread over a wave, entry j in lane j, best first (a higher value, then a
// lower position).  A candidate that beats entry k - 1 is inserted by a shift of the entries behind
// it.  After the first tile few candidates do, and a tile without one costs a compare.
#include "device_math.hpp"
#include "mss_internal.hpp"

namespace mss {
namespace {

constexpr int kE = 8;
constexpr int kTile = 64 * kE;

struct SArgs {
    const void* logits;      // (Bt, N, V)
    const float* scores;     // (Bt, N)
    const int32_t* finished; // (Bt, N), nullable
    float* next_scores;      // (Bt, K)
    int32_t* parents;
    int32_t* tokens;
    int32_t* next_finished;  // nullable
    double* part_s;          // (rows, splits): sum of exp(logit - part_m)
    float* part_m;           // (rows, splits): greatest logit, -inf when there is none
    float* cand_v;           // (rows, splits, K): logits, best first; -inf: no entry
    int32_t* cand_i;         // (rows, splits, K): tokens
    int64_t Bt, V, slice;
    int N, K, splits, end;   // end: -1 for none
};

__device__ __forceinline__ float lane_of(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ uint64_t join64(uint32_t hi, uint32_t lo) { return static_cast<uint64_t>(hi) << 32 | lo; }
__device__ __forceinline__ uint64_t lane_of(uint64_t v, int lane) {
    return join64(__builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane),
                  __builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ int shift_up(int v) { return __builtin_amdgcn_update_dpp(v, v, 0x138, 0xF, 0xF, false); }
__device__ __forceinline__ float shift_up(float v) { return __int_as_float(shift_up(__float_as_int(v))); }
__device__ __forceinline__ uint64_t shift_up(uint64_t v) {
    return join64(shift_up(static_cast<int>(v >> 32)), shift_up(static_cast<int>(v)));
}

// A 64-bit score as a whole number of the same order, 0 for a score that is -inf or not a number (a
// list's empty entry).  The second list holds these, and no double: the compiler here encodes a scalar
// move of a 64-bit -inf as one of 0 (the literal's low half).  For the same reason -inf is told by its
// two halves.
__device__ __forceinline__ uint64_t key_of(double s) {
    s += 0.0;  // -0 orders as +0
    const uint32_t hi = __double2hiint(s), lo = __double2loint(s);
    if (s != s || (hi == 0xFFF00000u && lo == 0u)) return 0;
    const uint32_t flip = static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31);
    return join64(hi ^ (flip | 0x80000000u), lo ^ flip);
}
__device__ __forceinline__ float score_of(uint64_t key) {  // of a key that is not 0
    const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
    const uint32_t flip = static_cast<uint32_t>(~(static_cast<int32_t>(hi) >> 31));
    return static_cast<float>(__hiloint2double(static_cast<int>(hi ^ (flip | 0x80000000u)), static_cast<int>(lo ^ flip)));
}

template <class T> __device__ __forceinline__ T none();
template <> __device__ __forceinline__ float none<float>() { return -INFINITY; }
template <> __device__ __forceinline__ uint64_t none<uint64_t>() { return 0; }

// The list of a wave: lane j holds the j-th best, none / INT_MAX where there is none yet.
template <class T>
struct List {
    T v;
    int i;
    T last_v;  // entry k - 1, the same in every lane
    int last_i;
    __device__ __forceinline__ void clear() {
        v = last_v = none<T>();
        i = last_i = INT32_MAX;
    }
    // true where (w, j) would enter; never for none or a value that is not a number
    __device__ __forceinline__ bool takes(T w, int j) const {
        return w > last_v || (w == last_v && j < last_i && w > none<T>());
    }
    // w and j the same in every lane
    __device__ __forceinline__ void insert(T w, int j, int k, int lane) {
        const bool ahead = v > w || (v == w && i < j);
        const int at = __popcll(__ballot(ahead));
        const T sv = shift_up(v);
        const int si = shift_up(i);
        if (lane > at) v = sv, i = si;
        else if (lane == at) v = w, i = j;
        last_v = lane_of(v, k - 1);
        last_i = lane_of(i, k - 1);
    }
    // every lane's (w, j) offered, in any order; w = none for a lane without one
    __device__ __forceinline__ void offer(T w, int j, int k, int lane) {
        uint64_t left = __ballot(takes(w, j));
        while (left) {
            const int src = __ffsll(static_cast<unsigned long long>(left)) - 1;
            insert(lane_of(w, src), lane_of(j, src), k, lane);
            if (lane == src) w = none<T>();
            left = __ballot(takes(w, j));
        }
    }
};

// One wave per (row, slice of the vocabulary).  VEC: rows are whole aligned 16-byte vectors.
template <class E, bool VEC>
__global__ __launch_bounds__(256) void beam_slices_kernel(SArgs a) {
    constexpr int V = E::kPerVec;
    const int lane = threadIdx.x & 63;
    const int64_t works = a.Bt * a.N * a.splits;
    for (int64_t g = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); g < works; g += (int64_t)gridDim.x * 4) {
        const int64_t row = g / a.splits, split = g % a.splits;
        const int64_t lo = split * a.slice, hi = lo + a.slice < a.V ? lo + a.slice : a.V;
        const auto* p = static_cast<const typename E::storage*>(a.logits) + row * a.V;
        List<float> list;
        list.clear();
        float m = -INFINITY, s = 0.0f;  // of this lane's elements
        // a beam at its end or without a score has no continuation that needs its logits
        const float score = a.scores[row];
        const bool skip = (a.finished && a.finished[row] != 0) || !(score > -INFINITY);
        for (int64_t t = lo; !skip && t < hi; t += kTile) {
            const int64_t t0 = t + lane * kE;
            float v[kE];
#pragma unroll
            for (int j = 0; j < kE / V; ++j) {
                const int64_t q = t0 + j * V;
                if (q + V <= hi) {
                    uint4 w;
                    if (VEC) w = *reinterpret_cast<const uint4*>(p + q);
                    else __builtin_memcpy(&w, p + q, 16);
                    E::unpack(w, v + j * V);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[j * V + e] = q + e < hi ? E::load1(p, q + e) : -INFINITY;
                }
            }
            float best = -INFINITY;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                v[e] = v[e] == v[e] ? v[e] : -INFINITY;  // a NaN logit is masked
                best = fmaxf(best, v[e]);
            }
            if (best > m) {
                s *= fast_exp2((m - best) * kLog2e);
                m = best;
            }
            const float ref = m > -INFINITY ? m : 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) s += fast_exp2((v[e] - ref) * kLog2e);
            // the lanes' best that enter the list, one at a time
            int bi = 0;
            for (;;) {
#pragma unroll
                for (int e = kE - 1; e >= 0; --e) bi = v[e] == best ? e : bi;
                const int at = static_cast<int>(t0) + bi;
                const uint64_t left = __ballot(list.takes(best, at));
                if (!left) break;
                const int src = __ffsll(static_cast<unsigned long long>(left)) - 1;
                list.insert(lane_of(best, src), lane_of(at, src), a.K, lane);
                if (lane == src) {
                    best = -INFINITY;
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        if (e == bi) v[e] = -INFINITY;
                        best = fmaxf(best, v[e]);
                    }
                }
            }
        }
        // the lanes' maxima and sums joined, the sums in 64 bits
        float top = m;
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
        double sum = top > -INFINITY ? static_cast<double>(s) * fast_exp2((m - top) * kLog2e) : 0.0;
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
        if (lane == 0) {
            a.part_m[g] = top;
            a.part_s[g] = sum;
        }
        if (lane < a.K) {
            a.cand_v[g * a.K + lane] = list.v;
            a.cand_i[g * a.K + lane] = list.i;
        }
    }
}

// One block per request: its waves join the slices of the beams in turn, then the first wave joins
// the beams.  Shared memory: N K scores (as keys), N K tokens, N flags.
__global__ __launch_bounds__(256) void beam_join_kernel(SArgs a) {
    extern __shared__ uint64_t shared[];
    uint64_t* sc = shared;
    int* tok = reinterpret_cast<int*>(sc + a.N * a.K);
    int* fin = tok + a.N * a.K;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t b = blockIdx.x; b < a.Bt; b += gridDim.x) {
        for (int n = wave; n < a.N; n += 4) {
            const int64_t row = b * a.N + n;
            const double score = a.scores[row];
            const bool done = a.finished && a.finished[row] != 0;
            uint64_t total = 0;
            int token = 0;
            if (done) {
                if (lane == 0) total = key_of(score), token = a.end;
            } else {
                List<float> list;
                list.clear();
                const int64_t first = row * a.splits;
                const float m = lane < a.splits ? a.part_m[first + lane] : -INFINITY;
                float top = m;
#pragma unroll
                for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
                double sum = 0.0;
                if (lane < a.splits && m > -INFINITY) sum = a.part_s[first + lane] * exp(static_cast<double>(m) - top);
#pragma unroll
                for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
                const double lse = static_cast<double>(top) + log(sum);
                const int all = a.splits * a.K;
                for (int c = 0; c < all; c += 64) {
                    const bool ok = c + lane < all;
                    list.offer(ok ? a.cand_v[first * a.K + c + lane] : -INFINITY,
                               ok ? a.cand_i[first * a.K + c + lane] : 0, a.K, lane);
                }
                if (list.v > -INFINITY) {
                    total = key_of(score + (static_cast<double>(list.v) - lse));
                    token = list.i;
                }
            }
            if (lane < a.K) {
                sc[n * a.K + lane] = total;
                tok[n * a.K + lane] = token;
            }
            if (lane == 0) fin[n] = done;
        }
        __syncthreads();
        if (wave == 0) {
            List<uint64_t> list;
            list.clear();
            const int all = a.N * a.K;
            for (int c = 0; c < all; c += 64)
                list.offer(c + lane < all ? sc[c + lane] : 0, c + lane, a.K, lane);
            if (lane < a.K) {
                const bool some = list.v != 0;
                const int at = some ? list.i : 0;
                const int parent = some ? at / a.K : 0, token = some ? tok[at] : 0;
                const int64_t o = b * a.K + lane;
                a.next_scores[o] = some ? score_of(list.v) : -INFINITY;
                a.parents[o] = parent;
                a.tokens[o] = token;
                if (a.next_finished) a.next_finished[o] = some && (fin[parent] || token == a.end);
            }
        }
        __syncthreads();
    }
}

// ---- reordering.  Thread per (tensor, request, 16-, 4- or 2-byte unit of a beam's state): every
// beam's unit is read before any is written, so the states move in place; a beam that is its own
// parent is neither read for itself nor written.
struct RArgs {
    char* data[kReorderMost];
    int64_t units[kReorderMost];  // per beam
    int64_t first[kReorderMost + 1];  // first block of each tensor
    const int32_t* parents;
    int64_t Bt;
    int count, N;
};

template <class U, int MOST>
__global__ __launch_bounds__(256) void beam_reorder_kernel(RArgs a) {
    for (int64_t blk = blockIdx.x; blk < a.first[a.count]; blk += gridDim.x) {
        int t = 0;
        while (blk >= a.first[t + 1]) ++t;
        const int64_t units = a.units[t], per = (units + 255) / 256;
        const int64_t b = (blk - a.first[t]) / per;
        const int64_t u = (blk - a.first[t]) % per * 256 + threadIdx.x;
        if (u >= units) continue;
        U* base = reinterpret_cast<U*>(a.data[t]) + b * a.N * units + u;
        const int32_t* par = a.parents + b * a.N;
        U v[MOST];
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            if (j < a.N) {
                const int p = par[j];
                if (p != j && p >= 0 && p < a.N) v[j] = base[p * units];
            }
        }
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            if (j < a.N) {
                const int p = par[j];
                if (p != j && p >= 0 && p < a.N) base[j * units] = v[j];
            }
        }
    }
}

template <class U>
void reorder_u(const RArgs& a, hipStream_t s) {
    const int64_t total = a.first[a.count];
    const dim3 grid(static_cast<unsigned>(total < (1 << 22) ? total : (1 << 22))), block(256);
    if (a.N <= 4) beam_reorder_kernel<U, 4><<<grid, block, 0, s>>>(a);
    else if (a.N <= 8) beam_reorder_kernel<U, 8><<<grid, block, 0, s>>>(a);
    else if (a.N <= 16) beam_reorder_kernel<U, 16><<<grid, block, 0, s>>>(a);
    else beam_reorder_kernel<U, 64><<<grid, block, 0, s>>>(a);
}

// Slices per row: enough waves to fill the chip, none shorter than a tile, at most one per lane of
// the joining wave.
void plan_select(int64_t rows, int64_t V, int64_t* slice, int* splits) {
    int64_t n = (4096 + rows - 1) / (rows < 1 ? 1 : rows);
    const int64_t tiles = (V + kTile - 1) / kTile;
    if (n > 64) n = 64;
    if (n > tiles) n = tiles;
    if (n < 1) n = 1;
    const int64_t per = (tiles + n - 1) / n;
    *slice = (per < 1 ? 1 : per) * kTile;
    *splits = static_cast<int>(tiles > 0 ? (V + *slice - 1) / *slice : 1);
}

}  // namespace

int64_t beam_select_scratch(int64_t Bt, int64_t N, int64_t V, int64_t K) {
    int64_t slice;
    int splits;
    plan_select(Bt * N, V, &slice, &splits);
    return Bt * N * splits * (3 + 2 * K);
}

hipError_t launch_beam_select(const BeamSelectLaunch& l, hipStream_t s) {
    SArgs a{};
    a.logits = l.logits; a.scores = l.scores; a.finished = l.finished; a.next_scores = l.next_scores;
    a.parents = l.parents; a.tokens = l.tokens; a.next_finished = l.next_finished;
    a.Bt = l.Bt; a.V = l.V; a.N = static_cast<int>(l.N); a.K = static_cast<int>(l.K); a.end = l.end;
    plan_select(l.Bt * l.N, l.V, &a.slice, &a.splits);
    const int64_t works = l.Bt * l.N * a.splits;
    a.part_s = reinterpret_cast<double*>(l.scratch);
    a.part_m = l.scratch + 2 * works;
    a.cand_v = a.part_m + works;
    a.cand_i = reinterpret_cast<int32_t*>(a.cand_v + works * l.K);
    const int64_t blocks = (works + 3) / 4;
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 22) ? blocks : (1 << 22))), block(256);
    if (l.bf16) {
        if (l.vec_ok) beam_slices_kernel<BF16, true><<<grid, block, 0, s>>>(a);
        else beam_slices_kernel<BF16, false><<<grid, block, 0, s>>>(a);
    } else {
        if (l.vec_ok) beam_slices_kernel<F32, true><<<grid, block, 0, s>>>(a);
        else beam_slices_kernel<F32, false><<<grid, block, 0, s>>>(a);
    }
    const size_t lds = static_cast<size_t>(a.N) * a.K * 12 + static_cast<size_t>(a.N) * 4;  // at most 49.5 KB
    beam_join_kernel<<<dim3(static_cast<unsigned>(l.Bt < (1 << 22) ? l.Bt : (1 << 22))), block, lds, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const BeamReorderLaunch* l, int count, const int32_t* parents, int64_t Bt, int N,
                               hipStream_t s) {
    // one launch per unit size and kReorderMost tensors
    for (int unit : {16, 4, 2}) {
        if (unit == 16 && N > 16) continue;  // 64 16-byte units would not stay in registers
        RArgs a{};
        a.parents = parents;
        a.Bt = Bt;
        a.N = N;
        auto flush = [&]() {
            if (a.count == 0) return;
            if (unit == 16) reorder_u<uint4>(a, s);
            else if (unit == 4) reorder_u<uint32_t>(a, s);
            else reorder_u<uint16_t>(a, s);
            a.count = 0;
        };
        for (int t = 0; t < count; ++t) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(l[t].data);
            const auto fits = [&](int64_t u) { return l[t].bytes % u == 0 && at % u == 0; };
            const int mine = N <= 16 && fits(16) ? 16 : fits(4) ? 4 : 2;
            if (mine != unit || l[t].bytes == 0) continue;
            a.data[a.count] = static_cast<char*>(l[t].data);
            a.units[a.count] = l[t].bytes / unit;
            a.first[a.count + 1] = a.first[a.count] + Bt * ((a.units[a.count] + 255) / 256);
            if (++a.count == kReorderMost) flush();
        }
        flush();
    }
    return hipGetLastError();
}

}  // namespace mss
