// linear_attention.hip -- linear attention with one decay per head, for gfx950: whole sequences (chunked, on the
// matrix cores), their gradients, and one token.
//
// Per batch and head, with l = exp(-rate): S_t = l S_{t-1} + k_t v_t^T, out_t = scale S_t^T q_t.  A chunk of C steps
// from the state S before it is
//     out_t = scale (l^(t+1) S^T q_t + sum_{s <= t} l^(t-s) (q_t . k_s) v_s)        t, s = 0 .. C-1
//     S'    = l^C S + sum_s l^(C-1-s) k_s v_s^T,
// four small products.  The gradients are the same sum in other roles: dq from (q, k, v) = (dout, v, k) and the
// transposed state; dv and dk backwards in time from (k, q, dout) and (v, dout, q), with dlast_state in front.  So one
// kernel serves all of them, by the tensors it is given, the order in which it takes the rows, and where the scale goes.
//
// A block holds a slice of 64 value columns of one head: its four waves 16 columns each, the state's rows of these
// columns in registers (fp32) all along the sequence.  Queries, keys and values of a chunk go through LDS; the next
// chunk's are on their way meanwhile.  Scores and state pass from product to product in registers: a product's result
// (lane: a column, four consecutive rows) is the next product's operand as it stands, when the other operand's rows are
// taken in the same order.
//
// bf16 products of fp32 values: a value is cut into bf16 parts (hi = bf16(x), mid = bf16(x - hi), ...), each exact,
// and the products of parts that matter are summed in fp32.  bf16 inputs are one part; states and scores, met by a
// rounding to bf16 of the output, are taken in two (2^-17), the decayed values that enter the state in three (2^-25).
// fp32 inputs are three parts everywhere, with the six products down to 2^-24 (2.7 times the rate of the fp32 matrix
// instruction).
#include <algorithm>

#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"

namespace mss {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

struct Rows {          // (Bt, L, heads, dim)
    const void* p;
    int heads;
};

struct AArgs {
    Rows q, k, v;
    const float* rate;       // (H)
    const int32_t* lens;     // (Bt), nullable
    const float* init;       // state before (Bt, H, Kd, Vd), or (Bt, H, Vd, Kd) with init_t; nullable
    float* last;             // state after, laid out alike; nullable
    float* segs;             // (Bt, H, nseg, Kd, Vd): states entering the segments (of 64 seg_len steps)
    void* out;               // (Bt, L, H, Vd)
    int64_t Bt, L;
    int H, Kd, Vd, nseg;
    int64_t seg_steps;       // a multiple of 64
    float s_add, s_out;      // factors of what enters the state, and of the outputs
    bool turned;             // init and last are (Vd, Kd)
    bool back;               // rows in reverse order
};

constexpr int kWaves = 4, kVTile = 16 * kWaves;
constexpr float kMostRate = 1e30f;  // beyond it l^n is 0 for every n but 0, which 0 times infinity would not be

__device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}
// Of a block of 4 rows x 16 columns in LDS, whose row r is held by the four lanes 4r .. 4r + 3 of 16 (p: this lane's
// four columns), lane c of the 16 gets column c.
__device__ __forceinline__ s16x4 turn4(const uint16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}
__device__ __forceinline__ s16x8 join8(s16x4 a, s16x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// Eight floats as N bf16 parts.
template <int N>
__device__ __forceinline__ void cut(const float* x, s16x8* part) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = pack_bf16x2(r[2 * e], r[2 * e + 1]);
            if (n + 1 < N) {
                r[2 * e] -= bf16_lo(w[e]);
                r[2 * e + 1] -= bf16_hi(w[e]);
            }
        }
        part[n] = __builtin_bit_cast(s16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

template <class E>
struct Form;
template <>
struct Form<BF16> {
    static constexpr int C = 64, NP = 1, NS = 2;  // steps a chunk; parts of inputs; of states and scores
};
template <>
struct Form<F32> {
    static constexpr int C = 32, NP = 3, NS = 3;
};

// sum of products of parts a (NA) and b (NB), down to the least part of either that is kept
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma_parts(const s16x8* a, const s16x8* b, f32x4 c) {
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j < most) c = mma(a[i], b[j], c);
    return c;
}

// STATES: only the state that a segment adds, from zero.  OUT: the outputs' type.
template <class E, class OUT, int KD, bool STATES>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_kernel(AArgs a) {
    using F = Form<E>;
    using S = typename E::storage;
    constexpr int C = F::C, NP = F::NP, NS = F::NS, MT = C / 16, M2 = C / 32, KJ = KD / 32;
    constexpr int QS = KD + 8, VS = kVTile + 8;              // elements between two rows in LDS
    constexpr int NQ = C * KD / 8 / 256, NV = C * kVTile / 8 / 256;
    __shared__ __align__(16) uint16_t qs[STATES ? 1 : NP][STATES ? 1 : C][STATES ? 8 : QS];
    __shared__ __align__(16) uint16_t ks[NP][C][QS];
    __shared__ __align__(16) uint16_t vs[NP][C][VS];

    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int vtiles = (a.Vd + kVTile - 1) / kVTile, nseg = STATES ? a.nseg - 1 : a.nseg;
    const int64_t bh = blockIdx.x / (vtiles * nseg);
    const int rest = static_cast<int>(blockIdx.x % (vtiles * nseg));
    const int seg = rest / vtiles, vt = rest % vtiles;
    const int64_t b = bh / a.H;
    const int h = static_cast<int>(bh % a.H);
    const int64_t len = a.lens ? (a.lens[b] < 0 ? 0 : a.lens[b] < a.L ? a.lens[b] : a.L) : a.L;
    const int64_t from = seg * a.seg_steps, to = from + a.seg_steps < a.L ? from + a.seg_steps : a.L;
    const int v0 = vt * kVTile + wave * 16;                  // this wave's columns
    const bool mine = v0 < a.Vd;
    const bool first_whole = a.back;                         // the state enters the first row undecayed

    const auto row_of = [&](const Rows& t, int dim) MSS_INLINED {
        return static_cast<const S*>(t.p) + (b * a.L * t.heads + h / (a.H / t.heads)) * dim;
    };
    const S* qp = row_of(a.q, a.Kd);
    const S* kp = row_of(a.k, a.Kd);
    const S* vp = row_of(a.v, a.Vd);
    const int64_t qn = static_cast<int64_t>(a.q.heads) * a.Kd, kn = static_cast<int64_t>(a.k.heads) * a.Kd,
                  vn = static_cast<int64_t>(a.v.heads) * a.Vd;

    Raw<E> rq[STATES ? 1 : NQ], rk[NQ], rv[NV];
    const auto load_rows = [&](const S* p, int64_t step, int dim, int col0, int64_t at, int units, int u, Raw<E>& r)
                               MSS_INLINED {
        const int row = u / units, col = col0 + u % units * 8;
        const int64_t t = at + row;
#pragma unroll
        for (int j = 0; j < kE / E::kPerVec; ++j) r.q[j] = make_uint4(0, 0, 0, 0);
        if (t < len && col < dim) {
            const S* s = p + (a.back ? len - 1 - t : t) * step + col;
#pragma unroll
            for (int j = 0; j < kE / E::kPerVec; ++j) r.q[j] = *reinterpret_cast<const uint4*>(s + j * E::kPerVec);
        }
    };
    const auto load = [&](int64_t at) MSS_INLINED {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            if constexpr (!STATES) load_rows(qp, qn, a.Kd, 0, at, KD / 8, threadIdx.x + j * 256, rq[j]);
            load_rows(kp, kn, a.Kd, 0, at, KD / 8, threadIdx.x + j * 256, rk[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            load_rows(vp, vn, a.Vd, vt * kVTile, at, kVTile / 8, threadIdx.x + j * 256, rv[j]);
    };
    const auto put = [&](const Raw<E>& r, uint16_t* p, int64_t plane) MSS_INLINED {
        if constexpr (NP == 1) {
            *reinterpret_cast<uint4*>(p) = r.q[0];
        } else {
            float x[kE];
            r.unpack(x);
            s16x8 part[NP];
            cut<NP>(x, part);
#pragma unroll
            for (int n = 0; n < NP; ++n) *reinterpret_cast<s16x8*>(p + n * plane) = part[n];
        }
    };
    const auto store = [&]() MSS_INLINED {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int u = threadIdx.x + j * 256, row = u / (KD / 8), col = u % (KD / 8) * 8;
            if constexpr (!STATES) put(rq[j], &qs[0][row][col], C * QS);
            put(rk[j], &ks[0][row][col], C * QS);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int u = threadIdx.x + j * 256;
            put(rv[j], &vs[0][u / (kVTile / 8)][u % (kVTile / 8) * 8], C * VS);
        }
    };

    // powers of the decay.  A score's lane is a column t = 16 b + r16, its rows s = 16 a + 4 g + i.
    const float rate = fminf(fmaxf(a.rate[h], 0.0f), kMostRate), rl = rate * kLog2e;
    const auto power = [&](int n) MSS_INLINED { return fast_exp2(-rl * static_cast<float>(n)); };
    float near[4], off[4], tail[4], step16[MT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = r16 - 4 * g - i;
        near[i] = n >= 0 ? power(n) * (a.s_add * a.s_out) : 0.0f;
        off[i] = power(16 + n) * (a.s_add * a.s_out);
        tail[i] = power(15 - 4 * g - i) * a.s_add;
    }
#pragma unroll
    for (int n = 0; n < MT; ++n) step16[n] = power(16 * n);
    const float since = power(r16 + 1) * a.s_out, since0 = power(r16) * a.s_out;
    const float less = expm1f(-rate * C);

    // the state: tile j holds rows 32 (j / 2) + 8 g + 4 (j % 2) + i of column v0 + r16
    f32x4 st[KD / 16];
    const auto state_at = [&](int j, int i) MSS_INLINED { return 32 * (j / 2) + 8 * g + 4 * (j % 2) + i; };
#pragma unroll
    for (int j = 0; j < KD / 16; ++j) {
        st[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (STATES || !mine) continue;
        const int v = v0 + r16;
        const float* from_segs = a.nseg > 1 ? a.segs + (bh * a.nseg + seg) * a.Kd * a.Vd : nullptr;
        const float* from_init = a.init ? a.init + bh * a.Kd * a.Vd : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = state_at(j, i);
            if (k >= a.Kd) continue;
            if (from_segs) st[j][i] = from_segs[k * a.Vd + v];
            else if (from_init) st[j][i] = from_init[a.turned ? v * a.Kd + k : k * a.Vd + v];
        }
    }

    const int64_t stop = to < len ? to : len;  // rows past it are 0
    if (from < stop) load(from);
    for (int64_t at = from; at < stop; at += C) {
        store();
        __syncthreads();
        if (at + C < stop) load(at + C);
        const int n = len - at < C ? static_cast<int>(len - at) : C;  // rows of this chunk
        s16x8 vf[M2][NP];
        if (mine) {
#pragma unroll
            for (int m = 0; m < M2; ++m)
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const uint16_t* s = &vs[p][32 * m + 4 * g + (r16 >> 2)][wave * 16 + 4 * (r16 & 3)];
                    vf[m][p] = join8(turn4(s), turn4(s + 16 * VS));
                }
            if constexpr (!STATES) {
                s16x8 sf[KJ][NS];
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = st[2 * j][i], x[4 + i] = st[2 * j + 1][i];
                    cut<NS>(x, sf[j]);
                }
                const float in = at == 0 && first_whole ? since0 : since;
#pragma unroll
                for (int tb = 0; tb < MT; ++tb) {
                    s16x8 qf[KJ][NP];
#pragma unroll
                    for (int j = 0; j < KJ; ++j)
#pragma unroll
                        for (int p = 0; p < NP; ++p)
                            qf[j][p] = *reinterpret_cast<const s16x8*>(&qs[p][16 * tb + r16][32 * j + 8 * g]);
                    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};  // rows: columns v, lanes: steps t
#pragma unroll
                    for (int j = 0; j < KJ; ++j) acc = mma_parts<NS, NP>(sf[j], qf[j], acc);
                    acc *= in * step16[tb];
                    float sc[MT][4];
#pragma unroll
                    for (int ta = 0; ta < (tb / 2 + 1) * 2; ++ta) {
                        if (ta > tb) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) sc[ta][i] = 0.0f;
                            continue;
                        }
                        f32x4 p4 = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int j = 0; j < KJ; ++j) {
                            s16x8 kf[NP];
#pragma unroll
                            for (int p = 0; p < NP; ++p)
                                kf[p] = *reinterpret_cast<const s16x8*>(&ks[p][16 * ta + r16][32 * j + 8 * g]);
                            p4 = mma_parts<NP, NP>(kf, qf[j], p4);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sc[ta][i] = ta < tb ? p4[i] * (off[i] * step16[tb - ta - 1])
                                                : r16 >= 4 * g + i ? p4[i] * near[i] : 0.0f;
                    }
#pragma unroll
                    for (int m = 0; m <= tb / 2; ++m) {
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = sc[2 * m][i], x[4 + i] = sc[2 * m + 1][i];
                        s16x8 pf[NS];
                        cut<NS>(x, pf);
                        acc = mma_parts<NP, NS>(vf[m], pf, acc);
                    }
                    const int64_t t = at + 16 * tb + r16;
                    if (t < stop) {
                        const int64_t token = a.back ? len - 1 - t : t;
                        auto* o = static_cast<typename OUT::storage*>(a.out) + ((b * a.L + token) * a.H + h) * a.Vd + v0 + 4 * g;
                        if (sizeof(typename OUT::storage) == 2) {
                            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
                        } else {
                            *reinterpret_cast<f32x4*>(o) = acc;
                        }
                    }
                }
            }
        }
        // the state after the chunk, if it is read
        if (mine && (STATES || at + C < stop || (a.last && seg == a.nseg - 1))) {
            const bool odd = n < C || (at == 0 && first_whole);
            const float gone = odd ? expm1f(-rate * static_cast<float>(at == 0 && first_whole ? n - 1 : n)) : less;
#pragma unroll
            for (int j = 0; j < KD / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) st[j][i] = fmaf(st[j][i], gone, st[j][i]);
#pragma unroll
            for (int m = 0; m < M2; ++m) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = 0.0f;
#pragma unroll
                    for (int p = 0; p < NP; ++p) v += bf16_to_f32(static_cast<uint16_t>(vf[m][p][e]));
                    const int tile = 2 * m + e / 4, s = 16 * tile + 4 * g + e % 4;
                    float w = tail[e % 4] * step16[MT - 1 - tile];
                    if (n < C) w = power(n - 1 - s > 0 ? n - 1 - s : 0) * a.s_add;  // rows past the end are zeros
                    x[e] = v * w;
                }
                s16x8 wf[3];
                cut<3>(x, wf);
#pragma unroll
                for (int j = 0; j < KD / 16; ++j) {
                    s16x8 kt[NP];
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const uint16_t* s = &ks[p][32 * m + 4 * g + (r16 >> 2)][32 * (j / 2) + 4 * (j % 2) + 8 * (r16 & 3)];
                        kt[p] = join8(turn4(s), turn4(s + 16 * QS));
                    }
                    st[j] = mma_parts<NP, 3>(kt, wf, st[j]);
                }
            }
        }
        __syncthreads();
    }
    if (!mine) return;
    const int v = v0 + r16;
    if constexpr (STATES) {
        float* o = a.segs + (bh * a.nseg + seg) * a.Kd * a.Vd;
#pragma unroll
        for (int j = 0; j < KD / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (state_at(j, i) < a.Kd) o[state_at(j, i) * a.Vd + v] = st[j][i];
    } else {
        for (int64_t t = (from > len ? from : len) + r16; t < to; t += 16) {  // past the end
            auto* o = static_cast<typename OUT::storage*>(a.out) + ((b * a.L + t) * a.H + h) * a.Vd + v0 + 4 * g;
            if (sizeof(typename OUT::storage) == 2) *reinterpret_cast<uint2*>(o) = make_uint2(0, 0);
            else *reinterpret_cast<f32x4*>(o) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if (a.last && seg == a.nseg - 1) {
            // walked backwards, the state is that of the first step: the one before it is a step further
            const float f = a.back && len > 0 ? power(1) : 1.0f;
            float* o = a.last + bh * a.Kd * a.Vd;
#pragma unroll
            for (int j = 0; j < KD / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = state_at(j, i);
                    if (k < a.Kd) o[a.turned ? v * a.Kd + k : k * a.Vd + v] = st[j][i] * f;
                }
        }
    }
}

// The states that enter the segments, from what each of them adds: a thread per element, in place.
__global__ __launch_bounds__(256) void attention_join_kernel(AArgs a) {
    const int64_t per = static_cast<int64_t>(a.Kd) * a.Vd, all = a.Bt * a.H * per;
    for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < all; e += gridDim.x * 256ll) {
        const int64_t bh = e / per, x = e % per, b = bh / a.H;
        const int64_t len = a.lens ? (a.lens[b] < 0 ? 0 : a.lens[b] < a.L ? a.lens[b] : a.L) : a.L;
        const float rate = fminf(fmaxf(a.rate[bh % a.H], 0.0f), kMostRate);
        float s = 0.0f;
        if (a.init) s = a.init[bh * per + (a.turned ? x % a.Vd * a.Kd + x / a.Vd : x)];
        float* o = a.segs + bh * a.nseg * per + x;
        for (int seg = 0; seg < a.nseg; ++seg) {
            const float adds = seg + 1 < a.nseg ? o[seg * per] : 0.0f;
            o[seg * per] = s;
            int64_t n = len - seg * a.seg_steps;
            n = n < 0 ? 0 : n < a.seg_steps ? n : a.seg_steps;
            if (n > 0 && seg == 0 && a.back) --n;
            s = fmaf(s, expm1f(-rate * static_cast<float>(n)), s) + adds;
        }
    }
}

// out (rows, groups, dim) = sum over the heads of a group of part (rows, groups, each, dim), in their order.
template <class E>
__global__ __launch_bounds__(256) void attention_groups_kernel(const float* part, void* out, int64_t n, int each, int dim) {
    // a thread per four elements
    for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < n; e += gridDim.x * 256ll) {
        const int64_t group = e / (dim / 4);
        const int c = static_cast<int>(e % (dim / 4)) * 4;
        const float* p = part + group * each * dim + c;
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < each; ++j) s += *reinterpret_cast<const f32x4*>(p + static_cast<int64_t>(j) * dim);
        auto* o = static_cast<typename E::storage*>(out) + e * 4;
        if (sizeof(typename E::storage) == 2)
            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
        else *reinterpret_cast<f32x4*>(o) = s;
    }
}

// ---- one token.  A block per (batch, head): a thread holds four columns of every R-th row of the state; the rows'
// parts of the output are summed through LDS.
template <class E>
__global__ __launch_bounds__(256) void attention_update_kernel(AttnUpdateLaunch a) {
    __shared__ float qk[2][kAttnMostDim];
    __shared__ float part[256 * 4];
    const int64_t bh = blockIdx.x, b = bh / a.H;
    const int h = static_cast<int>(bh % a.H), tid = threadIdx.x;
    const int quads = a.V / 4, R = 256 / quads, r = tid / quads, c = tid % quads;
    if (tid < a.K) {
        qk[0][tid] = E::load1(a.q, (b * a.Hq + h / (a.H / a.Hq)) * a.K + tid) * a.scale;
        qk[1][tid] = E::load1(a.k, (b * a.Hk + h / (a.H / a.Hk)) * a.K + tid);
    }
    const float less = expm1f(-fminf(fmaxf(a.rate[h], 0.0f), kMostRate));
    f32x4 v, out = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t at = (b * a.Hv + h / (a.H / a.Hv)) * a.V + 4 * c;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = E::load1(a.v, at + i);
    __syncthreads();
    if (r < R) {
        f32x4* s = reinterpret_cast<f32x4*>(a.state + bh * a.K * a.V) + c;
#pragma unroll 8
        for (int k = r; k < a.K; k += R) {
            f32x4 x = s[k * quads];
            const float q = qk[0][k], kk = qk[1][k];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = fmaf(kk, v[i], fmaf(x[i], less, x[i]));
                out[i] = fmaf(q, x[i], out[i]);
            }
            s[k * quads] = x;
        }
        *reinterpret_cast<f32x4*>(part + (r * quads + c) * 4) = out;
    }
    __syncthreads();
    if (tid < a.V) {
        float s = 0.0f;
        const int rows = a.K < R ? a.K : R;
        for (int j = 0; j < rows; ++j) s += part[j * a.V + tid];
        E::store1(a.out, bh * a.V + tid, s);
    }
}

// Segments, and steps of each: blocks for every CU twice over, but none of under 256 steps (each re-reads its keys and
// values).
void plan_segments(int64_t Bt, int64_t L, int H, int Vd, int* nseg, int64_t* steps) {
    const int64_t blocks = Bt * H * ((Vd + kVTile - 1) / kVTile);
    const int64_t most = std::max<int64_t>(1, L / 256);
    const int64_t n = std::min(most, std::max<int64_t>(1, 512 / std::max<int64_t>(1, blocks)));
    *steps = std::max<int64_t>(64, ((L + n - 1) / n + 63) / 64 * 64);
    *nseg = static_cast<int>(std::max<int64_t>(1, (L + *steps - 1) / *steps));
}

template <class E, class OUT, int KD>
void walk_kd(const AArgs& a, hipStream_t s) {
    const int64_t heads = a.Bt * a.H * ((a.Vd + kVTile - 1) / kVTile);
    if (a.nseg > 1) {
        attention_kernel<E, E, KD, true><<<dim3(static_cast<unsigned>(heads * (a.nseg - 1))), dim3(64 * kWaves), 0, s>>>(a);
        attention_join_kernel<<<dim3(blocks_for(a.Bt * a.H * a.Kd * a.Vd, 256)), dim3(256), 0, s>>>(a);
    }
    attention_kernel<E, OUT, KD, false><<<dim3(static_cast<unsigned>(heads * a.nseg)), dim3(64 * kWaves), 0, s>>>(a);
}
template <class E, class OUT>
void walk(const AArgs& a, hipStream_t s) {
    if (a.Kd <= 64) walk_kd<E, OUT, 64>(a, s);
    else walk_kd<E, OUT, 128>(a, s);
}

template <class E>
void backward(const AttnLaunch& l, hipStream_t s) {
    // (queries, keys, values) of each walk; K x V states are read the other way round where the roles of K and V are
    const Rows q{l.q, l.Hq}, k{l.k, l.Hk}, v{l.v, l.Hv}, d{l.dout, l.H};
    struct Walk {
        Rows q, k, v;
        void* out;
        int heads, Kd, Vd;
        bool back, turned;
    };
    const Walk walks[3] = {{d, v, k, l.dq, l.Hq, l.V, l.K, false, true},
                           {v, d, q, l.dk, l.Hk, l.V, l.K, true, true},
                           {k, q, d, l.dv, l.Hv, l.K, l.V, true, false}};
    for (const Walk& w : walks) {
        AArgs a{};
        a.q = w.q; a.k = w.k; a.v = w.v; a.rate = l.rate; a.lens = l.lens; a.Bt = l.Bt; a.L = l.L; a.H = l.H;
        a.Kd = w.Kd; a.Vd = w.Vd; a.back = w.back;
        a.turned = w.turned;
        a.init = w.back ? l.dlast : l.h0;
        a.last = w.back && !w.turned ? l.dh0 : nullptr;
        a.s_add = w.back ? l.scale : 1.0f;
        a.s_out = w.back ? 1.0f : l.scale;
        plan_segments(l.Bt, l.L, l.H, w.Vd, &a.nseg, &a.seg_steps);
        a.segs = l.scratch;
        if (w.heads == l.H) {
            a.out = w.out;
            walk<E, E>(a, s);
        } else {
            const int64_t states = a.nseg > 1 ? l.Bt * l.H * a.nseg * l.K * l.V : 0;
            float* part = l.scratch + states;
            a.out = part;
            walk<E, F32>(a, s);
            const int64_t n = l.Bt * l.L * w.heads * w.Vd / 4;
            if (n) attention_groups_kernel<E><<<dim3(blocks_for(n, 256)), dim3(256), 0, s>>>(part, w.out, n, l.H / w.heads, w.Vd);
        }
    }
}

}  // namespace

int64_t attn_fwd_scratch(int64_t Bt, int64_t L, int H, int K, int V) {
    int nseg;
    int64_t steps;
    plan_segments(Bt, L, H, V, &nseg, &steps);
    return nseg > 1 ? Bt * H * nseg * K * V : 0;
}

int64_t attn_bwd_scratch(int64_t Bt, int64_t L, int H, int Hq, int Hk, int Hv, int K, int V) {
    int64_t most = 0;
    for (const auto& w : {std::pair<int, int>{Hq, K}, {Hk, K}, {Hv, V}}) {
        int nseg;
        int64_t steps;
        plan_segments(Bt, L, H, w.second, &nseg, &steps);
        const int64_t n = (nseg > 1 ? Bt * H * nseg * K * V : 0) + (w.first < H ? Bt * L * H * w.second : 0);
        most = std::max(most, n);
    }
    return most;
}

hipError_t launch_attn_fwd(const AttnLaunch& l, hipStream_t s) {
    AArgs a{};
    a.q = {l.q, l.Hq}; a.k = {l.k, l.Hk}; a.v = {l.v, l.Hv}; a.rate = l.rate; a.lens = l.lens; a.init = l.h0;
    a.last = l.last_state; a.segs = l.scratch; a.out = l.out; a.Bt = l.Bt; a.L = l.L; a.H = l.H; a.Kd = l.K; a.Vd = l.V;
    a.s_add = 1.0f; a.s_out = l.scale;
    plan_segments(l.Bt, l.L, l.H, l.V, &a.nseg, &a.seg_steps);
    if (l.bf16) walk<BF16, BF16>(a, s);
    else walk<F32, F32>(a, s);
    return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnLaunch& l, hipStream_t s) {
    if (l.bf16) backward<BF16>(l, s);
    else backward<F32>(l, s);
    return hipGetLastError();
}

hipError_t launch_attn_update(const AttnUpdateLaunch& l, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(l.Bt * l.H)), block(256);
    if (l.bf16) attention_update_kernel<BF16><<<grid, block, 0, s>>>(l);
    else attention_update_kernel<F32><<<grid, block, 0, s>>>(l);
    return hipGetLastError();
}

}  // namespace mss
