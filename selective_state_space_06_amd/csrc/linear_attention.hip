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
// A block walks a head's sequence, or a segment of it, in chunks of 32 steps.  A wave has 16 value columns and keeps the
// state's rows of these columns in registers (fp32) all along: 32 registers for 128 keys; a block has all columns of the
// head, four waves or eight, so that queries and keys are read once.  Queries, keys and values of a chunk go through LDS;
// the next chunk's are on their way meanwhile, by loads that give 0 outside of the chunk instead of being branched
// around.  The scores of a chunk are made once for the block, a 16 x 16 tile a wave, and shared through LDS; states and
// values pass from product to product in registers: a product's result (lane: a column, four consecutive rows) is the
// next product's operand as it stands, when the other operand's rows are taken in the same order, and what has to be
// turned is read from LDS by the instruction that turns.
//
// What bounds it: neither memory nor the matrix cores, but the instructions of a chunk and their waits, 2.7 us for 32 steps
// with 128 x 128 state (343 VALU instructions a wave, 55 of them MFMA, 79 SALU, 40 LDS), of which decaying the state, cutting
// it into parts and reading keys turned are most.  So what counts is instructions, and blocks on a CU at once: chunks of 64
// steps have twice the scores' work and fewer fit, chunks of 16 leave half of the matrix instruction empty.  A long sequence
// with few heads is cut into segments; the states between them come from a pass over keys and values alone, whose parts are
// added up by the block that reads them (up to eight) or by a kernel of their own.
// The gradients of shared heads are sums over the heads of a group: a block does as many of them side by side as 16 waves
// hold and adds the outputs up in LDS, in their order; what is left goes through memory and attention_groups_kernel
// (4 x 2048 x 80 heads, of queries and keys 8, when this was built: 553 us for the three gradients, 600 with all through
// memory).
//
// bf16 products of fp32 values: a value is cut into bf16 parts (hi = bf16(x), mid = bf16(x - hi), ...), each exact,
// and the products of parts that matter are summed in fp32.  bf16 inputs are one part; states, scores and the decayed values
// that enter the state are taken in three (2^-25): fp32's precision, so that terms that cancel leave what they do in fp32
// (states and scores in two parts: 4 x 2048 x 32 heads of 128 x 128 bf16 7% faster, and 2^-17 of the terms off).
// fp32 inputs are three parts everywhere, with the six products down to 2^-24 (2.7 times the rate of the fp32 matrix
// instruction).
//
// Measured, on several cards: 4 x 2048 x 32 heads of 128 x 128 bf16 107 to 112 us (2.5 TB/s, 157 TFLOP/s of the formula's
// products), of them states 24; 1 x 32768 x 16 heads of 64 x 64 f32, keys and values of 4, 160 to 166 us, of them states 48 and
// their sums 9; output and gradients of 4 x 2048 x 80 heads of 128 x 64 bf16 with queries and keys of 8 heads 602 us, of
// 3 x 1531 x 12 heads of 64 x 96 f32 170 to 180.
#include <algorithm>

#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"

namespace mss {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
    float* parts;            // (Bt, H, nparts, Kd, Vd): what the parts of all segments but the last add to the state
    void* out;               // (Bt, L, outs, Vd)
    int64_t Bt, L;
    int H, Kd, Vd;
    int each, outs;          // heads of a group, whose outputs are summed (1: none are); outputs: H, or groups times the
                             // blocks of a group
    int nseg, nparts;        // segments; parts of them: `cuts` to each but the last
    int cuts;
    int64_t part_steps;      // a multiple of 64
    float s_add, s_out;      // factors of what enters the state, and of the outputs
    bool turned;             // init and last are (Vd, Kd)
    bool back;               // rows in reverse order
};
constexpr int kMostWalks = 3;
struct Walks {  // of one launch: those of the same sizes side by side, so that there are blocks for every CU
    AArgs w[kMostWalks];
    int64_t each;  // sets of blocks of a walk (attention_join_kernel: blocks)
    int count;
    int set;       // blocks of a set: neighbouring heads of a segment
};
// Blocks go to the eight XCDs in turn, each with an L2 of its own.  A set's blocks, which share rows of queries, keys or
// values, go to one: 4 x 2048 x 80 heads of 128 x 64 bf16, queries and keys of 8 heads, reads 153 MB instead of 389, the
// states of 16 heads with keys and values of 4 (f32) 65 instead of 260; the Infinity Cache had hidden most of that (450 -> 442
// us for the former's gradients, 167 -> 163 for the latter).
constexpr int kXcds = 8;

constexpr int kFold = 8;  // more parts than these are joined by a kernel of their own
constexpr int kChunk = 32;  // steps
constexpr float kMostRate = 200.0f;  // from there on l^n is 0 in fp32 for every n but 0, also for a rate of infinity

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

// x minus the low or the high half of a word of two bf16: exact, and one instruction.  The factors (-1, 0) and (0, -1) are
// kept in registers: as an inline constant of the instruction, -1.0 is not the pair that the compiler takes it for.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float less_half(float x, uint32_t w, uint32_t factors) {
    asm("" : "+s"(factors));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, factors), x, false);
}
__device__ __forceinline__ float less_lo(float x, uint32_t w) { return less_half(x, w, 0x0000BF80u); }
__device__ __forceinline__ float less_hi(float x, uint32_t w) { return less_half(x, w, 0xBF800000u); }
// M pairs of floats as N words of bf16 parts each; r is left with what the parts lack.
template <int N, int M>
__device__ __forceinline__ void cut_words(float* r, uint32_t (*w)[M]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < M; ++e) {
            w[n][e] = pack_bf16x2(r[2 * e], r[2 * e + 1]);
            if (n + 1 < N) {
                r[2 * e] = less_lo(r[2 * e], w[n][e]);
                r[2 * e + 1] = less_hi(r[2 * e + 1], w[n][e]);
            }
        }
}
// Eight floats as N bf16 parts.
template <int N>
__device__ __forceinline__ void cut(float* x, s16x8* part) {
    uint32_t w[N][4];
    cut_words<N, 4>(x, w);
#pragma unroll
    for (int n = 0; n < N; ++n) part[n] = __builtin_bit_cast(s16x8, make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]));
}

template <class E>
struct Form;
template <>
struct Form<BF16> {
    static constexpr int NP = 1, NS = 3;  // parts of inputs; of states and scores
};
template <>
struct Form<F32> {
    static constexpr int NP = 3, NS = 3;
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

// N tiles of such sums, part by part: products that follow each other do not wait for each other.
template <int N, int NA, int NB, class A, class B>
__device__ __forceinline__ void mma_each(A a, B b, f32x4* c) {
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j < most) {
#pragma unroll
                for (int n = 0; n < N; ++n) c[n] = mma(a(n)[i], b(n)[j], c[n]);
            }
}

// The LDS reads before this are issued before what comes after it (the compiler would issue each in front of its use).
__device__ __forceinline__ void issue_reads() { __builtin_amdgcn_sched_barrier(0); }

// What a state decays by in some steps: l^n where that is under 1/2, l^n - 1 otherwise.  Near 1 the power's own rounding would be
// the same for every chunk and add up; far from 1 a rounding of l^n - 1 is one of the undecayed state, and 6% of what is left
// at a rate of 1/2 and 32 steps.
struct Decay {
    float by;
    int whole;  // by is l^n itself
};
__device__ __forceinline__ float decayed(float x, Decay d) { return d.whole ? x * d.by : fmaf(x, d.by, x); }
__device__ __forceinline__ Decay decay_of(float d, float lost) {
    const bool whole = d > kLn2;
    return {whole ? exact_exp(-d, -lost) : expm1f(-d), whole};
}
// Of the steps that a state decays by in part i of a sequence of len steps.
__device__ __forceinline__ Decay part_decay(const AArgs& a, float rate, int64_t len, int i) {
    int64_t n = len - i * a.part_steps;
    n = n < 0 ? 0 : n < a.part_steps ? n : a.part_steps;
    if (n > 0 && i == 0 && a.back) --n;
    const double exact = static_cast<double>(rate) * static_cast<double>(n);
    const float d = static_cast<float>(exact);
    return decay_of(d, static_cast<float>(exact - d));
}

// Waves a SIMD that a kernel's registers leave room for: as many as its LDS does.
constexpr int waves_wanted(bool bf16, int KD, int NW, bool states) {
    return bf16 ? 4 : !states && KD == 64 && NW == 4 ? 3 : KD == 128 && NW == 4 ? (states ? 2 : 1) : states && KD == 64 ? 4 : 2;
}

// STATES: only the state that a part of a segment adds, from zero.  OUT: the outputs' type.  NW: waves, 16 columns each.
// SUB: heads of a group that a block does side by side, NW waves each, and whose outputs it sums.
template <class E, class OUT, int KD, int NW, int SUB, bool STATES>
__global__ __launch_bounds__(64 * NW * SUB, waves_wanted(Form<E>::NP == 1, KD, NW, STATES)) void attention_kernel(Walks all) {
    const uint32_t turn = blockIdx.x / kXcds, in_set = turn % static_cast<uint32_t>(all.set);
    const uint32_t set = turn / static_cast<uint32_t>(all.set) * kXcds + blockIdx.x % kXcds, walk = set / static_cast<uint32_t>(all.each);
    if (walk >= static_cast<uint32_t>(all.count)) return;  // (sets are not always a multiple of kXcds)
    const AArgs& a = all.w[walk];
    using F = Form<E>;
    using O = typename OUT::storage;
    constexpr int C = kChunk, NP = F::NP, NS = F::NS, MT = C / 16, M2 = C / 32, KJ = KD / 32, KT = KD / 16;
    constexpr int T = 64 * NW, VT = 16 * NW;                 // threads and columns of a block
    // Elements between two rows in LDS, which has 64 banks of four bytes.  Rows that lanes read 16 bytes of (queries, scores)
    // lie an odd multiple of eight banks apart (1 KB in 4.4 cycles; 8.4 at four banks).  Rows read turned, and rows of both
    // uses, also have their columns moved by bits of the row (key_at, value_at), so that the eight rows of 16 columns that 32
    // lanes read turned, and the 16 rows of 4 that they read for scores, meet in no bank.
    // (fp32 with 64 keys and four waves: rows close enough for three blocks on a CU; the gradients of 4 x 2048 x 24 heads of
    // 64 x 64 177 -> 169 us.)
    constexpr bool kClose = NP == 3 && KD == 64 && NW == 4;
    constexpr int QS = KD + 16, KS = kClose ? KD + 16 : KD + 32, VS = VT + 16, PS = kClose ? C + 8 : C + 16;
    constexpr int QU = KD / 8, VU = VT / 8;                  // units of eight elements a row
    constexpr int QR = T / QU, VR = T / VU;                  // rows that the block loads at once
    constexpr int NQ = C > QR ? C / QR : 1, NV = C / VR;     // (f32 with 64 keys: half of eight waves load them)
    constexpr int ES = sizeof(typename E::storage);
    __shared__ __align__(16) uint16_t all_qs[SUB][STATES ? 1 : NP][STATES ? 1 : C][STATES ? 8 : QS];
    __shared__ __align__(16) uint16_t all_ks[SUB][NP][C][KS];
    __shared__ __align__(16) uint16_t all_vs[SUB][NP][C][VS];
    __shared__ __align__(16) uint16_t all_ps[SUB][STATES ? 1 : NS][STATES ? 1 : C][STATES ? 8 : PS];  // scores, a step's in a row
    __shared__ f32x4 others[SUB > 1 ? SUB - 1 : 1][MT][SUB > 1 ? T : 1];  // outputs of the heads but the first

    const int tid = SUB > 1 ? threadIdx.x % T : threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int sub = SUB > 1 ? __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / T)) : 0;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto& qs = all_qs[sub];
    auto& ks = all_ks[sub];
    auto& vs = all_vs[sub];
    auto& ps = all_ps[sub];
    const int outs = STATES ? a.H : a.outs, nseg = STATES ? a.nparts : a.nseg;
    const uint32_t of_walk = set % static_cast<uint32_t>(all.each), of_seg = of_walk / static_cast<uint32_t>(nseg),
                   sets = static_cast<uint32_t>(outs) / static_cast<uint32_t>(all.set);  // of a batch's segment
    const int64_t b = of_seg / sets;
    const int o_head = static_cast<int>(of_seg % sets * all.set + in_set), seg = static_cast<int>(of_walk % static_cast<uint32_t>(nseg));
    // (a group's last block may have fewer heads: the others of its waves go along with nothing)
    const int in_group = SUB > 1 ? o_head % ((a.each + SUB - 1) / SUB) * SUB + sub : 0;
    const bool there = SUB == 1 || in_group < a.each;
    const int h = SUB == 1 ? o_head : o_head / ((a.each + SUB - 1) / SUB) * a.each + (there ? in_group : 0);
    const int64_t bh = b * a.H + h;
    const int given = a.lens ? __builtin_amdgcn_readfirstlane(a.lens[b]) : 0;
    const int64_t len = a.lens ? (given < 0 ? 0 : given < a.L ? given : a.L) : a.L;
    const int64_t steps = STATES ? a.part_steps : a.part_steps * a.cuts, from = seg * steps,
                  to = from + steps < a.L ? from + steps : a.L;
    const int64_t stop = to < len ? to : len;                // rows past it are 0
    const int v0 = wave * 16;                                // this wave's columns
    const bool mine = v0 < a.Vd && there;                    // others go along with zeros

    // Rows of a chunk in the order of the walk: row r is token at + r, or, walked backwards, len - 1 - at - r.  A chunk of n
    // rows of a tensor is a buffer that begins at its lowest token; a thread's place in it is an offset.  Rows behind the
    // end and columns beside the head's lie outside of it, where loads give 0 and stores do nothing.  The buffers move from
    // chunk to chunk by whole rows: addresses made anew for each were a third of a chunk's instructions.
    const bool back = a.back;
    const int todo = stop > from ? static_cast<int>(stop - from) : 0;  // rows of this segment
    const int64_t token0 = b * a.L + (back ? len - from - (todo < C ? todo : C) : from);
    const auto start_of = [&](const void* t, int heads, int head, int dim, int size) MSS_INLINED {
        return static_cast<const char*>(t) + (token0 * heads + head) * dim * static_cast<int64_t>(size);
    };
    constexpr uint32_t kOutside = 0x80000000u;  // no chunk is as large
    const auto offset_of = [&](int row, int row_bytes, int col, bool in, int size) MSS_INLINED {
        return in ? static_cast<uint32_t>((back ? C - 1 - row : row) * row_bytes + col * size) : kOutside;
    };
    const auto move = [&](const char*& p, int row_bytes, int n) MSS_INLINED {  // to the next chunk, of n rows
        p += static_cast<int64_t>((back ? -n : C) * row_bytes);
    };
    const auto buffer_at = [](const char* p, int bytes) MSS_INLINED {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, bytes, 0x00027000);
    };
    const int q_row = tid / QU, q_col = tid % QU * 8, v_row = tid / VU, v_col = tid % VU * 8;
    const int q_bytes = a.q.heads * a.Kd * ES, k_bytes = a.k.heads * a.Kd * ES, v_bytes = a.v.heads * a.Vd * ES,
              o_bytes = a.outs * a.Vd * static_cast<int>(sizeof(O));
    const bool q_in = q_col < a.Kd && q_row < C, v_in = v_col < a.Vd;
    const uint32_t q_off = offset_of(q_row, q_bytes, q_col, q_in, ES), k_off = offset_of(q_row, k_bytes, q_col, q_in, ES),
                   v_off = offset_of(v_row, v_bytes, v_col, v_in, ES),
                   o_off = offset_of(r16, o_bytes, v0 + 4 * g, mine, sizeof(O));

    const char* q_at = start_of(a.q.p, a.q.heads, h / (a.H / a.q.heads), a.Kd, ES);
    const char* k_at = start_of(a.k.p, a.k.heads, h / (a.H / a.k.heads), a.Kd, ES);
    const char* v_at = start_of(a.v.p, a.v.heads, h / (a.H / a.v.heads), a.Vd, ES);
    const char* o_at = start_of(a.out, a.outs, o_head, a.Vd, sizeof(O));

    Raw<E> rq[STATES ? 1 : NQ], rk[NQ], rv[NV];
    const auto load = [&](int n) MSS_INLINED {
        const int rows_there = there ? n : 0, missing = back ? C - n : 0;
        const auto rows = [&](const char* at, int row_bytes, uint32_t off, int step, auto& r) MSS_INLINED {
            const auto p = buffer_at(at, rows_there * row_bytes);
            off -= missing * row_bytes;
            const int next = (back ? -step : step) * row_bytes;
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(r) / sizeof(r[0])); ++j)
#pragma unroll
                for (int i = 0; i < kE / E::kPerVec; ++i)
                    r[j].q[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(p, off + j * next + 16 * i, 0, 0));
        };
        if constexpr (!STATES) rows(q_at, q_bytes, q_off, QR, rq);
        rows(k_at, k_bytes, k_off, QR, rk);
        rows(v_at, v_bytes, v_off, VR, rv);
    };
    // Powers of the decay.  A score's lane is a step t = 16 tb + r16, its rows are s = 16 ta + 4 g + i.
    const float rate = fminf(fmaxf(a.rate[h], 0.0f), kMostRate);
    const auto power = [&](int n) MSS_INLINED {
        const float steps = static_cast<float>(n), d = rate * steps;
        return exact_exp(-d, -fmaf(rate, steps, -d));
    };
    // fp32 values that only enter the state are weighed where they are cut into parts, not joined, weighed and cut again
    // (1 x 32768 x 16 heads of 64 x 64: 163 -> 157 us).
    constexpr bool kWeighed = STATES && NP > 1;
    float weights[kWeighed ? NV : 1];
    if constexpr (kWeighed) {
#pragma unroll
        for (int j = 0; j < NV; ++j) weights[j] = power(C - 1 - v_row - j * VR) * a.s_add;
    }
    const auto put = [&](const Raw<E>& r, float weight, int plane, auto write) MSS_INLINED {
        if constexpr (NP == 1) {
            write(r.q[0], 0);
        } else {
            float x[kE];
            r.unpack(x);
            if constexpr (kWeighed) {
#pragma unroll
                for (int e = 0; e < kE; ++e) x[e] *= weight;
            }
            s16x8 part[NP];
            cut<NP>(x, part);
#pragma unroll
            for (int n = 0; n < NP; ++n) write(__builtin_bit_cast(uint4, part[n]), n * plane);
        }
    };
    const auto put8 = [&](const Raw<E>& r, uint16_t* p, int plane, float weight = 1.0f) MSS_INLINED {
        put(r, weight, plane, [&](uint4 q, int to) MSS_INLINED { *reinterpret_cast<uint4*>(p + to) = q; });
    };
    const auto put4 = [&](const Raw<E>& r, uint16_t* lo, uint16_t* hi, int plane) MSS_INLINED {
        put(r, 1.0f, plane, [&](uint4 q, int to) MSS_INLINED {
            *reinterpret_cast<uint2*>(lo + to) = make_uint2(q.x, q.y);
            *reinterpret_cast<uint2*>(hi + to) = make_uint2(q.z, q.w);
        });
    };
    const auto key_at = [](int row, int col) MSS_INLINED { return col ^ (row & 8) >> 1 ^ (row & 4) << 2; };
    const auto value_at = [](int row, int col) MSS_INLINED { return col ^ (row & 8) * (VT / 32); };
    const auto store = [&](int n) MSS_INLINED {
        if (QR <= C || q_row < C) {
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                const int row = q_row + j * QR;
                if constexpr (!STATES) put8(rq[j], &qs[0][row][q_col], C * QS);
                put4(rk[j], &ks[0][row][key_at(row, q_col)], &ks[0][row][key_at(row, q_col + 4)], C * KS);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int row = v_row + j * VR;
            float weight = 1.0f;
            if constexpr (kWeighed) weight = n == C ? weights[j] : power(n - 1 - row > 0 ? n - 1 - row : 0) * a.s_add;
            put8(rv[j], &vs[0][row][value_at(row, v_col)], C * VS, weight);
        }
    };
    // eight values of a column, rows 32 m + 8 g ...
    const auto read_values = [&](int m, s16x8* f) MSS_INLINED {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const uint16_t* s = &vs[p][32 * m + 8 * g + (r16 >> 2)][value_at(8 * g, v0 + 4 * (r16 & 3))];
            f[p] = join8(turn4(s), turn4(s + 4 * VS));
        }
    };

    const auto uniform = [](float x) MSS_INLINED {
        return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
    };
    float small[8];  // l^0 .. l^7, in scalar registers: the powers of a lane's rows are products of one of its own and these
#pragma unroll
    for (int e = 0; e < 8; ++e) small[e] = uniform(power(e));
    // The scores of a chunk are three tiles, one to each of the first three waves: (ta, tb) = (0, 0), (0, 1), (1, 1).
    static_assert(MT == 2 && NW >= 3, "a wave has at most one tile of scores");
    const int ta = wave >> 1, tb_of_wave = (wave + 1) >> 1;
    float decay[4];  // of this wave's tile
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int steps = 16 * (tb_of_wave - ta) + r16 - 4 * g - i;
        decay[i] = power(steps > 0 ? steps : 0) * (a.s_add * a.s_out);
    }
    const float since = power(r16) * a.s_out, tail = power(24 - 8 * g) * a.s_add, step16 = uniform(power(16));
    const float tail32 = uniform(power(32));
    const auto decay_over = [&](int n) MSS_INLINED {  // the same for all lanes
        const float steps = static_cast<float>(n), d = rate * steps;
        const Decay gone = decay_of(d, fmaf(rate, steps, -d));
        return Decay{uniform(gone.by), __builtin_amdgcn_readfirstlane(gone.whole)};
    };
    // l^C as a float and what that lacks.  Chunks decay by the float; what it lacks is owed, and goes into the factor of a
    // later chunk once it is a step of it: a rounding that is the same for every chunk would add up.  (A branch between the two
    // forms of Decay parts the factors from the products behind them: 4 x 2048 x 32 heads of 128 x 128 bf16 3% slower.)
    const Decay of_chunk = decay_over(C);
    const float chunk_kept = of_chunk.whole ? of_chunk.by : 1.0f + of_chunk.by;
    const float chunk_rest = of_chunk.whole ? 0.0f : of_chunk.by - (chunk_kept - 1.0f);
    float owed = 0.0f;
    // The state: tile j holds rows 32 (j / 2) + 8 g + 4 (j % 2) + i of a column, so that two tiles are eight rows in turn.
    f32x4 st[KT];
    const int64_t per = static_cast<int64_t>(a.Kd) * a.Vd;
    // every element of the state that there is, with its place in memory (turned: (Vd, Kd))
    const auto each_of_state = [&](bool turned, auto f) MSS_INLINED {
        const int nk = turned ? 1 : a.Vd, nv = turned ? a.Kd : 1;
        const int lane_at = 8 * g * nk + (v0 + r16) * nv;
        if (!mine) return;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            if (32 * j + 8 * g >= a.Kd) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                st[2 * j + i / 4][i % 4] = f(st[2 * j + i / 4][i % 4], lane_at + (32 * j + i) * nk);
        }
    };
#pragma unroll
    for (int j = 0; j < KT; ++j) st[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // where a lane reads keys turned: four rows from 8 g, and the four behind them, in a tile of either kind
    const uint16_t* turned[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * g + (r16 >> 2) + 4 * (i % 2);
        turned[i / 2][i % 2] = &ks[0][row][key_at(row, 8 * (r16 & 3) + 4 * (i / 2))];
    }
    const auto rows_at = [&](int at) MSS_INLINED {  // of a chunk (the compiler takes the vector unit's median for it)
        return __builtin_amdgcn_readfirstlane(todo - at < 0 ? 0 : todo - at < C ? todo - at : C);
    };
    load(rows_at(0));
    if constexpr (!STATES) {
        // the state before the segment: what the join kernel made of it, or the first one and what the parts before add
        const bool joined = a.nparts > kFold && seg > 0;
        for (int i = joined ? seg * a.cuts - 1 : -1; i < seg * a.cuts; ++i) {
            const float* p = i < 0 ? a.init + bh * per : a.parts + (bh * a.nparts + i) * per;
            const Decay gone = i < 0 || joined ? Decay{0.0f, 0} : part_decay(a, rate, len, i);
            if (i >= 0 || a.init)
                each_of_state(i < 0 && a.turned, [&](float x, int j) MSS_INLINED { return decayed(x, gone) + p[j]; });
        }
        // scores behind a step stay 0: only the others are written
        for (int e = tid; e < NS * C * PS / 8; e += T) reinterpret_cast<uint4*>(&ps[0][0][0])[e] = make_uint4(0, 0, 0, 0);
    }

    const auto write = [&](int n, const f32x4* acc) MSS_INLINED {
        const auto o = buffer_at(o_at, n * o_bytes);
        const uint32_t first = o_off - (back ? C - n : 0) * o_bytes;
#pragma unroll
        for (int tb = 0; tb < MT; ++tb) {
            const uint32_t off = first + (back ? -16 : 16) * tb * o_bytes;
            const f32x4 x = acc[tb];
            if constexpr (sizeof(O) == 2)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])}, o, off, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), o, off, 0, 0);
        }
    };
    // what the state's part of an output decays by; walked backwards, the state enters the sequence's first row undecayed
    const bool keep = !STATES && a.last && seg == a.nseg - 1;
    int early = back && from == 0 ? 1 : 0;
    float faded = since * power(1 - early);
    for (int at = 0; at < todo; at += C) {
        const int n = rows_at(at), ahead = rows_at(at + C);
        store(n);
        move(q_at, q_bytes, ahead);
        move(k_at, k_bytes, ahead);
        move(v_at, v_bytes, ahead);
        __syncthreads();
        load(ahead);
        s16x8 vf[M2][NP];
        f32x4 acc[MT];
        if constexpr (!STATES) {
            if (wave < 3) {  // scores
                constexpr int G = NP == 1 && NW == 4 ? 2 : KJ;  // as many at once as registers hold
                f32x4 p4 = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j0 = 0; j0 < KJ; j0 += G) {
                    s16x8 qf[G][NP], kf[G][NP];
#pragma unroll
                    for (int j = 0; j < G; ++j)
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            qf[j][p] = *reinterpret_cast<const s16x8*>(&qs[p][16 * tb_of_wave + r16][32 * (j0 + j) + 8 * g]);
                            const uint16_t* row = ks[p][16 * ta + r16] + 32 * (j0 + j);  // (key_at moves columns within 32)
                            kf[j][p] = join8(*reinterpret_cast<const s16x4*>(row + key_at(r16, 8 * g)),
                                             *reinterpret_cast<const s16x4*>(row + key_at(r16, 8 * g + 4)));
                        }
                    issue_reads();
#pragma unroll
                    for (int j = 0; j < G; ++j) p4 = mma_parts<NP, NP>(kf[j], qf[j], p4);
                }
                uint32_t w[NS][2];
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = wave == 1 || r16 >= 4 * g + i ? p4[i] * decay[i] : 0.0f;
                cut_words<NS, 2>(x, w);
#pragma unroll
                for (int p = 0; p < NS; ++p)
                    *reinterpret_cast<uint2*>(&ps[p][16 * tb_of_wave + r16][16 * ta + 4 * g]) = make_uint2(w[p][0], w[p][1]);
            }
            // what the state before the chunk gives: rows of a tile are columns v, lanes are steps t
#pragma unroll
            for (int tb = 0; tb < MT; ++tb) acc[tb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            constexpr int B = SUB == 1 && (NP > 1 || NW == 8 || KD == 64) ? 2 : 1;  // 2: the next step's are read ahead
            s16x8 qf[B][MT][NP];
            const auto read_queries = [&](int j) MSS_INLINED {
#pragma unroll
                for (int tb = 0; tb < MT; ++tb)
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        qf[j % B][tb][p] = *reinterpret_cast<const s16x8*>(&qs[p][16 * tb + r16][32 * j + 8 * g]);
                issue_reads();
            };
            if (B == 2) read_queries(0);
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                if (B == 1 || j + 1 < KJ) read_queries(j + B - 1);
                s16x8 sf[NS];
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = st[2 * j][i], x[4 + i] = st[2 * j + 1][i];
                cut<NS>(x, sf);
                mma_each<MT, NS, NP>([&](int) MSS_INLINED { return sf; }, [&](int tb) MSS_INLINED { return qf[j % B][tb]; }, acc);
            }
#pragma unroll
            for (int tb = 0; tb < MT; ++tb) acc[tb] *= tb ? faded * step16 : faded;
            __syncthreads();
#pragma unroll
            for (int m = 0; m < M2; ++m) {
                read_values(m, vf[m]);
#pragma unroll
                for (int j = NS - 1; j >= 0; --j) {
                    s16x8 pf[MT];
#pragma unroll
                    for (int tb = 2 * m; tb < MT; ++tb)
                        pf[tb] = *reinterpret_cast<const s16x8*>(&ps[j][16 * tb + r16][32 * m + 8 * g]);
                    issue_reads();
#pragma unroll
                    for (int i = NP - 1; i >= 0; --i)
#pragma unroll
                        for (int tb = 2 * m; tb < MT; ++tb)
                            if (i + j < NS) acc[tb] = mma(vf[m][i], pf[tb], acc[tb]);
                }
            }
            if (SUB == 1) write(n, acc);
            else if (sub > 0) {
#pragma unroll
                for (int tb = 0; tb < MT; ++tb) others[sub - 1][tb][tid] = acc[tb];
            }
        } else {
#pragma unroll
            for (int m = 0; m < M2; ++m) read_values(m, vf[m]);
        }
        // the state after the chunk, if it is read
        if (STATES || ahead || keep) {
            float kept;  // l^n
            if (n - early == C) {
                owed += chunk_rest;
                kept = chunk_kept + owed;
                owed -= kept - chunk_kept;
            } else {
                const Decay gone = decay_over(n - early);
                kept = gone.whole ? gone.by : 1.0f + gone.by;
            }
#pragma unroll
            for (int j = 0; j < KT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) st[j][i] *= kept;
#pragma unroll
            for (int m = 0; m < M2; ++m) {
                s16x8 wf[3];
                if constexpr (kWeighed) {
#pragma unroll
                    for (int p = 0; p < 3; ++p) wf[p] = vf[m][p];
                } else {
                    float w[8], x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = (m + 1 < M2 ? tail * tail32 : tail) * small[7 - e];
                    if (n < C) {  // rows past the end are zeros
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int s = n - 1 - (32 * m + 8 * g + e);
                            w[e] = power(s > 0 ? s : 0) * a.s_add;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = bf16_to_f32(static_cast<uint16_t>(vf[m][0][e]));
#pragma unroll
                        for (int p = 1; p < NP; ++p) x[e] += bf16_to_f32(static_cast<uint16_t>(vf[m][p][e]));
                        x[e] *= w[e];
                    }
                    cut<3>(x, wf);
                }
                constexpr int G = NP == 1 && SUB == 4 ? 2 : 4;  // tiles at once
#pragma unroll
                for (int j0 = 0; j0 < KT; j0 += G) {
                    s16x8 kt[G][NP];
#pragma unroll
                    for (int j = 0; j < G; ++j)
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            const int to = (p * C + 32 * m) * KS + 16 * ((j0 + j) & ~1);
                            kt[j][p] = join8(turn4(turned[j % 2][0] + to), turn4(turned[j % 2][1] + to));
                        }
                    issue_reads();
                    mma_each<G, NP, 3>([&](int j) MSS_INLINED { return kt[j]; }, [&](int) MSS_INLINED { return wf; }, st + j0);
                }
            }
        }
        __syncthreads();
        if (!STATES && SUB > 1 && sub == 0) {  // (the others write theirs again behind two barriers)
#pragma unroll
            for (int x = 0; x < SUB - 1; ++x)
#pragma unroll
                for (int tb = 0; tb < MT; ++tb) acc[tb] += others[x][tb][tid];
            write(n, acc);
        }
        move(o_at, o_bytes, ahead);
        if (early) {
            early = 0;
            faded = since * power(1);
        }
    }
    if (!mine) return;
    if constexpr (STATES) {
        float* p = a.parts + (bh * a.nparts + seg) * per;
        each_of_state(false, [&](float x, int i) MSS_INLINED { return p[i] = x; });
    } else {
        for (int64_t t = (from > len ? from : len) + r16; t < to && sub == 0; t += 16) {  // past the end
            char* p = static_cast<char*>(a.out) + (((b * a.L + t) * a.outs + o_head) * a.Vd + v0 + 4 * g) * static_cast<int64_t>(sizeof(O));
            if (sizeof(O) == 2) *reinterpret_cast<uint2*>(p) = make_uint2(0, 0);
            else *reinterpret_cast<f32x4*>(p) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if (keep) {
            // walked backwards, the state is that of the first step: the one before it is a step further
            const float f = back && len > 0 ? power(1) : 1.0f;
            float* p = a.last + bh * per;
            each_of_state(a.turned, [&](float x, int i) MSS_INLINED { return p[i] = x * f; });
        }
    }
}

// The states that enter the segments but the first, from what the parts add, in place (in the last part of the segment
// before): a block per (batch, head) and 256 elements.  The parts' decays are made once for the block, not by every thread.
__global__ __launch_bounds__(256) void attention_join_kernel(Walks all, int blocks) {
    __shared__ Decay gone[256];
    const AArgs& a = all.w[blockIdx.x / all.each];
    const int64_t block = blockIdx.x % all.each, bh = block / blocks, b = bh / a.H;
    const int per = a.Kd * a.Vd, x = static_cast<int>(block % blocks) * 256 + threadIdx.x;
    const int64_t len = a.lens ? (a.lens[b] < 0 ? 0 : a.lens[b] < a.L ? a.lens[b] : a.L) : a.L;
    const float rate = fminf(fmaxf(a.rate[bh % a.H], 0.0f), kMostRate);
    float s = 0.0f;
    if (a.init && x < per) s = a.init[bh * per + (a.turned ? x % a.Vd * a.Kd + x / a.Vd : x)];
    float* o = a.parts + bh * a.nparts * per + (x < per ? x : 0);
    constexpr int G = 16;  // on their way at once
    int left = a.cuts;     // parts of this segment: the last gives the next one's state, the others what no one reads
    for (int i0 = 0; i0 < a.nparts; i0 += G) {
        if (i0 % 256 == 0) {
            __syncthreads();
            if (i0 + static_cast<int>(threadIdx.x) < a.nparts) gone[threadIdx.x] = part_decay(a, rate, len, i0 + threadIdx.x);
            __syncthreads();
        }
        float adds[G];
#pragma unroll
        for (int i = 0; i < G; ++i) adds[i] = o[static_cast<int64_t>(i0 + i < a.nparts ? i0 + i : i0) * per];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            if (i0 + i >= a.nparts) break;
            s = decayed(s, gone[(i0 + i) % 256]) + adds[i];
            if (--left == 0) {
                left = a.cuts;
                if (x < per) o[static_cast<int64_t>(i0 + i) * per] = s;
            }
        }
    }
}

// out (rows, groups, dim) = sum over the heads of a group of part (rows, groups, each, dim), in their order.  No one reads the
// parts again: they pass the Infinity Cache by (the gradients of 4 x 2048 x 80 heads of 128 x 64 bf16, queries and keys of 8
// heads: 441 -> 424 us).
template <class E>
__global__ __launch_bounds__(256) void attention_groups_kernel(const float* part, void* out, int64_t n, int each, int dim) {
    // a thread per four elements
    for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < n; e += gridDim.x * 256ll) {
        const int64_t group = e / (dim / 4);
        const int c = static_cast<int>(e % (dim / 4)) * 4;
        const float* p = part + group * each * dim + c;
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < each; ++j) s += __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + static_cast<int64_t>(j) * dim));
        auto* o = static_cast<typename E::storage*>(out) + e * 4;
        if (sizeof(typename E::storage) == 2)
            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
        else *reinterpret_cast<f32x4*>(o) = s;
    }
}

// ---- one token.  A block per (batch, head): a thread holds four columns of every R-th row of the state; the rows'
// parts of the output are summed through LDS.  Bound by memory, the state read and written: 64 x 80 heads of 128 x 64 65 us
// (5.1 TB/s), 59 (5.7) where the state passes the Infinity Cache by.  That is done from kPassBy bytes of it on, of which two
// layers' do not fit the 256 MB anyway (a single state of 168 MB that does fit: 52 us, passing by 58).
constexpr int64_t kPassBy = int64_t{1} << 27;
template <class E, bool PASS>
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
    const Decay gone = decay_of(fminf(fmaxf(a.rate[h], 0.0f), kMostRate), 0.0f);
    f32x4 v, out = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t at = (b * a.Hv + h / (a.H / a.Hv)) * a.V + 4 * c;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = E::load1(a.v, at + i);
    __syncthreads();
    if (r < R) {
        f32x4* s = reinterpret_cast<f32x4*>(a.state + bh * a.K * a.V) + c;
#pragma unroll 8
        for (int k = r; k < a.K; k += R) {
            f32x4 x = PASS ? __builtin_nontemporal_load(s + k * quads) : s[k * quads];
            const float q = qk[0][k], kk = qk[1][k];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = fmaf(kk, v[i], decayed(x[i], gone));
                out[i] = fmaf(q, x[i], out[i]);
            }
            if (PASS) __builtin_nontemporal_store(x, s + k * quads);
            else s[k * quads] = x;
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

// How a sequence is cut.  A block walks a segment in about the same time for every 64 steps (3.5 us with 128 keys), and a CU
// with more than one block takes longer by what they share: measured for c blocks of eight waves 0.9 c, for four waves
// 0.1 + 0.7 c, for 16 waves 1.3; blocks that find no room come after.  The start of a segment is worth one such time.  More
// segments (at most 128) fill the CUs better but need the states between them: a pass over keys and values at 0.6 (eight
// waves) or 0.3 (four) of the walk, and a launch; and then to be added up, a microsecond a part of 128 x 128 state in the
// blocks that read them, or in a launch more.  The pass, whose blocks wait for nothing, is cut further, into parts of 128
// steps or more, up to a block for every CU; the parts are what is added up (priced by segments, 1 x 1000 x 4 heads of
// 64 x 64 f32 28 us instead of 21).
// Times by the number of segments, the one that is taken in brackets: 4 x 2048 x 32 heads of 128 x 128 bf16, 1 to 4: 139,
// [108], 118, 117 us; 4 x 2048 x 80 of 128 x 64 bf16, queries and keys of 8 heads: 155, 143, [135], 146; 3 x 1531 x 12 of
// 64 x 96 f32, 4, 5, 6, 8, 24: 55, 49, [47], 67, 65; 1 x 2048 x 32 of 128 x 128 bf16, keys and values of 8 heads, 4, 6, 8, 16:
// 65, 59, [52], 55.
struct Plan {
    int nseg, nparts, cuts;
    int64_t part_steps, cost;
};
// Blocks that find room on a CU by registers and LDS: 16 waves; in fp32 three blocks of four waves with up to 64 keys, one of any
// other kind.  (Three and not two: gradients of 2 x 4096 x 16 heads of 64 x 64 184 -> 176 us, 6 x 1531 x 50 heads forward 152 ->
// 156.)
int blocks_a_cu(bool bf16, int waves, int Kd) { return bf16 ? 16 / waves : waves == 4 && Kd <= 64 ? 3 : 1; }
// Parts of each segment but the last: as many as give a block for every CU, of 128 steps or more.
int cuts_of(int64_t heads, int64_t segs, int64_t segment) {
    int cuts = 1;
    while (segs > 1 && segment % (2 * cuts) == 0 && segment / (2 * cuts) >= 2 && heads * (segs - 1) * cuts < 256) cuts *= 2;
    return cuts;
}
// blocks: of each segment; heads: whose states are wanted; waves: of a block, of one of those that make states
Plan plan_segments(bool bf16, int Kd, int Vd, int64_t blocks, int64_t heads, int waves, int state_waves, int64_t L) {
    const int64_t steps64 = std::max<int64_t>(1, (L + 63) / 64), most = blocks_a_cu(bf16, waves, Kd);
    const auto time_of = [&](int64_t c) {
        return waves == 16 ? 13 * c : std::max<int64_t>(c > 0 ? 10 : 0, waves == 8 ? 9 * c : 1 + 7 * c);
    };
    int64_t best = 0, segment = 0, each = 0;
    for (int64_t n = 1; n <= std::min<int64_t>(128, steps64); ++n) {
        if ((steps64 + n - 1) / n == each) continue;
        each = (steps64 + n - 1) / n;
        const int64_t segs = (steps64 + each - 1) / each;  // of 64 steps, and how many there are
        const int64_t c = (blocks * segs + 255) / 256;
        int64_t cost = (c / most * time_of(most) + (c % most ? time_of(c % most) : 0)) * (each + 1);
        if (segs > 1) {
            const int64_t parts = (segs - 1) * cuts_of(heads, segs, each);
            cost += (state_waves == 8 ? 6 : 3) * heads * (segs - 1) * each / 256 + 15;
            cost += parts <= kFold ? 3 * parts * Kd * Vd / (128 * 128) : 13;
        }
        if (n == 1 || cost < best) best = cost, segment = each;
    }
    Plan p;
    p.cost = best;
    p.nseg = static_cast<int>((steps64 + segment - 1) / segment);
    p.cuts = cuts_of(heads, p.nseg, segment);
    p.part_steps = segment * 64 / p.cuts;
    p.nparts = (p.nseg - 1) * p.cuts;
    return p;
}
// Columns of a block.
int columns(int Vd) { return Vd > 64 ? 128 : 64; }
// Heads of a group that a block does: 16 waves of bf16's kernels find room on a CU, eight of fp32's smallest.
constexpr int heads_at_once(bool bf16, int KD, int NW) { return bf16 ? 16 / NW : KD == 64 && NW == 4 ? 2 : 1; }

// Sizes of the walks of a launch.
struct Sizes {
    bool bf16;
    int64_t Bt, L;
    int H, outs, each, Kd, Vd, count;
    int waves() const {
        const int w = columns(Vd) / 16;
        return each > 1 ? w * heads_at_once(bf16, Kd <= 64 ? 64 : 128, w) : w;
    }
    Sizes of(int64_t batches) const {
        Sizes s = *this;
        s.Bt = batches;
        return s;
    }
};
Plan plan_walks(const Sizes& z) {
    return plan_segments(z.bf16, z.Kd, z.Vd, z.Bt * z.outs * z.count, z.Bt * z.H * z.count, z.waves(), columns(z.Vd) / 16, z.L);
}
// Batches of a first launch: all, or as many as fill the CUs in whole rounds, when the others, cut finer, are done sooner in
// one of their own than as the rest of a round (320 blocks of 16 waves, twice in the gradients
// of 4 x 2048 x 80 heads of 128 x 64 bf16, queries and keys of 8: 468 us, 535 in one launch each).
int64_t first_batches(const Sizes& z) {
    const int64_t blocks = z.outs * z.count, room = 256 * blocks_a_cu(z.bf16, z.waves(), z.Kd);
    const int64_t first = z.Bt * blocks / room * room / blocks;
    if (first < 1 || first == z.Bt) return z.Bt;
    return plan_walks(z.of(first)).cost + plan_walks(z.of(z.Bt - first)).cost + 15 < plan_walks(z).cost ? first : z.Bt;
}
int64_t state_floats(const Sizes& z) {
    const int64_t first = first_batches(z), rest = z.Bt - first;
    int64_t n = first * plan_walks(z.of(first)).nparts;
    if (rest) n = std::max(n, rest * plan_walks(z.of(rest)).nparts);
    return z.count * n * z.H * z.Kd * z.Vd;
}

template <class E, class OUT, int KD, int NW>
void walk_waves(Walks& w, int count, hipStream_t s) {
    constexpr int SUB = heads_at_once(Form<E>::NP == 1, KD, NW);
    const AArgs& a = w.w[0];
    const dim3 block(64 * NW);
    w.count = count;
    // sets of `share` blocks, or of a divisor of it if their number would leave XCDs idle
    const auto grid = [&](int64_t segs, int heads, int share) {
        const auto rounded = [&](int f) { return (segs * heads / f * count + kXcds - 1) / kXcds * kXcds * f; };
        int f = share;
        while (f > 1 && (share % f || rounded(f) > segs * heads * count * 9 / 8)) --f;
        w.set = f;
        w.each = segs * heads / f;
        return dim3(static_cast<unsigned>(rounded(f)));
    };
    const int share_kv = a.H / std::min(a.k.heads, a.v.heads), share = std::max(share_kv, a.H / a.q.heads);
    if (a.nparts > 0) {
        attention_kernel<E, E, KD, NW, 1, true><<<grid(a.Bt * a.nparts, a.H, share_kv), block, 0, s>>>(w);
        const int blocks = (a.Kd * a.Vd + 255) / 256;
        if (a.nparts > kFold) {
            w.each = a.Bt * a.H * blocks;
            attention_join_kernel<<<dim3(static_cast<unsigned>(w.each * count)), dim3(256), 0, s>>>(w, blocks);
        }
    }
    if constexpr (SUB > 1) {
        if (a.each > 1) {
            const int sums = (a.each + SUB - 1) / SUB;
            attention_kernel<E, OUT, KD, NW, SUB, false><<<grid(a.Bt * a.nseg, a.outs, sums), dim3(64 * NW * SUB), 0, s>>>(w);
            return;
        }
    }
    attention_kernel<E, OUT, KD, NW, 1, false><<<grid(a.Bt * a.nseg, a.outs, share), block, 0, s>>>(w);
}
// Walks of the same sizes and type of outputs, side by side, of some batches; their states in scratch.
template <class E, class OUT>
void walk_batches(Walks w, const Sizes& z, int64_t from, float* scratch, hipStream_t s) {
    const Plan p = plan_walks(z);
    for (int i = 0; i < z.count; ++i) {
        AArgs& a = w.w[i];
        const auto rows = [&](const void* t, int64_t row, size_t size) {
            return static_cast<const char*>(t) + from * z.L * row * static_cast<int64_t>(size);
        };
        constexpr size_t ES = sizeof(typename E::storage);
        const int64_t states = from * z.H * z.Kd * z.Vd;
        a.q.p = rows(a.q.p, a.q.heads * z.Kd, ES);
        a.k.p = rows(a.k.p, a.k.heads * z.Kd, ES);
        a.v.p = rows(a.v.p, a.v.heads * z.Vd, ES);
        a.out = const_cast<char*>(rows(a.out, z.outs * z.Vd, sizeof(typename OUT::storage)));
        if (a.lens) a.lens += from;
        if (a.init) a.init += states;
        if (a.last) a.last += states;
        a.Bt = z.Bt;
        a.nseg = p.nseg; a.nparts = p.nparts; a.cuts = p.cuts; a.part_steps = p.part_steps;
        a.parts = scratch + i * z.Bt * z.H * p.nparts * z.Kd * z.Vd;
    }
    const bool wide = columns(z.Vd) == 128;
    if (z.Kd <= 64) {
        if (wide) walk_waves<E, OUT, 64, 8>(w, z.count, s);
        else walk_waves<E, OUT, 64, 4>(w, z.count, s);
    } else {
        if (wide) walk_waves<E, OUT, 128, 8>(w, z.count, s);
        else walk_waves<E, OUT, 128, 4>(w, z.count, s);
    }
}
template <class E, class OUT>
void walk(const Walks& w, int count, float* scratch, hipStream_t s) {
    const AArgs& a = w.w[0];
    const Sizes z{Form<E>::NP == 1, a.Bt, a.L, a.H, a.outs, a.each, a.Kd, a.Vd, count};
    const int64_t first = first_batches(z);
    walk_batches<E, OUT>(w, z.of(first), 0, scratch, s);
    if (first < a.Bt) walk_batches<E, OUT>(w, z.of(a.Bt - first), first, scratch, s);
}

// The backward's walks: of what sizes, from and to where.  Those of equal sizes whose outputs are alike go in one launch.
struct Role {
    Rows q, k, v;
    void* out;
    int heads, Kd, Vd;  // heads of out
    bool back, turned;
    int each, outs;     // as the kernel takes them
    int sums;           // outputs of a group that are still to be added up (1: none)
};
struct Roles {
    Role r[kMostWalks];
    int first[kMostWalks + 1], count;  // launches
};
Roles roles_of(const AttnLaunch& l) {
    const Rows q{l.q, l.Hq}, k{l.k, l.Hk}, v{l.v, l.Hv}, d{l.dout, l.H};
    Roles o{{{d, v, k, l.dq, l.Hq, l.V, l.K, false, true, 1, l.H, 1},
             {v, d, q, l.dk, l.Hk, l.V, l.K, true, true, 1, l.H, 1},
             {k, q, d, l.dv, l.Hv, l.K, l.V, true, false, 1, l.H, 1}}, {0, 1, 2, 3}, 0};
    for (int i = 0; i < kMostWalks; ++i) {
        Role& a = o.r[i];
        if (a.heads < l.H) {
            const int sub = heads_at_once(l.bf16, a.Kd <= 64 ? 64 : 128, columns(a.Vd) / 16), each = l.H / a.heads;
            a.sums = sub > 1 ? (each + sub - 1) / sub : each;
            a.each = sub > 1 ? each : 1;
            a.outs = a.heads * a.sums;
        }
        const Role& b = o.r[i > 0 ? i - 1 : 0];
        if (i == 0 || a.Kd != b.Kd || a.Vd != b.Vd || a.each != b.each || a.sums != b.sums || a.outs != b.outs)
            o.first[o.count++] = i;
    }
    o.first[o.count] = kMostWalks;
    return o;
}
// Floats of scratch of a launch's states, and of a walk's sums before they are added up.
int64_t states_of(const AttnLaunch& l, const Role& r, int count) {
    return state_floats({l.bf16, l.Bt, l.L, l.H, r.outs, r.each, r.Kd, r.Vd, count});
}
int64_t sums_of(const AttnLaunch& l, const Role& r) { return r.sums > 1 ? l.Bt * l.L * r.outs * r.Vd : 0; }

template <class E>
void backward(const AttnLaunch& l, hipStream_t s) {
    const Roles o = roles_of(l);
    for (int n = 0; n < o.count; ++n) {
        const int from = o.first[n], count = o.first[n + 1] - from;
        Walks w{};
        float* sums = l.scratch + states_of(l, o.r[from], count);
        for (int i = 0; i < count; ++i) {
            const Role& r = o.r[from + i];
            AArgs& a = w.w[i];
            a.q = r.q; a.k = r.k; a.v = r.v; a.rate = l.rate; a.lens = l.lens; a.Bt = l.Bt; a.L = l.L; a.H = l.H;
            a.Kd = r.Kd; a.Vd = r.Vd; a.back = r.back; a.turned = r.turned; a.each = r.each; a.outs = r.outs;
            a.init = r.back ? l.dlast : l.h0;
            a.last = r.back && !r.turned ? l.dh0 : nullptr;
            a.s_add = r.back ? l.scale : 1.0f;
            a.s_out = r.back ? 1.0f : l.scale;
            a.out = r.sums == 1 ? r.out : sums + i * sums_of(l, r);
        }
        if (o.r[from].sums == 1) {
            walk<E, E>(w, count, l.scratch, s);
            continue;
        }
        walk<E, F32>(w, count, l.scratch, s);
        for (int i = 0; i < count; ++i) {
            const Role& r = o.r[from + i];
            const int64_t all = l.Bt * l.L * r.heads * r.Vd / 4;
            if (all)
                attention_groups_kernel<E><<<dim3(blocks_for(all, 256)), dim3(256), 0, s>>>(
                    static_cast<const float*>(w.w[i].out), r.out, all, r.sums, r.Vd);
        }
    }
}

}  // namespace

int64_t attn_fwd_scratch(int64_t Bt, int64_t L, int H, int K, int V, bool bf16) {
    return state_floats({bf16, Bt, L, H, H, 1, K, V, 1});
}

int64_t attn_bwd_scratch(int64_t Bt, int64_t L, int H, int Hq, int Hk, int Hv, int K, int V, bool bf16) {
    AttnLaunch l{};
    l.bf16 = bf16;
    l.Bt = Bt; l.L = L; l.H = H; l.Hq = Hq; l.Hk = Hk; l.Hv = Hv; l.K = K; l.V = V;
    const Roles o = roles_of(l);
    int64_t most = 0;
    for (int n = 0; n < o.count; ++n) {
        const int from = o.first[n], count = o.first[n + 1] - from;
        most = std::max(most, states_of(l, o.r[from], count) + count * sums_of(l, o.r[from]));
    }
    return most;
}

hipError_t launch_attn_fwd(const AttnLaunch& l, hipStream_t s) {
    Walks w{};
    AArgs& a = w.w[0];
    a.q = {l.q, l.Hq}; a.k = {l.k, l.Hk}; a.v = {l.v, l.Hv}; a.rate = l.rate; a.lens = l.lens; a.init = l.h0;
    a.last = l.last_state; a.out = l.out; a.Bt = l.Bt; a.L = l.L; a.H = l.H; a.Kd = l.K; a.Vd = l.V;
    a.s_add = 1.0f; a.s_out = l.scale; a.each = 1; a.outs = l.H;
    if (l.bf16) walk<BF16, BF16>(w, 1, l.scratch, s);
    else walk<F32, F32>(w, 1, l.scratch, s);
    return hipGetLastError();
}

hipError_t launch_attn_bwd(const AttnLaunch& l, hipStream_t s) {
    if (l.bf16) backward<BF16>(l, s);
    else backward<F32>(l, s);
    return hipGetLastError();
}

hipError_t launch_attn_update(const AttnUpdateLaunch& l, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(l.Bt * l.H)), block(256);
    const bool pass = l.Bt * l.H * l.K * l.V * 4 >= kPassBy;
    if (l.bf16) {
        if (pass) attention_update_kernel<BF16, true><<<grid, block, 0, s>>>(l);
        else attention_update_kernel<BF16, false><<<grid, block, 0, s>>>(l);
    } else {
        if (pass) attention_update_kernel<F32, true><<<grid, block, 0, s>>>(l);
        else attention_update_kernel<F32, false><<<grid, block, 0, s>>>(l);
    }
    return hipGetLastError();
}

}  // namespace mss
