// gated_scan.hip -- gated linear recurrence (one state per channel): forward over a sequence, its
// gradients, and the one-token step, for gfx950.
//
// Per row (b, d) with the raw gates f, i and the channel's rate > 0:
//     r = sigmoid(f_t), s = rate r, a = e^-s, m = sqrt(1 - a^2), p = sigmoid(i_t)
//     h_t = a h_{t-1} + m p x_t,    out_t = h_t
// and backwards, with w_t = dL/dh_{t-1} through step t (w after the last step: dL/d last_state)
//     G_t = dout_t + w_{t+1},  w_t = a G_t
//     dx = G m p,  di = G m p x (1 - p),  ds = G (a^2 / m p x - a h_{t-1}),
//     df = ds s (1 - r),  drate = sum over batch and time of ds r
// (dm/ds = a^2 / m).  A step is the map h -> a h + v; maps compose as (a, v)(a', v') =
// (a a', a v' + v), so a wave covers 512 consecutive steps of a row (a tile): each lane folds its own
// eight, an in-wave scan of the lanes' maps gives every lane the state it starts from, and the lane
// then runs its steps again from there.  The backward scan is the same with time reversed; it starts
// each tile from the state the forward saved for it.
#include <algorithm>

#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"

namespace mss {
namespace {

static_assert(kTile == kGatedTile, "the ABI's saved_states spacing");

struct GArgs {
    const void* x;
    const void* f;
    const void* i;
    const float* rate;
    const float* h0;        // nullable
    const int32_t* lens;    // nullable
    void* out;              // nullable
    float* last;            // nullable
    float* saved;           // (R, tiles): forward writes (nullable), backward reads
    const void* dout;
    const float* dlast;     // nullable
    void* dx;
    void* df;
    void* di;
    float* drate;           // (Dn)
    float* drate_part;      // (R, S), or null: drate is written itself
    float* dh0;             // nullable
    float2* seg;            // (R, S): the segments' maps, when S > 1
    int64_t Bt, Dn, L, R, tiles;
    int64_t seg_tiles;      // tiles per segment
    int S;                  // segments per row
};

// ---- gates
// q = 1 - a^2 = 1 - e^-y, y = 2 s, formed as such loses its digits as y -> 0 (a decay of 0.99 leaves
// five), so up to y = 1/2 it is y (k0 + .. + k4 y^4), a fit of (1 - e^-y) / y there (relative error up to 1.04e-7, at
// y = 1/2; with fp32's rounding 2.0e-7, and 2.3e-7 in the form by r below).
constexpr float kQ[5] = {0.9999999403953552f, -0.4999924898147583f, 0.16654814779758453f, -0.04100127890706062f,
                         0.006771037820726633f};

// The rate's share of every step, the same for a whole row.  Rows whose decay stays within the fit
// (rate < 1/4: every step of them has y < 1/2) take its coefficients in r directly and need neither y
// nor the other branch (2.8B layer bf16: 65 us against 67 forward, 115 against 122 backward).
struct Row {
    float rate, nrl;  // -rate log2 e
    float c[5];       // kQ[k] (2 rate)^(k + 1)
    bool small;
};
// The least q under 1 / m, which it keeps finite where the gate is closed (r = 0, m = 0; 1 / m is then 2^62), and
// a normal number, which a reciprocal root takes.
constexpr float kLeastQ = 0x1p-124f;
__device__ __forceinline__ Row row_of(float rate) {
    Row w;
    w.rate = rate;
    w.nrl = -rate * kLog2e;
    w.small = rate < 0.25f && rate > 0.0f;
    float p = 2.0f * rate;
#pragma unroll
    for (int k = 0; k < 5; ++k) w.c[k] = kQ[k] * p, p *= 2.0f * rate;
    return w;
}
__device__ __forceinline__ float q_of(float y, float a) {
    const float t = y * fmaf(y, fmaf(y, fmaf(y, fmaf(y, kQ[4], kQ[3]), kQ[2]), kQ[1]), kQ[0]);
    return y < 0.5f ? t : fmaf(-a, a, 1.0f);
}
template <bool SMALL>
__device__ __forceinline__ float q_of(const Row& w, float r, float a) {
    if (SMALL) return r * fmaf(r, fmaf(r, fmaf(r, fmaf(r, w.c[4], w.c[3]), w.c[2]), w.c[1]), w.c[0]);
    return q_of(2.0f * w.rate * r, a);
}
__device__ __forceinline__ float exp_neg(float v) { return fast_exp2(v * -kLog2e); }

// ---- scans over the lanes
// One round of a scan: the map of the lane CTRL names applied before this lane's.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ void join(float& P, float& H) {
    const float p = dpp<CTRL, ROWS>(1.0f, P), h = dpp<CTRL, ROWS>(0.0f, H);
    H = fmaf(P, h, H);
    P *= p;
}
// Inclusive scan of the lanes' maps in lane order: lane l ends with the composition of lanes 0 .. l.
__device__ __forceinline__ void scan_up(float& P, float& H) {
    join<0x111>(P, H);  // row_shr 1, 2, 4, 8: within the 16-lane rows
    join<0x112>(P, H);
    join<0x114>(P, H);
    join<0x118>(P, H);
    join<0x142, 0xA>(P, H);  // row_bcast 15 into rows 1 and 3, then row_bcast 31 into rows 2 and 3
    join<0x143, 0xC>(P, H);
}
// What enters lane l's map after an inclusive scan when h enters lane 0's.
__device__ __forceinline__ float enter_up(float P, float H, float h) {
    return fmaf(dpp<0x138>(1.0f, P), h, dpp<0x138>(0.0f, H));  // wave_shr 1
}
// The same from the last lane down.  The wave's whole map ends in (P0, W0), and rp, rw hold the map
// of the 16-lane rows after the lane's.
struct Down {
    float P, W;    // inclusive within the row
    float rp, rw;  // of the rows after this lane's
    float P0, W0;
};
__device__ __forceinline__ Down scan_down(float P, float W, int lane) {
    join<0x101>(P, W);  // row_shl 1, 2, 4, 8
    join<0x102>(P, W);
    join<0x104>(P, W);
    join<0x108>(P, W);
    const float p3 = lane_of(P, 48), w3 = lane_of(W, 48);
    const float p2 = lane_of(P, 32), w2 = lane_of(W, 32);
    const float p1 = lane_of(P, 16), w1 = lane_of(W, 16);
    const float q2 = p2 * p3, v2 = fmaf(p2, w3, w2);
    const float q1 = p1 * q2, v1 = fmaf(p1, v2, w1);
    Down d;
    d.P = P;
    d.W = W;
    d.rp = lane < 16 ? q1 : lane < 32 ? q2 : lane < 48 ? p3 : 1.0f;
    d.rw = lane < 16 ? v1 : lane < 32 ? v2 : lane < 48 ? w3 : 0.0f;
    d.P0 = lane_of(P, 0) * q1;
    d.W0 = fmaf(lane_of(P, 0), v1, lane_of(W, 0));
    return d;
}
// What enters lane l's map when w enters lane 63's.
__device__ __forceinline__ float enter_down(const Down& d, float w) {
    const float row = fmaf(d.rp, w, d.rw);
    return fmaf(dpp<0x101>(1.0f, d.P), row, dpp<0x101>(0.0f, d.W));
}
__device__ __forceinline__ int64_t length_of(const GArgs& a, int64_t row) {
    if (!a.lens) return a.L;
    const int64_t n = a.lens[row / a.Dn];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// Who does what.  W waves share a row, W tiles a round, and hand their maps on through LDS; with W = 1 a
// block of four waves holds four rows.  With S > 1 a row is cut into S segments of whole rounds, and
// a work item is a (row, segment).
template <int W>
struct Place {
    static constexpr int kRows = W == 1 ? 4 : 1;              // work items per block
    static constexpr int kThreads = W == 1 ? 256 : 64 * W;
    int lane, wave, item;
    __device__ __forceinline__ Place() {
        lane = threadIdx.x & 63;
        const int v = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        wave = W == 1 ? 0 : v;
        item = W == 1 ? v : 0;
    }
};

// The maps of a round's W tiles joined through LDS (two buffers in turn: a wave may enter the next round
// while another still reads this one's).  In: this wave's map.  Out: the map of the waves before it in
// order (UP) or after it (!UP), and of all of them.
template <int W, bool UP>
__device__ __forceinline__ void join_waves(float2 (*sh)[W], int64_t round, const Place<W>& at, float P, float H,
                                           float2& mine, float2& all) {
    float2* buf = sh[round & 1];
    if (at.lane == 0) buf[at.wave] = make_float2(P, H);
    __syncthreads();
    mine = all = make_float2(1.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const int v = UP ? k : W - 1 - k;
        if (v == at.wave) mine = all;
        const float2 m = buf[v];
        all = make_float2(all.x * m.x, fmaf(m.x, all.y, m.y));
    }
}

// ---- forward.  FOLD: only the segments' maps are wanted (nothing is written but a.seg).
template <class E, bool VEC, int W, bool FOLD>
__global__ __launch_bounds__(Place<W>::kThreads) void gated_fwd_kernel(GArgs a) {
    using S = typename E::storage;
    __shared__ float2 sh[2][W];
    const Place<W> at;
    const int64_t items = a.R * a.S;
    for (int64_t it = (int64_t)blockIdx.x * Place<W>::kRows + at.item; it < items;
         it += (int64_t)gridDim.x * Place<W>::kRows) {
        const int64_t row = a.S == 1 ? it : it / a.S;
        const int seg = a.S == 1 ? 0 : static_cast<int>(it % a.S);
        const int64_t first = seg * a.seg_tiles;
        const int64_t end = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
        const int64_t len = length_of(a, row);
        const Row w = row_of(a.rate[row % a.Dn]);
        float h = !FOLD && a.h0 ? a.h0[row] : 0.0f, all_p = 1.0f;
        if (!FOLD && seg > 0) {  // the segments before this one, a lane each
            const float2 m = at.lane < seg ? a.seg[row * a.S + at.lane] : make_float2(1.0f, 0.0f);
            float P = m.x, H = m.y;
            scan_up(P, H);
            h = fmaf(lane_of(P, 63), h, lane_of(H, 63));
        }
        const auto x_ = static_cast<const S*>(a.x) + row * a.L, f_ = static_cast<const S*>(a.f) + row * a.L;
        const auto i_ = static_cast<const S*>(a.i) + row * a.L;
        Raw<E> nx{}, nf{}, ni{};  // the next tile's inputs, on their way while this one is computed
        const auto load = [&](int64_t k) MSS_INLINED {
            const int64_t t = k * kTile;
            const int rem = clamp_tile(len - t);  // nothing past the sequence's end is read...
            if (rem > 0) {
                const int in = rem == kTile ? kTile : clamp_tile(a.L - t);  // ...but whole vectors of the row
                load8<E, VEC>(f_ + t, a.L, in, at.lane, nf);
                load8<E, VEC>(i_ + t, a.L, in, at.lane, ni);
                load8<E, VEC>(x_ + t, a.L, in, at.lane, nx);
            }
        };
        load(first + at.wave);
        // A round of W tiles from tile k0.  FAST: every step of it lies inside the sequence, and w.small.
        const auto round = [&](int64_t k0, auto fast) MSS_INLINED {
            constexpr bool FAST = decltype(fast)::value;
            const int64_t k = k0 + at.wave, t = k * kTile;
            const int on = FAST ? kTile : k < end ? clamp_tile(len - t) : 0;  // this tile's steps in the sequence
            const int rem = FAST ? kTile : k < end ? clamp_tile(a.L - t) : 0;
            float v[kE], f[kE], i[kE], P = 1.0f, H = 0.0f;
            if (!FAST) {
                settle8<E, VEC>(a.L, rem, at.lane, nf);
                settle8<E, VEC>(a.L, rem, at.lane, ni);
                settle8<E, VEC>(a.L, rem, at.lane, nx);
            }
            nf.unpack(f);
            ni.unpack(i);
            nx.unpack(v);
            if (k0 + W < end) load(k + W);
#pragma unroll
            for (int e = 0; e < kE; ++e) {  // f becomes a, v the input term
                const float r = fast_rcp(1.0f + exp_neg(f[e])), p = fast_rcp(1.0f + exp_neg(i[e]));
                f[e] = fast_exp2(r * w.nrl);
                v[e] *= __builtin_amdgcn_sqrtf(q_of<FAST>(w, r, f[e])) * p;
                if (!FAST && at.lane * kE + e >= on) f[e] = 1.0f, v[e] = 0.0f;
                H = fmaf(f[e], H, v[e]);
                P *= f[e];
            }
            scan_up(P, H);
            float start = h;
            if (W == 1) {
                if (FOLD) all_p *= lane_of(P, 63);
                h = fmaf(lane_of(P, 63), h, lane_of(H, 63));
            } else {
                float2 mine, all;
                join_waves<W, true>(sh, k0 / W, at, lane_of(P, 63), lane_of(H, 63), mine, all);
                start = fmaf(mine.x, h, mine.y);
                if (FOLD) all_p *= all.x;
                h = fmaf(all.x, h, all.y);
            }
            if (FOLD || rem == 0) return;
            if (a.saved && at.lane == 0) a.saved[row * a.tiles + k] = start;
            if (!a.out) return;
            float s = enter_up(P, H, start);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                s = fmaf(f[e], s, v[e]);
                v[e] = FAST || at.lane * kE + e < on ? s : 0.0f;
            }
            store8<E, VEC>(static_cast<S*>(a.out) + row * a.L + t, rem, at.lane, v);
        };
        const int64_t inside = w.small ? len / kTile : 0;  // tiles a fast round may end at
        const int64_t fast = inside < end ? inside : end;
        int64_t k0 = first;
        for (; k0 + W <= fast; k0 += W) round(k0, True{});
        for (; k0 < end; k0 += W) round(k0, False{});
        if (at.lane == 0 && at.wave == 0) {
            if (FOLD) a.seg[it] = make_float2(all_p, h);
            else if (a.last && end == a.tiles) a.last[row] = h;
        }
        if (W > 1) __syncthreads();  // the next item's first round writes the buffer this one's last may read
    }
}

// ---- backward.  FOLD: only the segments' maps are wanted; they need the decays and dout alone.
template <class E, bool VEC, int W, bool FOLD>
__global__ __launch_bounds__(Place<W>::kThreads, W == 1 || VEC ? 4 : 3) void gated_bwd_kernel(GArgs a) {
    using S = typename E::storage;
    __shared__ float2 sh[2][W];
    __shared__ float sums[W == 1 ? 4 : W];
    const Place<W> at;
    // One row's segment; returns this wave's share of its part of drate.
    const auto pass = [&](int64_t row, int seg) MSS_INLINED {
        const int64_t first = seg * a.seg_tiles;
        const int64_t end = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
        const int64_t len = length_of(a, row);
        const Row w = row_of(a.rate[row % a.Dn]);
        float g = !FOLD && a.dlast ? a.dlast[row] : 0.0f, all_p = 1.0f, drate = 0.0f;
        if (!FOLD && seg < a.S - 1) {  // the segments after this one, a lane each, the last one first
            const float2 m = at.lane < a.S - 1 - seg ? a.seg[row * a.S + a.S - 1 - at.lane] : make_float2(1.0f, 0.0f);
            float P = m.x, H = m.y;
            scan_up(P, H);
            g = fmaf(lane_of(P, 63), g, lane_of(H, 63));
        }
        // Not MSS_INLINED, which is inlined before it is simplified and then spills (rows that are no whole vectors, one
        // wave: 20 registers in f32); each form has one call site, and the build checks that no call is left.
        const auto round = [&](int64_t k0, auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            const int64_t k = k0 + at.wave, t = k * kTile, p0 = row * a.L + t;
            const int on = FAST ? kTile : k < end ? clamp_tile(len - t) : 0;  // this tile's steps in the sequence
            const int rem = FAST ? kTile : k < end ? clamp_tile(a.L - t) : 0;
            Raw<E> rf{}, rd{}, rx{}, ri{};
            float start = 0.0f;
            if (on > 0) {
                load8<E, VEC>(static_cast<const S*>(a.f) + p0, a.L, rem, at.lane, rf);
                load8<E, VEC>(static_cast<const S*>(a.dout) + p0, a.L, rem, at.lane, rd);
                if (!FOLD) {
                    load8<E, VEC>(static_cast<const S*>(a.i) + p0, a.L, rem, at.lane, ri);
                    load8<E, VEC>(static_cast<const S*>(a.x) + p0, a.L, rem, at.lane, rx);
                    start = a.saved[row * a.tiles + k];
                }
            }
            if (!FAST) {
                settle8<E, VEC>(a.L, rem, at.lane, rf);
                settle8<E, VEC>(a.L, rem, at.lane, rd);
                if (!FOLD) {
                    settle8<E, VEC>(a.L, rem, at.lane, ri);
                    settle8<E, VEC>(a.L, rem, at.lane, rx);
                }
            }
            // of every step: a, r, s (1 - r), a^2 p x / m, p m, x (1 - p), p m x, dout: no more of them than the
            // second pass needs, so that four waves share a SIMD (2.8B layer bf16: 115 us, 120 at three).  bf16 rows
            // with one wave spill two registers all the same (12 bytes a lane; 4% more is written on that layer;
            // aligned rows compiled without the loop over the batch around the walk spill none).
            float av[kE], rv[kE], sc[kE], into[kE], pm[kE], xc[kE], v[kE], d[kE];
            float P = 1.0f, H = 0.0f, V = 0.0f;
            rf.unpack(rv);
            rd.unpack(d);
            if (!FOLD) {
                ri.unpack(pm);
                rx.unpack(xc);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const bool off = !FAST && at.lane * kE + e >= on;
                const float ef = exp_neg(rv[e]);
                rv[e] = fast_rcp(1.0f + ef);
                av[e] = fast_exp2(rv[e] * w.nrl);
                if (!FOLD) {
                    // 1 - sigmoid without its cancellation; where e^-f overflows the product is inf * 0 and the
                    // minimum picks its limit, 1
                    const float x = xc[e], ei = exp_neg(pm[e]), p = fast_rcp(1.0f + ei);
                    const float q = q_of<FAST>(w, rv[e], av[e]);
                    float im = __builtin_amdgcn_rsqf(fmaxf(q, kLeastQ));  // 1 / m
                    if (!FAST) im = w.rate == 0.0f ? 0.0f : im;
                    sc[e] = w.rate * rv[e] * fminf(ef * rv[e], 1.0f);
                    xc[e] = x * fminf(ei * p, 1.0f);
                    into[e] = av[e] * av[e] * im * (p * x);
                    pm[e] = p * (q * im);  // q as it is: 0 of a closed gate stays 0, and a NaN, which fmaxf drops, a NaN
                    v[e] = pm[e] * x;
                    if (off) rv[e] = sc[e] = xc[e] = into[e] = pm[e] = v[e] = 0.0f;
                }
                if (off) av[e] = 1.0f, d[e] = 0.0f;
                P *= av[e];
                if (!FOLD) H = fmaf(av[e], H, v[e]);
            }
#pragma unroll
            for (int e = kE - 1; e >= 0; --e) V = av[e] * (d[e] + V);
            const Down down = scan_down(P, V, at.lane);
            float in = g;  // what enters this tile from the later ones
            if (W == 1) {
                if (FOLD) all_p *= down.P0;
                g = fmaf(down.P0, g, down.W0);
            } else {
                float2 mine, all;
                join_waves<W, false>(sh, k0 / W, at, down.P0, down.W0, mine, all);
                in = fmaf(mine.x, g, mine.y);
                if (FOLD) all_p *= all.x;
                g = fmaf(all.x, g, all.y);
            }
            if (FOLD || rem == 0) return;
            scan_up(P, H);
            float s = enter_up(P, H, start), wt = enter_down(down, in);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                into[e] = fmaf(-av[e], s, into[e]);  // ds / G
                s = fmaf(av[e], s, v[e]);
            }
#pragma unroll
            for (int e = kE - 1; e >= 0; --e) {
                const bool off = !FAST && at.lane * kE + e >= on;
                const float G = d[e] + wt, ds = G * into[e];
                wt = av[e] * G;
                pm[e] = off ? 0.0f : pm[e] * G;     // dx
                xc[e] = off ? 0.0f : xc[e] * pm[e]; // di
                sc[e] = off ? 0.0f : sc[e] * ds;    // df
                drate += off ? 0.0f : ds * rv[e];
            }
            store8<E, VEC>(static_cast<S*>(a.dx) + p0, rem, at.lane, pm);
            store8<E, VEC>(static_cast<S*>(a.di) + p0, rem, at.lane, xc);
            store8<E, VEC>(static_cast<S*>(a.df) + p0, rem, at.lane, sc);
        };
        const int64_t inside = w.small ? len / kTile : 0;  // tiles a fast round may end at
        for (int64_t k0 = first + (end - first - 1) / W * W; k0 >= first; k0 -= W) {
            if (k0 + W <= inside && k0 + W <= end) round(k0, True{});
            else round(k0, False{});
        }
        if (at.lane == 0 && at.wave == 0) {
            if (FOLD) a.seg[row * a.S + seg] = make_float2(all_p, g);
            else if (a.dh0 && first == 0) a.dh0[row] = g;
        }
        if (W > 1) __syncthreads();  // the next pass writes sh
        return FOLD ? 0.0f : wave_sum(drate);
    };
    // the waves' parts added in order, for the wave that leads `ways` of them
    const auto total = [&](int wave, int ways, float part) MSS_INLINED {
        if (ways == 1) return part;
        if (at.lane == 0) sums[wave] = part;
        __syncthreads();
        float s = 0.0f;
        for (int v = 0; v < ways; ++v) s += sums[wave / ways * ways + v];
        __syncthreads();
        return s;
    };
    const bool parts = FOLD || a.drate_part;  // an item is a row's segment, else a channel
    if (W == 1) {
        const int ways = parts ? 1 : channel_ways(a.Bt), channels = 4 / ways, lead = at.item % ways;
        const int64_t items = parts ? a.R : a.Dn, rows = parts ? 1 : a.Bt;
        for (int64_t c = (int64_t)blockIdx.x * channels; c < items; c += (int64_t)gridDim.x * channels) {
            const int64_t it = c + at.item / ways;
            float part = 0.0f;
            if (it < items)
                for (int64_t b = lead; b < rows; b += ways) part += pass(b * a.Dn + it, 0);
            part = total(at.item, ways, part);
            if (it < items && lead == 0 && at.lane == 0) (parts ? a.drate_part : a.drate)[it] = part;
        }
    } else {
        const int64_t items = parts ? a.R * a.S : a.Dn, rows = parts ? 1 : a.Bt;
        for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
            float part = 0.0f;
            for (int64_t b = 0; b < rows; ++b)
                part += pass(parts ? it / a.S : b * a.Dn + it, parts ? static_cast<int>(it % a.S) : 0);
            part = total(at.wave, W, part);
            if (!FOLD && at.lane == 0 && at.wave == 0) (parts ? a.drate_part : a.drate)[it] = part;
        }
    }
}

// drate[d] = sum over the rows of channel d and their segments: a wave per channel, each lane every 64th
// part in order, then the lanes.  All of drate's sums are fp32: over time a lane's at most L / 64 terms in a row.
__global__ __launch_bounds__(256) void gated_rate_kernel(const float* part, float* drate, int64_t Dn, int64_t Bt, int S) {
    const int lane = threadIdx.x & 63;
    for (int64_t d = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); d < Dn; d += (int64_t)gridDim.x * 4) {
        float s = 0.0f;
        for (int64_t n = lane; n < Bt * S; n += 64) s += part[(n / S * Dn + d) * S + n % S];
        s = wave_sum(s);
        if (lane == 0) drate[d] = s;
    }
}

// One token, a thread per channel of a row (four to a thread with wide loads took the same 3.1 us for 64 x
// 5120 bf16: the step is a launch and a round trip to memory).  I: a 32-bit index where it will do, whose
// division is far shorter.
template <class E, class I>
__global__ __launch_bounds__(256) void gated_step_kernel(float* state, const void* x, const void* f, const void* i,
                                                         const float* rate, void* out, int64_t Dn, int64_t R) {
    for (I k = static_cast<I>(blockIdx.x) * 256 + static_cast<I>(threadIdx.x); k < static_cast<I>(R);
         k += static_cast<I>(gridDim.x) * 256) {
        const int64_t n = static_cast<int64_t>(k);
        const float rt = rate[k % static_cast<I>(Dn)];
        const float r = fast_rcp(1.0f + exp_neg(E::load1(f, n))), p = fast_rcp(1.0f + exp_neg(E::load1(i, n)));
        const float av = fast_exp2(-rt * r * kLog2e);
        const float h = fmaf(av, state[n], __builtin_amdgcn_sqrtf(q_of(2.0f * rt * r, av)) * p * E::load1(x, n));
        state[n] = h;
        E::store1(out, n, h);
    }
}

// Waves and segments per row, by sizes alone (so scratch can be named without a device).
struct Plan {
    int W, S;
    int64_t tiles, seg_tiles;
    // Whether the backward leaves parts of drate for a second kernel to add up (4.7 us); otherwise a block takes
    // a channel's rows in turn (3 x 1531 x 2041 f32: 57 us, 61 in parts).
    bool parts(int64_t Bt, int64_t Dn) const {
        return S > 1 || (W == 1 ? goes_by_parts(Bt, Dn, channel_ways(Bt), channel_ways(Bt)) : goes_by_parts(Bt, Dn, W, 1));
    }
};
// Four waves to a row read it in longer runs and hand the map on; they pay where a row has at least two
// rounds for them (bf16) or one (f32, whose rounds move twice the bytes).  Rows of 16-bit elements that
// are no whole vectors hold more registers and stay with one wave while there are waves enough.  With
// few rows a row's waves are all the waves there are: eight, and below 128 rows segments too, whose maps
// cost a launch and a second reading.  Microseconds, forward / backward (rows x steps):
//                          one wave      four          eight
//   20480 x  2048 bf16    66.5 / 111    69.0 / 125
//   20480 x  4096 bf16     127 / 224     125 / 216     174 / 274
//   20480 x  4095 bf16     150 / 248     155 / 302     219 / 509
//   20480 x  2048 f32      126 / 233     114 / 205
//    4608 x  8192 bf16    64.4 / 121    57.1 / 103    66.0 / 113
//    1536 x 131072 bf16    370 / 632     368 / 588     315 / 563
//     512 x 32768 f32     82.3 / 201    52.1 / 98.9   49.9 / 96.5
//      64 x 131072 f32     296 / 488    93.2 / 169    95.1 / 137    four, eight segments: 42.7 / 58.4
// Up to 1024 rows any second tile brings four waves, for the few rows' sake; near 1024 rows, and where the rows of a
// channel then go by parts, one wave is as fast or faster in the backward (kernels alone):
//      64 x   3584 bf16    8.6 / 10.7    4.6 / 6.3
//     512 x   1024 f32     4.5 / 7.4     4.5 / 6.8
//    1024 x   1536 f32     7.3 / 11.8    7.7 / 12.2
//    1024 x   3584 bf16   10.0 / 14.8   10.0 / 18.2
//    1024 x   1024 bf16    4.4 / 6.7     6.0 / 11.7
Plan plan_of(int64_t R, int64_t L, bool bf16, bool vec) {
    Plan p;
    p.tiles = (L + kTile - 1) / kTile;
    p.W = p.tiles >= (bf16 ? 8 : 4) && (R <= 4096 || vec || !bf16) ? 4 : 1;
    p.S = 1;
    if (R <= 1024 && p.tiles > 1) p.W = 4;
    if (R <= 2048 && p.tiles >= 64) p.W = 8;
    if (R <= 128 && p.tiles >= 128) {
        p.W = 4;
        p.S = static_cast<int>(512 / R < 64 ? 512 / R : 64);
    }
    // whole rounds per segment, and as many segments as that leaves
    const int64_t rounds = (p.tiles + p.W - 1) / p.W;
    p.seg_tiles = (rounds + p.S - 1) / p.S * p.W;
    p.S = p.tiles > 0 ? static_cast<int>((p.tiles + p.seg_tiles - 1) / p.seg_tiles) : 1;
    return p;
}

GArgs args_of(const GatedLaunch& l, const Plan& p) {
    GArgs a{};
    a.x = l.x; a.f = l.f; a.i = l.i; a.rate = l.rate; a.h0 = l.h0; a.lens = l.lens; a.out = l.out;
    a.last = l.last_state; a.saved = l.saved; a.dout = l.dout; a.dlast = l.dlast; a.dx = l.dx; a.df = l.df;
    a.di = l.di; a.dh0 = l.dh0; a.Dn = l.Dn; a.L = l.L; a.R = l.Bt * l.Dn;
    a.Bt = l.Bt; a.drate = l.drate;
    a.tiles = p.tiles; a.seg_tiles = p.seg_tiles; a.S = p.S;
    a.seg = reinterpret_cast<float2*>(l.scratch);  // R S maps when S > 1, then R S parts of drate
    a.drate_part = p.parts(l.Bt, l.Dn) ? l.scratch + (p.S > 1 ? 2 * a.R * p.S : 0) : nullptr;
    return a;
}

template <class E, bool VEC, int W>
void run_w(const GArgs& a, bool bwd, hipStream_t s) {
    const dim3 grid(blocks_for(a.R * a.S, Place<W>::kRows)), block(Place<W>::kThreads);
    if (bwd) {
        if constexpr (W == 1) {
            const dim3 channels = a.drate_part ? grid : dim3(blocks_for(a.Dn, 4 / channel_ways(a.Bt)));
            gated_bwd_kernel<E, VEC, 1, false><<<channels, block, 0, s>>>(a);
        } else {
            if (a.S > 1) gated_bwd_kernel<E, VEC, W, true><<<grid, block, 0, s>>>(a);
            const dim3 rows = a.drate_part ? grid : dim3(blocks_for(a.Dn, 1));
            gated_bwd_kernel<E, VEC, W, false><<<rows, block, 0, s>>>(a);
        }
    } else {
        if constexpr (W > 1)
            if (a.S > 1) gated_fwd_kernel<E, VEC, W, true><<<grid, block, 0, s>>>(a);
        gated_fwd_kernel<E, VEC, W, false><<<grid, block, 0, s>>>(a);
    }
}
template <class E, bool VEC>
void run_v(const GArgs& a, int W, bool bwd, hipStream_t s) {
    if (W == 1) run_w<E, VEC, 1>(a, bwd, s);
    else if (W == 4) run_w<E, VEC, 4>(a, bwd, s);
    else run_w<E, VEC, 8>(a, bwd, s);
}
hipError_t run(const GatedLaunch& l, bool bwd, hipStream_t s) {
    if (l.Bt * l.Dn == 0) {  // no rows: drate alone is written, with zeros
        if (bwd) gated_rate_kernel<<<dim3(blocks_for(l.Dn, 4)), dim3(256), 0, s>>>(nullptr, l.drate, l.Dn, 0, 1);
        return hipGetLastError();
    }
    const Plan p = plan_of(l.Bt * l.Dn, l.L, l.bf16, l.vec_ok);
    const GArgs a = args_of(l, p);
    if (l.bf16) l.vec_ok ? run_v<BF16, true>(a, p.W, bwd, s) : run_v<BF16, false>(a, p.W, bwd, s);
    else l.vec_ok ? run_v<F32, true>(a, p.W, bwd, s) : run_v<F32, false>(a, p.W, bwd, s);
    if (bwd && a.drate_part)
        gated_rate_kernel<<<dim3(blocks_for(a.Dn, 4)), dim3(256), 0, s>>>(a.drate_part, l.drate, a.Dn, l.Bt, p.S);
    return hipGetLastError();
}

}  // namespace

// Of any type and alignment these sizes may come in.
int64_t gated_fwd_scratch(int64_t Bt, int64_t Dn, int64_t L) {
    int64_t n = 0;
    for (int k = 0; k < 4 && Bt * Dn > 0; ++k) {
        const Plan p = plan_of(Bt * Dn, L, k & 1, k & 2);
        n = std::max(n, p.S > 1 ? 2 * Bt * Dn * p.S : 0);
    }
    return n;
}
int64_t gated_bwd_scratch(int64_t Bt, int64_t Dn, int64_t L) {
    int64_t n = 0;
    for (int k = 0; k < 4 && Bt * Dn > 0; ++k) {
        const Plan p = plan_of(Bt * Dn, L, k & 1, k & 2);
        n = std::max(n, Bt * Dn * ((p.S > 1 ? 2 * p.S : 0) + (p.parts(Bt, Dn) ? p.S : 0)));
    }
    return n;
}

hipError_t launch_gated_fwd(const GatedLaunch& l, hipStream_t s) { return run(l, false, s); }
hipError_t launch_gated_bwd(const GatedLaunch& l, hipStream_t s) { return run(l, true, s); }

hipError_t launch_gated_update(const GatedUpdateLaunch& l, hipStream_t s) {
    const dim3 grid(blocks_for(l.R, 256)), block(256);
    const auto go = [&](auto kernel) { kernel<<<grid, block, 0, s>>>(l.state, l.x, l.f, l.i, l.rate, l.out, l.Dn, l.R); };
    const bool small = l.R < int64_t{1} << 31;
    if (l.bf16) small ? go(gated_step_kernel<BF16, uint32_t>) : go(gated_step_kernel<BF16, int64_t>);
    else small ? go(gated_step_kernel<F32, uint32_t>) : go(gated_step_kernel<F32, int64_t>);
    return hipGetLastError();
}

}  // namespace mss
