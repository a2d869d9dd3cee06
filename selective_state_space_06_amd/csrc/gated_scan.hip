// gated_scan.hip -- gated linear recurrence (one state per channel): forward over a sequence, its
// gradients, and the one-token step, for gfx950.
//
// Per row (b, d) with the raw gates f, i and the channel's rate > 0:
//     r = sigmoid(f_t), s = rate r, a = e^-s, m = sqrt(1 - a^2), p = sigmoid(i_t)
//     h_t = a h_{t-1} + m p x_t,    out_t = h_t
// and backwards, with w_t = dL/dh_{t-1} through step t (w after the last step: dL/d last_state)
//     G_t = dout_t + w_{t+1},  w_t = a G_t
//     dx = G m p,  di = G m x p (1 - p),  ds = G (a^2 / m p x - a h_{t-1}),
//     df = ds s (1 - r),  drate = sum over batch and time of ds r
// (dm/ds = a^2 / m).  A step is the map h -> a h + v; maps compose as (a, v)(a', v') =
// (a a', a v' + v), so a wave covers 512 consecutive steps of a row: each lane folds its own eight,
// an in-wave scan of the lanes' maps gives every lane the state it starts from, and the lane then
// runs its steps again from there.  The backward scan is the same with time reversed.
#include "device_math.hpp"
#include "mss_internal.hpp"

namespace mss {
namespace {

constexpr int kE = 8;              // steps per lane
constexpr int kTile = 64 * kE;     // steps per wave and round; also the spacing of saved states
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
    float* saved;           // (R, ceil(L / 512)): forward writes (nullable), backward reads
    const void* dout;
    const float* dlast;     // nullable
    void* dx;
    void* df;
    void* di;
    float* drate_part;      // (R)
    float* dh0;             // nullable
    int64_t Dn, L, R;
};

// What one step needs of its gates.  q = 1 - a^2 = 1 - e^-2s directly loses its digits as s -> 0
// (a rate of 0.01 leaves two), so below 2s = 1/4 it is the series of 1 - e^-y up to y^6 (the next
// term is y^6 / 5040 < 5e-8 of it).
struct Gate {
    float r, a, m, p, s;
    float rc, pc;  // 1 - r, 1 - p
};
// sigmoid(v) and, without the cancellation of 1 - sigmoid for v >> 0, its complement e^-v sigmoid(v).
// Where e^-v overflows the product is inf * 0, and the minimum picks its limit, 1.
__device__ __forceinline__ float sigmoid(float v, float& rest) {
    const float e = fast_exp2(-v * kLog2e), r = fast_rcp(1.0f + e);
    rest = fminf(e * r, 1.0f);
    return r;
}
__device__ __forceinline__ Gate gate_of(float f, float i, float rate) {
    Gate g;
    g.r = sigmoid(f, g.rc);
    g.p = sigmoid(i, g.pc);
    g.s = rate * g.r;
    g.a = fast_exp2(-g.s * kLog2e);
    const float y = 2.0f * g.s;
    float q = fmaf(y, -1.0f / 6.0f, 1.0f);
    q = fmaf(y * (-1.0f / 5.0f), q, 1.0f);
    q = fmaf(y * (-1.0f / 4.0f), q, 1.0f);
    q = fmaf(y * (-1.0f / 3.0f), q, 1.0f);
    q = fmaf(y * (-1.0f / 2.0f), q, 1.0f);
    q = y < 0.25f ? y * q : fmaf(-g.a, g.a, 1.0f);
    g.m = __builtin_amdgcn_sqrtf(q);
    return g;
}

// Eight consecutive elements from step t0 of a row of L (zeros past the end).  VEC: rows are whole
// aligned 16-byte vectors; otherwise element-aligned 16-byte accesses and the row's last, partial
// vector element by element.
template <class E, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t row, int64_t t0, int64_t L, float* v) {
    constexpr int V = E::kPerVec;
    const auto* p = static_cast<const typename E::storage*>(base) + row * L;
#pragma unroll
    for (int j = 0; j < kE / V; ++j) {
        const int64_t t = t0 + j * V;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (t + V <= L) {
            if (VEC) w = *reinterpret_cast<const uint4*>(p + t);
            else __builtin_memcpy(&w, p + t, 16);
            E::unpack(w, v + j * V);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[j * V + e] = (!VEC && t + e < L) ? E::load1(p, t + e) : 0.0f;
        }
    }
}
template <class E, bool VEC>
__device__ __forceinline__ void store8(void* base, int64_t row, int64_t t0, int64_t L, const float* v) {
    constexpr int V = E::kPerVec;
    auto* p = static_cast<typename E::storage*>(base) + row * L;
#pragma unroll
    for (int j = 0; j < kE / V; ++j) {
        const int64_t t = t0 + j * V;
        const uint4 w = E::pack(v + j * V);
        if (t + V <= L) {
            if (VEC) *reinterpret_cast<uint4*>(p + t) = w;
            else __builtin_memcpy(p + t, &w, 16);
        } else if (!VEC) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (t + e < L) E::store1(p, t + e, v[j * V + e]);
        }
    }
}

// v of the lane CTRL names (a DPP move), `old` where there is none.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float old, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Inclusive scan of the lanes' maps in lane order: lane l ends with the composition of lanes 0 .. l.
__device__ __forceinline__ void scan_up(float& P, float& H) {
#define MSS_STEP(CTRL, ROWS)                       \
    {                                              \
        const float p = dpp<CTRL, ROWS>(1.0f, P);  \
        const float h = dpp<CTRL, ROWS>(0.0f, H);  \
        H = fmaf(P, h, H);                         \
        P *= p;                                    \
    }
    MSS_STEP(0x111, 0xF)  // row_shr 1, 2, 4, 8: within the 16-lane rows
    MSS_STEP(0x112, 0xF)
    MSS_STEP(0x114, 0xF)
    MSS_STEP(0x118, 0xF)
    MSS_STEP(0x142, 0xA)  // row_bcast 15 into rows 1 and 3, then row_bcast 31 into rows 2 and 3
    MSS_STEP(0x143, 0xC)
}
// The same from the last lane down, applied to the value w that enters after lane 63: returns what
// enters the lane's own map, and leaves in w what leaves lane 0.
__device__ __forceinline__ float scan_down(float P, float W, float& w, int lane) {
#define MSS_STEP_DOWN(CTRL)                 \
    {                                       \
        const float p = dpp<CTRL>(1.0f, P); \
        const float h = dpp<CTRL>(0.0f, W); \
        W = fmaf(P, h, W);                  \
        P *= p;                             \
    }
    MSS_STEP_DOWN(0x101)  // row_shl 1, 2, 4, 8
    MSS_STEP_DOWN(0x102)
    MSS_STEP_DOWN(0x104)
    MSS_STEP_DOWN(0x108)
    // each row's whole map sits in its first lane
    const float w3 = w;
    const float w2 = fmaf(lane_of(P, 48), w3, lane_of(W, 48));
    const float w1 = fmaf(lane_of(P, 32), w2, lane_of(W, 32));
    const float w0 = fmaf(lane_of(P, 16), w1, lane_of(W, 16));
    w = fmaf(lane_of(P, 0), w0, lane_of(W, 0));
    const float in = lane < 16 ? w0 : lane < 32 ? w1 : lane < 48 ? w2 : w3;
    const float p = dpp<0x101>(1.0f, P), h = dpp<0x101>(0.0f, W);
    return fmaf(p, in, h);
#undef MSS_STEP
#undef MSS_STEP_DOWN
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

__device__ __forceinline__ int64_t length_of(const GArgs& a, int64_t row) {
    if (!a.lens) return a.L;
    const int64_t n = a.lens[row / a.Dn];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// One wave per row, tile after tile.
template <class E, bool VEC>
__global__ __launch_bounds__(256) void gated_fwd_kernel(GArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t tiles = (a.L + kTile - 1) / kTile;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.R; row += (int64_t)gridDim.x * 4) {
        const int64_t len = length_of(a, row);
        const float rate = a.rate[row % a.Dn];
        float h = a.h0 ? a.h0[row] : 0.0f;
        for (int64_t k = 0; k < tiles; ++k) {
            if (a.saved && lane == 0) a.saved[row * tiles + k] = h;
            const int64_t t0 = k * kTile + lane * kE;
            float x[kE], f[kE], i[kE], av[kE], vv[kE];
            load8<E, VEC>(a.x, row, t0, a.L, x);
            load8<E, VEC>(a.f, row, t0, a.L, f);
            load8<E, VEC>(a.i, row, t0, a.L, i);
            float P = 1.0f, H = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const Gate g = gate_of(f[e], i[e], rate);
                const bool on = t0 + e < len;
                av[e] = on ? g.a : 1.0f;
                vv[e] = on ? g.m * g.p * x[e] : 0.0f;
                H = fmaf(av[e], H, vv[e]);
                P *= av[e];
            }
            scan_up(P, H);
            const float p = dpp<0x138>(1.0f, P), q = dpp<0x138>(0.0f, H);  // wave_shr 1
            float s = fmaf(p, h, q);
            h = fmaf(lane_of(P, 63), h, lane_of(H, 63));
            if (a.out) {
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    s = fmaf(av[e], s, vv[e]);
                    vv[e] = t0 + e < len ? s : 0.0f;
                }
                store8<E, VEC>(a.out, row, t0, a.L, vv);
            }
        }
        if (a.last && lane == 0) a.last[row] = h;
    }
}

// One wave per row, tiles from the last to the first; each tile's forward states are run again
// from the saved state it starts with.
template <class E, bool VEC>
__global__ __launch_bounds__(256) void gated_bwd_kernel(GArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t tiles = (a.L + kTile - 1) / kTile;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.R; row += (int64_t)gridDim.x * 4) {
        const int64_t len = length_of(a, row);
        const float rate = a.rate[row % a.Dn];
        float w = a.dlast ? a.dlast[row] : 0.0f;
        float drate = 0.0f;
        for (int64_t k = tiles - 1; k >= 0; --k) {
            const int64_t t0 = k * kTile + lane * kE;
            const float h = a.saved[row * tiles + k];
            float x[kE], f[kE], i[kE], d[kE], before[kE];
            Gate g[kE];
            load8<E, VEC>(a.x, row, t0, a.L, x);
            load8<E, VEC>(a.f, row, t0, a.L, f);
            load8<E, VEC>(a.i, row, t0, a.L, i);
            load8<E, VEC>(a.dout, row, t0, a.L, d);
            float P = 1.0f, H = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                g[e] = gate_of(f[e], i[e], rate);
                if (t0 + e >= len) {  // a step past the end: the identity, and no gradient
                    g[e].a = 1.0f;
                    g[e].m = g[e].s = g[e].p = g[e].r = 0.0f;
                    x[e] = d[e] = 0.0f;
                }
                H = fmaf(g[e].a, H, g[e].m * g[e].p * x[e]);
                P *= g[e].a;
            }
            const float Pl = P;
            scan_up(P, H);
            float s = fmaf(dpp<0x138>(1.0f, P), h, dpp<0x138>(0.0f, H));
            float W = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                before[e] = s;
                s = fmaf(g[e].a, s, g[e].m * g[e].p * x[e]);
            }
#pragma unroll
            for (int e = kE - 1; e >= 0; --e) W = g[e].a * (d[e] + W);
            float wt = scan_down(Pl, W, w, lane);
#pragma unroll
            for (int e = kE - 1; e >= 0; --e) {
                const float G = d[e] + wt;
                wt = g[e].a * G;
                const float mp = g[e].m * g[e].p;
                const float im = g[e].m > 0.0f ? g[e].a * g[e].a * fast_rcp(g[e].m) : 0.0f;
                const float ds = G * fmaf(-g[e].a, before[e], im * g[e].p * x[e]);
                d[e] = G * mp;                                   // dx
                i[e] = G * mp * x[e] * g[e].pc;                  // di
                f[e] = ds * g[e].s * g[e].rc;                    // df
                drate = fmaf(ds, g[e].r, drate);
            }
            store8<E, VEC>(a.dx, row, t0, a.L, d);
            store8<E, VEC>(a.di, row, t0, a.L, i);
            store8<E, VEC>(a.df, row, t0, a.L, f);
        }
        drate = wave_sum(drate);
        if (lane == 0) {
            a.drate_part[row] = drate;
            if (a.dh0) a.dh0[row] = w;
        }
    }
}

// drate[d] = sum of the rows of channel d, in row order.
__global__ __launch_bounds__(256) void gated_rate_kernel(const float* part, float* drate, int64_t Dn, int64_t n) {
    for (int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; d < Dn; d += (int64_t)gridDim.x * blockDim.x) {
        float s = 0.0f;
        for (int64_t b = 0; b < n; ++b) s += part[b * Dn + d];
        drate[d] = s;
    }
}

template <class E>
__global__ __launch_bounds__(256) void gated_step_kernel(float* state, const void* x, const void* f, const void* i,
                                                         const float* rate, void* out, int64_t Dn, int64_t R) {
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < R; r += (int64_t)gridDim.x * blockDim.x) {
        const Gate g = gate_of(E::load1(f, r), E::load1(i, r), rate[r % Dn]);
        const float h = fmaf(g.a, state[r], g.m * g.p * E::load1(x, r));
        state[r] = h;
        E::store1(out, r, h);
    }
}

unsigned blocks_for(int64_t n, int64_t per) {
    const int64_t b = (n + per - 1) / per;
    return static_cast<unsigned>(b < 1 ? 1 : b > (1 << 22) ? (1 << 22) : b);
}

GArgs args_of(const GatedLaunch& l) {
    GArgs a{};
    a.x = l.x; a.f = l.f; a.i = l.i; a.rate = l.rate; a.h0 = l.h0; a.lens = l.lens; a.out = l.out;
    a.last = l.last_state; a.saved = l.saved; a.dout = l.dout; a.dlast = l.dlast; a.dx = l.dx; a.df = l.df;
    a.di = l.di; a.drate_part = l.scratch; a.dh0 = l.dh0; a.Dn = l.Dn; a.L = l.L; a.R = l.Bt * l.Dn;
    return a;
}

}  // namespace

int64_t gated_fwd_scratch(int64_t, int64_t, int64_t) { return 0; }
int64_t gated_bwd_scratch(int64_t Bt, int64_t Dn, int64_t) { return Bt * Dn; }

hipError_t launch_gated_fwd(const GatedLaunch& l, hipStream_t s) {
    const GArgs a = args_of(l);
    const dim3 grid(blocks_for(a.R, 4)), block(256);
    if (l.bf16) {
        if (l.vec_ok) gated_fwd_kernel<BF16, true><<<grid, block, 0, s>>>(a);
        else gated_fwd_kernel<BF16, false><<<grid, block, 0, s>>>(a);
    } else {
        if (l.vec_ok) gated_fwd_kernel<F32, true><<<grid, block, 0, s>>>(a);
        else gated_fwd_kernel<F32, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedLaunch& l, hipStream_t s) {
    const GArgs a = args_of(l);
    const dim3 grid(blocks_for(a.R, 4)), block(256);
    if (l.bf16) {
        if (l.vec_ok) gated_bwd_kernel<BF16, true><<<grid, block, 0, s>>>(a);
        else gated_bwd_kernel<BF16, false><<<grid, block, 0, s>>>(a);
    } else {
        if (l.vec_ok) gated_bwd_kernel<F32, true><<<grid, block, 0, s>>>(a);
        else gated_bwd_kernel<F32, false><<<grid, block, 0, s>>>(a);
    }
    gated_rate_kernel<<<dim3(blocks_for(a.Dn, 256)), block, 0, s>>>(a.drate_part, l.drate, a.Dn, l.Bt);
    return hipGetLastError();
}

hipError_t launch_gated_update(const GatedUpdateLaunch& l, hipStream_t s) {
    const dim3 grid(blocks_for(l.R, 256)), block(256);
    if (l.bf16) gated_step_kernel<BF16><<<grid, block, 0, s>>>(l.state, l.x, l.f, l.i, l.rate, l.out, l.Dn, l.R);
    else gated_step_kernel<F32><<<grid, block, 0, s>>>(l.state, l.x, l.f, l.i, l.rate, l.out, l.Dn, l.R);
    return hipGetLastError();
}

}  // namespace mss
