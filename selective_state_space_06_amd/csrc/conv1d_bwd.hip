// conv1d_bwd.hip -- gradients of the causal depthwise conv1d (+ silu) of conv1d.hip.
//
// Per channel d, with window[j] the K - 1 carried inputs followed by the row's own (window[t + k]
// meets weight k at step t):
//     y_t = bias + sum_k w_k window[t + k],   dy_t = dout_t silu'(y_t)   (dout_t without silu)
//     silu'(y) = sigma (1 + y (1 - sigma)),   sigma = sigmoid(y)
//     dwindow[j] = sum_k w_k dy_{j - k}  (+ dfinal_state, which are the last K - 1 window entries)
//     dw_k = sum over batch and time of dy_t window[t + k],   dbias = sum of dy_t
// dx is dwindow past its first K - 1 entries, dinitial_state those.
//
// A wave walks a row from its end, 512 steps a round, eight to a lane: y needs the last K - 1 inputs
// of the lane before (a whole-wave shift), dx the first K - 1 dy of the lane after; the first lane's
// dy is kept for the round that precedes it in time.  The sums over time stay in registers.
#include "device_math.hpp"
#include "mss_internal.hpp"

namespace mss {
namespace {

constexpr int kE = 8;
constexpr int kTile = 64 * kE;

struct CArgs {
    const void* x;
    const float* w;
    const float* bias;      // nullable
    const void* st;         // (R, K-1), nullable
    const void* dout;
    const void* dfin;       // (R, K-1), nullable
    void* dx;
    void* dst;              // (R, K-1), nullable
    float* part;            // (K + 1, R): the row's dw_0 .. dw_{K-1}, dbias
    int64_t Dn, L, R;
};

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
template <int CTRL>
__device__ __forceinline__ float dpp(float old, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

template <class E, int K, bool SILU, bool VEC>
__global__ __launch_bounds__(256) void conv_bwd_kernel(CArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t tiles = (a.L + kTile - 1) / kTile;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.R; row += (int64_t)gridDim.x * 4) {
        const int64_t ch = row % a.Dn;
        float w[K], dw[K], db = 0.0f, later[K];  // later: the first K - 1 dy of the following round
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = a.w[ch * K + k], dw[k] = 0.0f, later[k] = 0.0f;
        const float b = a.bias ? a.bias[ch] : 0.0f;
        const auto* xr = static_cast<const typename E::storage*>(a.x) + row * a.L;
        for (int64_t t = tiles - 1; t >= 0; --t) {
            const int64_t t0 = t * kTile + lane * kE;
            float v[K - 1 + kE], d[kE + K - 1], o[kE];
            load8<E, VEC>(a.x, row, t0, a.L, v + K - 1);
            load8<E, VEC>(a.dout, row, t0, a.L, d);
            // the K - 1 inputs before this lane's: from the lane below, for the first lane from the
            // row (always inside it: t0 is at least 512 then) or the carried state
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                float first = 0.0f;
                if (lane == 0) {
                    if (t > 0) first = E::load1(xr, t0 - (K - 1) + j);
                    else if (a.st) first = E::load1(a.st, row * (K - 1) + j);
                }
                v[j] = dpp<0x138>(first, v[kE + j]);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                if (SILU) {
                    float y = b;
#pragma unroll
                    for (int k = 0; k < K; ++k) y = fmaf(w[k], v[e + k], y);
                    const float s = fast_rcp(1.0f + fast_exp2(-y * kLog2e));
                    d[e] *= s * fmaf(y, 1.0f - s, 1.0f);
                }
                if (t0 + e >= a.L) d[e] = 0.0f;
                db += d[e];
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k] = fmaf(d[e], v[e + k], dw[k]);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                d[kE + j] = dpp<0x130>(later[j], d[j]);  // wave_shl 1
                later[j] = lane_of(d[j], 0);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                o[e] = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) o[e] = fmaf(w[k], d[e + K - 1 - k], o[e]);
                const int64_t j = t0 + e - (a.L - (K - 1));
                if (K > 1 && a.dfin && j >= 0 && j < K - 1) o[e] += E::load1(a.dfin, row * (K - 1) + j);
            }
            store8<E, VEC>(a.dx, row, t0, a.L, o);
        }
        // `later` now holds dy_0 .. dy_{K-2} (zeros past the row's end)
        if (K > 1 && a.dst && lane == 0) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k <= j; ++k) s = fmaf(w[k], later[j - k], s);
                if (a.dfin && j >= a.L) s += E::load1(a.dfin, row * (K - 1) + (j - a.L));
                E::store1(a.dst, row * (K - 1) + j, s);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float s = wave_sum(dw[k]);
            if (lane == 0) a.part[k * a.R + row] = s;
        }
        db = wave_sum(db);
        if (lane == 0) a.part[K * a.R + row] = db;
    }
}

// The rows of channel d summed in row order.
template <int K>
__global__ __launch_bounds__(256) void conv_sums_kernel(const float* part, float* dw, float* db, int64_t Dn, int64_t n) {
    const int64_t R = Dn * n;
    for (int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g < Dn * (K + 1);
         g += (int64_t)gridDim.x * blockDim.x) {
        const int64_t d = g % Dn, k = g / Dn;
        float s = 0.0f;
        for (int64_t b = 0; b < n; ++b) s += part[k * R + b * Dn + d];
        if (k < K) dw[d * K + k] = s;
        else if (db) db[d] = s;
    }
}

unsigned blocks_for(int64_t n, int64_t per) {
    const int64_t b = (n + per - 1) / per;
    return static_cast<unsigned>(b < 1 ? 1 : b > (1 << 22) ? (1 << 22) : b);
}

template <class E, int K, bool SILU>
void launch_v(const CArgs& a, bool vec, hipStream_t s) {
    const dim3 grid(blocks_for(a.R, 4)), block(256);
    if (vec) conv_bwd_kernel<E, K, SILU, true><<<grid, block, 0, s>>>(a);
    else conv_bwd_kernel<E, K, SILU, false><<<grid, block, 0, s>>>(a);
}

template <class E, int K>
hipError_t launch_k(const CArgs& a, const ConvBwdLaunch& l, hipStream_t s) {
    if (l.silu) launch_v<E, K, true>(a, l.vec_ok, s);
    else launch_v<E, K, false>(a, l.vec_ok, s);
    conv_sums_kernel<K><<<dim3(blocks_for(a.Dn * (K + 1), 256)), dim3(256), 0, s>>>(a.part, l.dw, l.db, a.Dn, a.R / a.Dn);
    return hipGetLastError();
}

template <class E>
hipError_t launch_e(const CArgs& a, const ConvBwdLaunch& l, hipStream_t s) {
    switch (l.K) {
        case 1: return launch_k<E, 1>(a, l, s);
        case 2: return launch_k<E, 2>(a, l, s);
        case 3: return launch_k<E, 3>(a, l, s);
        default: return launch_k<E, 4>(a, l, s);
    }
}

}  // namespace

int64_t conv1d_bwd_scratch(int64_t Bt, int64_t Dn, int64_t, int64_t K) { return (K + 1) * Bt * Dn; }

hipError_t launch_conv1d_bwd(const ConvBwdLaunch& l, hipStream_t s) {
    CArgs a{};
    a.x = l.x; a.w = l.w; a.bias = l.bias; a.st = l.state_in; a.dout = l.dout; a.dfin = l.dfinal; a.dx = l.dx;
    a.dst = l.dstate; a.part = l.scratch; a.Dn = l.Dn; a.L = l.L; a.R = l.R;
    return l.bf16 ? launch_e<BF16>(a, l, s) : launch_e<F32>(a, l, s);
}

}  // namespace mss
