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
// A wave walks a row (or a segment of one) from its end, a tile of 512 steps a round, eight to a lane:
// y needs the last K - 1 inputs of the lane before (a whole-wave shift; those before the tile
// are loaded with it), dx the first K - 1 dy of the lane after; the first lane's dy is kept for the tile that
// precedes it in time.  A tile's loads are issued before the one after it in time is computed.  The
// sums over time stay in registers, in fp32 (8 x 1536 x 2047 f32: all gradients together are
// 1.5e-7 off, 0.8e-7 with 64-bit sums).
#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"

namespace mss {
namespace {

struct CArgs {
    const void* x;
    const float* w;
    const float* bias;      // nullable
    const void* st;         // (R, K-1), nullable
    const void* dout;
    const void* dfin;       // (R, K-1), nullable
    void* dx;
    void* dst;              // (R, K-1), nullable
    float* dw;              // (Dn, K)
    float* db;              // (Dn), nullable
    float* part;            // (K + 1, R, S): a segment's dw_0 .. dw_{K-1}, dbias; null: dw and db are written
    int64_t Bt, Dn, L, R, tiles;
    int64_t seg_tiles;      // tiles per segment
    int S;                  // segments per row
};

// dy = dout silu'(y).  1 - s loses digits where s is near 1: up to u y = 6e-8 y, against a silu' of about 1 there.
__device__ __forceinline__ float silu_grad(float y) {
    const float s = fast_rcp(1.0f + fast_exp2(-y * kLog2e));
    return s * fmaf(y, 1.0f - s, 1.0f);
}

// Five waves a SIMD for aligned bf16 rows (2.8B layer with silu: 52.6 us, 54.5 at four); the other rows' kernels would
// spill (8 x 1536 x 2047 f32: 58 us at four, 70 at five).  Of the aligned ones K = 4 without silu does spill at
// five, 13 registers in 36 bytes a lane: 35.8 MB more are written on the 2.8B layer and the call takes 53.5 us where
// silu's takes 48.8.  Rows that are no whole vectors spill 119 (bf16) and 138 (f32) scalar registers to lanes of
// vector ones: the row's walk is inlined twice, for parts and for whole channels.
template <class E, int K, bool SILU, bool VEC>
__global__ __launch_bounds__(256, VEC && E::kPerVec == 8 ? 5 : 4) void conv_bwd_kernel(CArgs a) {
    using S = typename E::storage;
    __shared__ float sums[4][K + 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int64_t items = a.R * a.S;
    // One row's segment; adds the wave's dw_0 .. dw_{K-1}, dbias to s.
    const auto pass = [&](int64_t row, int seg, float* s) MSS_INLINED {
        const int64_t first = seg * a.seg_tiles;
        const int64_t end = first + a.seg_tiles < a.tiles ? first + a.seg_tiles : a.tiles;
        const int64_t ch = row % a.Dn, base = row * a.L;
        const S* xr = static_cast<const S*>(a.x) + base;
        float w[K], dw[K], db = 0.0f, later[K];  // later: the first K - 1 dy of the following tile
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = a.w[ch * K + k], dw[k] = 0.0f, later[k] = 0.0f;
        const float b = a.bias ? a.bias[ch] : 0.0f;
        if (K > 1 && end < a.tiles) {  // the following segment's first dy, a lane each
            const int64_t t = end * kTile + lane;
            float dy = 0.0f;
            if (lane < K - 1 && t < a.L) {
                dy = E::load1(a.dout, base + t);
                if (SILU) {
                    float y = b;
#pragma unroll
                    for (int k = 0; k < K; ++k) y = fmaf(w[k], E::load1(xr, t - (K - 1) + k), y);
                    dy *= silu_grad(y);
                }
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) later[j] = lane_of(dy, j);
        }
        // lane j: entry j of the final window's gradient
        const S fin = K > 1 && a.dfin ? static_cast<const S*>(a.dfin)[row * (K - 1) + (lane < K - 1 ? lane : 0)] : 0;
        Raw<E> nx, nd;
        S nh = 0;  // lane j: input j of the K - 1 before the tile, as it lies in memory (converted here, each load was
                   // waited for: 65 us)
        const auto load = [&](int64_t k, auto whole) MSS_INLINED {
            const int rem = decltype(whole)::value ? kTile : clamp_tile(a.L - k * kTile);
            load8<E, VEC>(xr + k * kTile, a.L, rem, lane, nx);
            load8<E, VEC>(static_cast<const S*>(a.dout) + base + k * kTile, a.L, rem, lane, nd);
            if (K > 1) {
                const S* h = k > 0 ? xr + (k * kTile - (K - 1)) : a.st ? static_cast<const S*>(a.st) + row * (K - 1) : nullptr;
                nh = h ? h[lane < K - 1 ? lane : 0] : 0;
            }
        };
        // Not MSS_INLINED, which would spill (aligned bf16 rows, K = 4: 19 registers); the build checks that no call is
        // left.
        // WHOLE: the tile lies inside the row.  Rows that are no whole vectors have code of their own for such tiles (8 x
        // 1536 x 2047 f32: 60.5 us, 65 without; aligned bf16 rows would spill at five waves: 55 us for 50).
        const auto tile = [&](int64_t k, auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            const int64_t t = k * kTile;
            const int rem = WHOLE ? kTile : clamp_tile(a.L - t);
            float v[K - 1 + kE], d[kE + K - 1], o[kE];
            if (!WHOLE) {
                settle8<E, VEC>(a.L, rem, lane, nx);
                settle8<E, VEC>(a.L, rem, lane, nd);
            }
            nx.unpack(v + K - 1);
            nd.unpack(d);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) v[j] = dpp<0x138>(lane_of(E::value(nh), j), v[kE + j]);  // wave_shr 1
            if (k > first) load(k - 1, True{});
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                if (SILU) {
                    float y = b;
#pragma unroll
                    for (int q = 0; q < K; ++q) y = fmaf(w[q], v[e + q], y);
                    d[e] *= silu_grad(y);  // past the row's end x and dout are zeros
                }
                db += d[e];
#pragma unroll
                for (int q = 0; q < K; ++q) dw[q] = fmaf(d[e], v[e + q], dw[q]);
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
                for (int q = 0; q < K; ++q) o[e] = fmaf(w[q], d[e + K - 1 - q], o[e]);
            }
            if (K > 1 && a.dfin && t + kTile > a.L - (K - 1)) {  // the row's last K - 1 inputs left as its window
                const int64_t j0 = t + lane * kE - (a.L - (K - 1));
#pragma unroll
                for (int j = 0; j < K - 1; ++j) {
                    const float g = lane_of(E::value(fin), j);
#pragma unroll
                    for (int e = 0; e < kE; ++e) o[e] += j0 + e == j ? g : 0.0f;
                }
            }
            store8<E, VEC>(static_cast<S*>(a.dx) + base + t, rem, lane, o);
        };
        int64_t k = end - 1;
        if (k >= first) load(k, False{});
        if (VEC) {
            for (; k >= first; --k) tile(k, False{});
        } else {  // the row's last tile by itself
            if (k >= first && end * kTile > a.L) tile(k--, False{});
            for (; k >= first; --k) tile(k, True{});
        }
        // `later` now holds dy_0 .. dy_{K-2} of the row (zeros past its end)
        if (K > 1 && a.dst && first == 0 && lane == 0) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                float o = 0.0f;
#pragma unroll
                for (int q = 0; q <= j; ++q) o = fmaf(w[q], later[j - q], o);
                if (a.dfin && j >= a.L) o += E::load1(a.dfin, row * (K - 1) + (j - a.L));
                E::store1(a.dst, row * (K - 1) + j, o);
            }
        }
#pragma unroll
        for (int q = 0; q < K; ++q) s[q] += wave_sum(dw[q]);
        s[K] += wave_sum(db);
    };
    if (a.part) {
        for (int64_t it = (int64_t)blockIdx.x * 4 + wave; it < items; it += (int64_t)gridDim.x * 4) {
            float s[K + 1] = {};
            pass(it / a.S, static_cast<int>(it % a.S), s);
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q <= K; ++q) a.part[q * items + it] = s[q];
            }
        }
        return;
    }
    const int ways = channel_ways(a.Bt), channels = 4 / ways, lead = wave % ways;
    for (int64_t c = (int64_t)blockIdx.x * channels; c < a.Dn; c += (int64_t)gridDim.x * channels) {
        const int64_t ch = c + wave / ways;
        float s[K + 1] = {};
        if (ch < a.Dn)
            for (int64_t b = lead; b < a.Bt; b += ways) pass(b * a.Dn + ch, 0, s);
        if (lane == 0) {
#pragma unroll
            for (int q = 0; q <= K; ++q) sums[wave][q] = s[q];
        }
        __syncthreads();
        if (ch < a.Dn && lead == 0 && lane <= K) {
            float t = 0.0f;
            for (int v = 0; v < ways; ++v) t += sums[wave + v][lane];
            if (lane < K) a.dw[ch * K + lane] = t;
            else if (a.db) a.db[ch] = t;
        }
        __syncthreads();
    }
}

// The parts of channel d's rows and their segments summed: a wave per sum, each lane every 64th part in
// order, then the lanes.
template <int K>
__global__ __launch_bounds__(256) void conv_sums_kernel(const float* part, float* dw, float* db, int64_t Dn, int64_t n,
                                                        int S) {
    const int64_t items = Dn * n * S;
    const int lane = threadIdx.x & 63;
    for (int64_t g = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); g < Dn * (K + 1); g += (int64_t)gridDim.x * 4) {
        const int64_t d = g % Dn, k = g / Dn;
        float s = 0.0f;
        for (int64_t j = lane; j < n * S; j += 64) s += part[k * items + (j / S * Dn + d) * S + j % S];
        s = wave_sum(s);
        if (lane != 0) continue;
        if (k < K) dw[d * K + k] = s;
        else if (db) db[d] = s;
    }
}

// Segments per row, by sizes alone: enough waves to fill the chip (8192, eight a SIMD), each with a tile.
struct Plan {
    int S;
    int64_t tiles, seg_tiles;
    bool parts(int64_t Bt, int64_t Dn) const {
        return S > 1 || goes_by_parts(Bt, Dn, channel_ways(Bt), channel_ways(Bt));
    }
};
Plan plan_of(int64_t R, int64_t L) {
    Plan p;
    p.tiles = (L + kTile - 1) / kTile;
    const int64_t want = R > 0 ? (8192 + R - 1) / R : 1;
    p.seg_tiles = (p.tiles + want - 1) / want;
    p.S = p.tiles > 0 ? static_cast<int>((p.tiles + p.seg_tiles - 1) / p.seg_tiles) : 1;
    return p;
}

template <class E, int K, bool SILU>
void launch_v(const CArgs& a, bool vec, hipStream_t s) {
    const dim3 grid(a.part ? blocks_for(a.R * a.S, 4) : blocks_for(a.Dn, 4 / channel_ways(a.Bt))), block(256);
    if (vec) conv_bwd_kernel<E, K, SILU, true><<<grid, block, 0, s>>>(a);
    else conv_bwd_kernel<E, K, SILU, false><<<grid, block, 0, s>>>(a);
}

template <class E, int K>
hipError_t launch_k(const CArgs& a, const ConvBwdLaunch& l, hipStream_t s) {
    if (l.silu) launch_v<E, K, true>(a, l.vec_ok, s);
    else launch_v<E, K, false>(a, l.vec_ok, s);
    if (a.part)
        conv_sums_kernel<K><<<dim3(blocks_for(a.Dn * (K + 1), 4)), dim3(256), 0, s>>>(a.part, l.dw, l.db, a.Dn, a.Bt, a.S);
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

int64_t conv1d_bwd_scratch(int64_t Bt, int64_t Dn, int64_t L, int64_t K) {
    const Plan p = plan_of(Bt * Dn, L);
    return p.parts(Bt, Dn) ? (K + 1) * Bt * Dn * p.S : 0;
}

hipError_t launch_conv1d_bwd(const ConvBwdLaunch& l, hipStream_t s) {
    const Plan p = plan_of(l.R, l.L);
    CArgs a{};
    a.x = l.x; a.w = l.w; a.bias = l.bias; a.st = l.state_in; a.dout = l.dout; a.dfin = l.dfinal; a.dx = l.dx;
    a.dst = l.dstate; a.dw = l.dw; a.db = l.db; a.Dn = l.Dn; a.L = l.L; a.R = l.R;
    a.Bt = l.R / l.Dn;
    a.part = p.parts(a.Bt, l.Dn) ? l.scratch : nullptr;
    a.tiles = p.tiles; a.seg_tiles = p.seg_tiles; a.S = p.S;
    return l.bf16 ? launch_e<BF16>(a, l, s) : launch_e<F32>(a, l, s);
}

}  // namespace mss
