// rms_norm.hip -- the RMS norm in front of a layer, with the residual stream's addition in it: forward (output in
// the activations' type, or in e4m3 with scales) and gradients, for gfx950.
//
// Forward, per row: z = x + residual (in the stream's type, as it is written and as the backward reads it),
// r = 1 / sqrt(mean z^2 + eps), y = z r w.  Backward, with zh = z r: dz = r (w dy - zh mean(w dy zh)) + dstream,
// dw = sum over rows of dy zh.  Both are bound by memory: each tensor is read or written once.  A block holds a row in
// registers (its waves on successive tiles of 512 columns, eight to a lane) between the sum and the outputs.  Forward, a
// block per row: 8192 x 4096 bf16 47.8 us (5.6 TB/s), 8192 x 2560 bf16 with the stream in fp32 48.1 (5.2 TB/s), 4096 x 5120
// into 8 bits with a scale per row 29.2 (5.0 TB/s); blocks that keep their weights and go over rows in turn 4 to 8% slower,
// and no better with the next row on its way.  Backward, a block goes over rows in turn and keeps its sums of dw, in 64 bits
// and rounded once; a second kernel joins them in a fixed order, in 64 bits too: 6123 x 2049 f32, forward and backward, 83 us
// (5.4 TB/s).
#include <algorithm>

#include "device_math.hpp"
#include "mss_internal.hpp"
#include "row_io.hpp"

namespace mss {
namespace {

struct NArgs {
    const void* x;         // (R, W)
    const void* res;       // (R, W), nullable
    const float* w;        // (W)
    void* out;             // (R, W)
    void* res_out;         // (R, W) with res
    float* rstd;           // (R), nullable
    float* scales;         // (R, G) of e4m3 outputs
    int64_t R, W;
    float eps, inv_w;
    int G;                 // 1: a scale per row; otherwise one per 128 columns
};

struct NoStream {};

constexpr int kMostWaves = 16;

// The joined value of the block's waves, each with its own v, the same in every thread.  `part` is one of two places
// used in turn: a wave is past a place when all of them have been at the other.
template <class Join>
__device__ __forceinline__ float join_waves(float v, float* part, int wave, int waves, int lane, Join join) {
    if (waves == 1) return v;
    if (lane == 0) part[wave] = v;
    __syncthreads();
    return join(lane < waves ? part[lane] : 0.0f);
}
__device__ __forceinline__ float wave_most(float v) {  // of values that are not negative
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) v = fmaxf(v, __shfl_xor(v, x));
    return v;
}

// The least value that an 8-bit output's scale is made for: a row of zeros has a scale that can be divided by.
constexpr float kLeastMost = 0x1p-100f, kE4m3Most = 448.0f;

template <class X, class S, bool F8, bool VEC, int NT>
__global__ __launch_bounds__(64 * kMostWaves) void rms_fwd_kernel(NArgs a) {
    constexpr bool kStream = !std::is_same<S, NoStream>::value;
    using ST = typename std::conditional<kStream, S, X>::type;
    __shared__ float parts[2][kMostWaves], mosts[2][kMostWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int waves = blockDim.x >> 6;
    const int64_t W = a.W;
    int rem[NT];
    int64_t at[NT];
    float w[NT][kE];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        at[j] = static_cast<int64_t>(wave + j * waves) * kTile;
        rem[j] = clamp_tile(W - at[j]);
        Raw<F32> q{};
        if (rem[j] > 0) {
            load8<F32, false>(a.w + at[j], W, rem[j], lane, q);
            settle8<F32, false>(W, rem[j], lane, q);
        }
        q.unpack(w[j]);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x, turn ^= 1) {
        const auto* x = static_cast<const typename X::storage*>(a.x) + row * W;
        Raw<X> rx[NT] = {};
        Raw<ST> rs[NT] = {};
#pragma unroll
        for (int j = 0; j < NT; ++j)
            if (rem[j] > 0) load8<X, VEC>(x + at[j], W, rem[j], lane, rx[j]);
        if constexpr (kStream) {
            const auto* s = static_cast<const typename ST::storage*>(a.res) + row * W;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (rem[j] > 0) load8<ST, VEC>(s + at[j], W, rem[j], lane, rs[j]);
        }
        float z[NT][kE], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (rem[j] > 0) settle8<X, VEC>(W, rem[j], lane, rx[j]);
            rx[j].unpack(z[j]);
            if constexpr (kStream) {
                if (rem[j] > 0) settle8<ST, VEC>(W, rem[j], lane, rs[j]);
                float s[kE];
                rs[j].unpack(s);
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    z[j][e] += s[e];
                    if (sizeof(typename ST::storage) == 2) z[j][e] = bf16_to_f32(f32_to_bf16(z[j][e]));
                }
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) sum = fmaf(z[j][e], z[j][e], sum);
        }
        if constexpr (kStream) {
            auto* so = static_cast<typename ST::storage*>(a.res_out) + row * W;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (rem[j] > 0) store8<ST, VEC>(so + at[j], rem[j], lane, z[j]);
        }
        sum = join_waves(wave_sum(sum), parts[turn], wave, waves, lane, [](float v) { return wave_sum(v); });
        const float r = rsqrtf(fmaf(sum, a.inv_w, a.eps));
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < kE; ++e) z[j][e] = z[j][e] * r * w[j][e];
        if constexpr (!F8) {
            auto* o = static_cast<typename X::storage*>(a.out) + row * W;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (rem[j] > 0) store8<X, VEC>(o + at[j], rem[j], lane, z[j]);
        } else {
            float most[NT];  // of the lane's columns, then of all that share its scale
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                most[j] = 0.0f;
#pragma unroll
                for (int e = 0; e < kE; ++e) most[j] = fmaxf(most[j], fabsf(z[j][e]));
            }
            if (a.G == 1) {
                float m = most[0];
#pragma unroll
                for (int j = 1; j < NT; ++j) m = fmaxf(m, most[j]);
                m = join_waves(wave_most(m), mosts[turn], wave, waves, lane, [](float v) { return wave_most(v); });
#pragma unroll
                for (int j = 0; j < NT; ++j) most[j] = m;
            } else {  // 128 columns are 16 lanes
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) most[j] = fmaxf(most[j], __shfl_xor(most[j], d));
            }
            auto* o = static_cast<uint8_t*>(a.out) + row * W;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float scale = fmaxf(most[j], kLeastMost) / kE4m3Most;
                if (a.G == 1) {
                    if (j == 0 && threadIdx.x == 0) a.scales[row] = scale;
                } else if ((lane & 15) == 0 && lane * kE < rem[j]) {
                    a.scales[row * a.G + at[j] / 128 + (lane >> 4)] = scale;
                }
                // The quotients z / scale as fp32 has them, at most 448: the product with the reciprocal and what it lacks,
                // put back.  The product alone has a rounding too many: next to the middle between two 8-bit values it
                // falls on the other side.
                const float inv = 1.0f / scale;
                int q[2];
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                    const float near = z[j][e] * inv;
                    z[j][e] = fmaf(fmaf(-near, scale, z[j][e]), inv, near);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // round to nearest even
                    const float* v = z[j] + 4 * h;
                    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                    q[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
                }
                const int t0 = lane * kE;
                uint8_t* p = o + at[j] + t0;
                if (t0 + kE <= rem[j]) {
                    if (VEC) *reinterpret_cast<int2*>(p) = make_int2(q[0], q[1]);
                    else __builtin_memcpy(p, q, 8);
                } else {
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        if (t0 + e < rem[j]) p[e] = static_cast<uint8_t>(q[e >> 2] >> (8 * (e & 3)));
                }
            }
        }
    }
}

struct NBArgs {
    const void* z;      // (R, W)
    const float* w;     // (W)
    const float* rstd;  // (R)
    const void* dy;     // (R, W)
    const void* dres;   // (R, W), nullable
    void* dx;           // (R, W)
    void* dz;           // (R, W), nullable
    float* part;        // (blocks, W), nullable
    int64_t R, W;
    float inv_w;
};

// X: the type of dy and dx, S: of z and the stream's gradients.
template <class X, class S, bool VEC, int NT>
__global__ __launch_bounds__(64 * kMostWaves) void rms_bwd_kernel(NBArgs a) {
    __shared__ float parts[2][kMostWaves];
    const int own_lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int waves = blockDim.x >> 6;
    const int64_t W = a.W;
    int rem[NT];
    int64_t at[NT];
    float w[NT][kE];
    double dw[NT][kE] = {};  // over many rows: 64 bits
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        at[j] = static_cast<int64_t>(wave + j * waves) * kTile;
        rem[j] = clamp_tile(W - at[j]);
        Raw<F32> q{};
        if (rem[j] > 0) {
            load8<F32, false>(a.w + at[j], W, rem[j], own_lane, q);
            settle8<F32, false>(W, rem[j], own_lane, q);
        }
        q.unpack(w[j]);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x, turn ^= 1) {
        // Rows that are no whole vectors: what a lane's place comes to in the last one is made for each row, not kept in
        // registers, of which two tiles leave none (1599 x 10001 bf16 with z in f32, forward and gradients: 156 -> 121 us).
        int lane = own_lane;
        if (!VEC && NT > 1) asm("" : "+v"(lane));
        const auto* zp = static_cast<const typename S::storage*>(a.z) + row * W;
        const auto* dp = static_cast<const typename X::storage*>(a.dy) + row * W;
        Raw<S> rz[NT] = {}, rr[NT] = {};
        Raw<X> rd[NT] = {};
        const float r = a.rstd[row];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            if (rem[j] > 0) {
                load8<S, VEC>(zp + at[j], W, rem[j], lane, rz[j]);
                load8<X, VEC>(dp + at[j], W, rem[j], lane, rd[j]);
            }
        if (a.dres) {
            const auto* rp = static_cast<const typename S::storage*>(a.dres) + row * W;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (rem[j] > 0) load8<S, VEC>(rp + at[j], W, rem[j], lane, rr[j]);
        }
        float z[NT][kE], d[NT][kE], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (rem[j] > 0) {
                settle8<S, VEC>(W, rem[j], lane, rz[j]);
                settle8<X, VEC>(W, rem[j], lane, rd[j]);
            }
            rz[j].unpack(z[j]);
            rd[j].unpack(d[j]);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                z[j][e] *= r;
                dw[j][e] += d[j][e] * z[j][e];
                d[j][e] *= w[j][e];
                sum = fmaf(d[j][e], z[j][e], sum);
            }
        }
        sum = join_waves(wave_sum(sum), parts[turn], wave, waves, lane, [](float v) { return wave_sum(v); });
        const float mean = sum * a.inv_w;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (rem[j] <= 0) continue;
            float s[kE];
            settle8<S, VEC>(W, rem[j], lane, rr[j]);
            rr[j].unpack(s);
#pragma unroll
            for (int e = 0; e < kE; ++e) s[e] = fmaf(r, fmaf(-mean, z[j][e], d[j][e]), s[e]);
            store8<X, VEC>(static_cast<typename X::storage*>(a.dx) + row * W + at[j], rem[j], lane, s);
            if (a.dz) store8<S, VEC>(static_cast<typename S::storage*>(a.dz) + row * W + at[j], rem[j], lane, s);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < NT; ++j)
        if (rem[j] > 0) {
            float part[kE];
#pragma unroll
            for (int e = 0; e < kE; ++e) part[e] = static_cast<float>(dw[j][e]);
            store8<F32, false>(a.part + blockIdx.x * W + at[j], rem[j], own_lane, part);
        }
}

// dw[c] = sum of part[p][c] over p, in 64 bits: 16 columns a block, 64 threads to a column, joined in a fixed order.
__global__ __launch_bounds__(1024) void rms_dw_kernel(const float* part, int64_t P, int64_t W, float* dw) {
    __shared__ double s[64][17];
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t col = blockIdx.x * 16ll + c;
    double v = 0.0;
    if (col < W)
#pragma unroll 8
        for (int64_t p = g; p < P; p += 64) v += part[p * W + col];
    s[g][c] = v;
    __syncthreads();
    for (int h = 32; h > 0; h >>= 1) {
        if (g < h) s[g][c] += s[g + h][c];
        __syncthreads();
    }
    if (g == 0 && col < W) dw[col] = static_cast<float>(s[0][c]);
}

// Waves a block and tiles a wave for rows of W columns.  One tile a wave as long as 16 waves reach: 8192 x 8192 bf16 92 us, 97
// with two.  But blocks that wait twice, for the row's greatest value too, are better small enough for several on a CU: into 8
// bits with a scale per row 8192 x 8192 117 us with one tile, 83 with two, 4096 x 5120 37.5 and 31.1.  Up to 4096 columns the wait
// costs as much as two tiles' fewer waves: 8192 x 2560 with the stream in fp32 44.5 and 46.8, in bf16 32.6 and 29.9.
struct NormPlan {
    int waves, nt;
};
NormPlan plan_norm(int64_t W, bool f8) {
    const int tiles = static_cast<int>((W + kTile - 1) / kTile);
    const int nt = tiles <= (f8 ? kMostWaves / 2 : kMostWaves) ? 1 : 2;
    return {(tiles + nt - 1) / nt, nt};
}
// The backward's blocks: ten waves for every CU, each block with the same number of rows, at least four if the CUs have work
// then, since a block's sums of dw are written and read again.  6123 x 2049 f32 45.6 us, 8192 x 2560 bf16 with z in f32 67.3, 2048
// x 1024 f32 13.8; 16 waves a CU and rows as they come 44.2, 69.1 and 16.7 (8192 x 5120 bf16 72.4 and 72.7).
int64_t bwd_blocks(int64_t R, int64_t W) {
    if (R == 0) return 0;
    const int64_t most = 256 * std::max(1, 10 / plan_norm(W, false).waves);
    const int64_t rows = std::max((R + most - 1) / most, std::min<int64_t>(4, (R + 255) / 256));
    return (R + rows - 1) / rows;
}

template <class X, class S, bool F8, bool VEC>
void fwd_nt(const NArgs& a, hipStream_t s) {
    const NormPlan p = plan_norm(a.W, F8);
    const dim3 grid(std::min(blocks_for(a.R, 1), 1u << 21)), block(64 * p.waves);  // (fewer than 2^32 threads)
    if (p.nt == 1) rms_fwd_kernel<X, S, F8, VEC, 1><<<grid, block, 0, s>>>(a);
    else rms_fwd_kernel<X, S, F8, VEC, 2><<<grid, block, 0, s>>>(a);
}
template <class X, class S>
void fwd_vec(const NArgs& a, bool f8, bool vec, hipStream_t s) {
    if (f8) vec ? fwd_nt<X, S, true, true>(a, s) : fwd_nt<X, S, true, false>(a, s);
    else vec ? fwd_nt<X, S, false, true>(a, s) : fwd_nt<X, S, false, false>(a, s);
}
template <class X, class S>
void bwd_vec(const NBArgs& a, bool vec, int64_t blocks, hipStream_t s) {
    const NormPlan p = plan_norm(a.W, false);
    const dim3 grid(static_cast<unsigned>(blocks)), block(64 * p.waves);
#define MSS_BWD(NT)                                                                \
    if (vec) rms_bwd_kernel<X, S, true, NT><<<grid, block, 0, s>>>(a);             \
    else rms_bwd_kernel<X, S, false, NT><<<grid, block, 0, s>>>(a)
    if (p.nt == 1) { MSS_BWD(1); }
    else { MSS_BWD(2); }
#undef MSS_BWD
}

}  // namespace

int64_t rms_norm_bwd_scratch(int64_t R, int64_t W) { return W == 0 ? 0 : (bwd_blocks(R, W) * W + 3) / 4 * 4; }

hipError_t launch_rms_norm_fwd(const NormLaunch& l, hipStream_t s) {
    NArgs a{};
    a.x = l.x; a.res = l.residual; a.w = l.weight; a.out = l.out; a.res_out = l.residual_out; a.rstd = l.rstd;
    a.scales = l.scales; a.R = l.R; a.W = l.W; a.eps = l.eps; a.inv_w = 1.0f / static_cast<float>(l.W); a.G = l.G;
    const bool f8 = l.scales != nullptr;
    if (l.x_bf16) {
        if (!l.residual) fwd_vec<BF16, NoStream>(a, f8, l.vec_ok, s);
        else if (l.residual_bf16) fwd_vec<BF16, BF16>(a, f8, l.vec_ok, s);
        else fwd_vec<BF16, F32>(a, f8, l.vec_ok, s);
    } else {
        if (!l.residual) fwd_vec<F32, NoStream>(a, f8, l.vec_ok, s);
        else if (l.residual_bf16) fwd_vec<F32, BF16>(a, f8, l.vec_ok, s);
        else fwd_vec<F32, F32>(a, f8, l.vec_ok, s);
    }
    return hipGetLastError();
}

hipError_t launch_rms_norm_bwd(const NormBwdLaunch& l, hipStream_t s) {
    NBArgs a{};
    a.z = l.z; a.w = l.weight; a.rstd = l.rstd; a.dy = l.dout; a.dres = l.dresidual_out; a.dx = l.dx; a.dz = l.dresidual;
    a.part = l.dweight ? l.scratch : nullptr;
    a.R = l.R; a.W = l.W; a.inv_w = 1.0f / static_cast<float>(l.W);
    const int64_t blocks = bwd_blocks(l.R, l.W);
    if (l.R > 0) {
        if (l.x_bf16) {
            if (l.z_bf16) bwd_vec<BF16, BF16>(a, l.vec_ok, blocks, s);
            else bwd_vec<BF16, F32>(a, l.vec_ok, blocks, s);
        } else {
            if (l.z_bf16) bwd_vec<F32, BF16>(a, l.vec_ok, blocks, s);
            else bwd_vec<F32, F32>(a, l.vec_ok, blocks, s);
        }
    }
    if (l.dweight) rms_dw_kernel<<<dim3(static_cast<unsigned>((l.W + 15) / 16)), dim3(1024), 0, s>>>(a.part, l.R > 0 ? blocks : 0, l.W, l.dweight);
    return hipGetLastError();
}

}  // namespace mss
