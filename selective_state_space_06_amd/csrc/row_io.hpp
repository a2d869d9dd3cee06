// row_io.hpp -- rows of a (rows, L) tensor read and written by waves in tiles of 512 steps, eight
// consecutive steps to a lane, and moves between a wave's lanes.
#pragma once

#include "device_math.hpp"

namespace mss {

// For a kernel's lambdas: they move values between lanes and meet at barriers, which must not end up behind a call
// (the gated scan's backward walk, which the compiler outlined when it had a second call site, gave wrong
// results).  The build refuses kernels with calls.
#define MSS_INLINED __attribute__((always_inline))

// Values as types, for lambdas that are built twice.
struct True { static constexpr bool value = true; };
struct False { static constexpr bool value = false; };

constexpr int kE = 8;           // steps per lane
constexpr int kTile = 64 * kE;  // steps per wave and tile

// Steps of a tile that begins n steps before an end: 0 .. 512.
__device__ __forceinline__ int clamp_tile(int64_t n) { return n < 0 ? 0 : n > kTile ? kTile : static_cast<int>(n); }

// v of the lane CTRL names (a DPP move), `old` where there is none.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float old, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
// The sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0x111>(0.0f, v);  // row_shr 1, 2, 4, 8: the last lane of each 16-lane row has its row
    v += dpp<0x112>(0.0f, v);
    v += dpp<0x114>(0.0f, v);
    v += dpp<0x118>(0.0f, v);
    v += dpp<0x142, 0xA>(0.0f, v);  // row_bcast 15 into rows 1 and 3, row_bcast 31 into rows 2 and 3
    v += dpp<0x143, 0xC>(0.0f, v);
    return lane_of(v, 63);
}

// A lane's eight elements of a tile as they lie in memory.
template <class E>
struct Raw {
    uint4 q[kE / E::kPerVec];
    __device__ __forceinline__ void unpack(float* v) const {
#pragma unroll
        for (int j = 0; j < kE / E::kPerVec; ++j) E::unpack(q[j], v + j * E::kPerVec);
    }
};

// w moved down by n elements (0 .. kPerVec, those that leave are dropped, zeros enter).
template <class E>
__device__ __forceinline__ uint4 drop(const uint4& w, int n) {
    if (E::kPerVec == 4) {
        const uint4 a = n & 1 ? make_uint4(w.y, w.z, w.w, 0) : w;
        const uint4 b = n & 2 ? make_uint4(a.z, a.w, 0, 0) : a;
        return n & 4 ? make_uint4(0, 0, 0, 0) : b;
    }
    uint64_t lo = static_cast<uint64_t>(w.y) << 32 | w.x, hi = static_cast<uint64_t>(w.w) << 32 | w.z;
    if (n & 8) lo = hi = 0;
    if (n & 4) lo = hi, hi = 0;
    const int k = 16 * (n & 3);
    if (k) lo = lo >> k | hi << (64 - k), hi >>= k;
    return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                      static_cast<uint32_t>(hi >> 32));
}

// Loads the lane's elements of the tile at p, of `rem` steps (512 inside a row of L), as settle8 then
// leaves them: zeros past the end.  VEC: rows are whole aligned 16-byte vectors; otherwise element-aligned
// 16-byte loads.  Of a row's last, partial vector (and of those past it) the last 16 bytes of the row are
// loaded, at an address that is always inside the row, and moved down when they are used: loaded element
// by element, or moved at once, each stream waits for its own tail
// (4 x 5120 x 2047 bf16 gated scan forward: 99 us by elements, 85 moved at once, 76 as here).
template <class E, bool VEC>
__device__ __forceinline__ void load8(const typename E::storage* p, int64_t L, int rem, int lane, Raw<E>& w) {
    constexpr int V = E::kPerVec;
    const int t0 = lane * kE;
    if (rem >= kTile) {
#pragma unroll
        for (int j = 0; j < kE / V; ++j) {
            if (VEC) w.q[j] = *reinterpret_cast<const uint4*>(p + t0 + j * V);
            else __builtin_memcpy(&w.q[j], p + t0 + j * V, 16);
        }
    } else if (VEC) {
#pragma unroll
        for (int j = 0; j < kE / V; ++j) {
            w.q[j] = make_uint4(0, 0, 0, 0);
            if (t0 + j * V < rem) w.q[j] = *reinterpret_cast<const uint4*>(p + t0 + j * V);
        }
    } else if (L >= V) {
#pragma unroll
        for (int j = 0; j < kE / V; ++j) {  // rem < V only past a row's first tile
            const int u = t0 + j * V < rem - V ? t0 + j * V : rem - V;
            __builtin_memcpy(&w.q[j], p + u, 16);
        }
    } else {  // a row shorter than a vector
        float v[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) v[e] = t0 + e < rem ? E::load1(p, t0 + e) : 0.0f;
#pragma unroll
        for (int j = 0; j < kE / V; ++j) w.q[j] = E::pack(v + j * V);  // exact: they came from this storage type
    }
}
template <class E, bool VEC>
__device__ __forceinline__ void settle8(int64_t L, int rem, int lane, Raw<E>& w) {
    constexpr int V = E::kPerVec;
    if (VEC || rem >= kTile || L < V) return;
#pragma unroll
    for (int j = 0; j < kE / V; ++j) {
        const int over = lane * kE + j * V + V - rem;  // elements past the end
        w.q[j] = drop<E>(w.q[j], over < 0 ? 0 : over > V ? V : over);
    }
}

// The lane's elements written to the tile.
template <class E, bool VEC>
__device__ __forceinline__ void store8(typename E::storage* p, int rem, int lane, const float* v) {
    constexpr int V = E::kPerVec;
    const int t0 = lane * kE;
    const bool whole = rem >= kTile;
#pragma unroll
    for (int j = 0; j < kE / V; ++j) {
        const int t = t0 + j * V;
        const uint4 w = E::pack(v + j * V);
        if (whole || t + V <= rem) {
            if (VEC) *reinterpret_cast<uint4*>(p + t) = w;
            else __builtin_memcpy(p + t, &w, 16);
        } else if (!VEC) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (t + e < rem) E::store1(p, t + e, v[j * V + e]);
        }
    }
}

// How the four waves of a block share channels when a sum over the batch is wanted: `ways` waves to a
// channel, each with every ways-th batch, joined through LDS in order; one launch then gives the sum,
// where partial sums per row and a second kernel take 4 to 5 us more.  A batch that leaves too few waves
// that way (under 4096, four a SIMD) goes by rows and parts.
__host__ __device__ inline int channel_ways(int64_t batch) { return batch == 1 ? 1 : batch == 2 ? 2 : 4; }
inline bool goes_by_parts(int64_t batch, int64_t channels, int waves_per_channel, int rows_at_once) {
    return batch > rows_at_once && channels * waves_per_channel < 4096;
}

// Blocks for n items, `per` a block; kernels stride over what a capped grid leaves.
inline unsigned blocks_for(int64_t n, int64_t per) {
    const int64_t b = (n + per - 1) / per;
    return static_cast<unsigned>(b < 1 ? 1 : b > (1 << 22) ? (1 << 22) : b);
}

}  // namespace mss
