// top_lists.hpp -- the k greatest of a row of logits, as lists of 64-bit keys that waves keep and merge (beam
// selection, token log probabilities).
//
// Logits are compared as whole numbers of the same order (order_of), with the token behind them as one
// 64-bit key (a higher value, then a lower token).  A wave keeps its k best as a list spread over its
// lanes, entry j in lane j, best first; a candidate that beats entry k - 1 is inserted by a shift of the
// entries behind it.  Of n values in no order about k (1 + ln(n / k)) do so when they come, and a tile
// without one costs a compare; the first tile is cut at (16 bits of) the k-th greatest of its lanes'
// greatest values first, which leaves little more than k of it.  Sorted lists are merged by taking the
// greatest head k times.
#pragma once

#include "device_math.hpp"
#include "row_io.hpp"

namespace mss {

__device__ __forceinline__ int shift_up(int v) { return __builtin_amdgcn_update_dpp(v, v, 0x138, 0xF, 0xF, false); }
__device__ __forceinline__ uint64_t join64(uint32_t hi, uint32_t lo) { return static_cast<uint64_t>(hi) << 32 | lo; }

__device__ __forceinline__ uint64_t ballot(bool b) { return __builtin_amdgcn_ballot_w64(b); }
__device__ __forceinline__ int first_of(uint64_t lanes) { return __builtin_ctzll(lanes); }
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ uint64_t lane_of(uint64_t v, int lane) {
    return join64(lane_of(static_cast<uint32_t>(v >> 32), lane), lane_of(static_cast<uint32_t>(v), lane));
}
// The greatest of every lane's w, the same in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t w) {
#define MSS_MAX(CTRL, ROWS)                                                                                      \
    {                                                                                                            \
        const uint32_t o = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), CTRL, ROWS, 0xF, false);          \
        w = o > w ? o : w;                                                                                       \
    }
    MSS_MAX(0x111, 0xF)  // the steps of wave_sum
    MSS_MAX(0x112, 0xF)
    MSS_MAX(0x114, 0xF)
    MSS_MAX(0x118, 0xF)
    MSS_MAX(0x142, 0xA)
    MSS_MAX(0x143, 0xC)
#undef MSS_MAX
    return lane_of(w, 63);
}

// Floats as whole numbers of the same order (-0 as +0), and back.
__device__ __forceinline__ uint32_t order_of(float v) {
    const int b = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(b ^ (b >> 31 | INT32_MIN));
}
__device__ __forceinline__ float value_of(uint32_t o) {
    const int b = static_cast<int>(o);
    return __int_as_float(b ^ (~(b >> 31) | INT32_MIN));
}
constexpr uint32_t kLeast = 0x00800000u;  // order_of the least finite value; -inf is one less
// A logit and its token.  kNone comes before every key of a finite or +inf logit and after those of -inf.
__device__ __forceinline__ uint64_t key_of(uint32_t order, int token) { return join64(order, ~static_cast<uint32_t>(token)); }
__device__ __forceinline__ int token_of(uint64_t key) { return static_cast<int>(~static_cast<uint32_t>(key)); }
constexpr uint64_t kNone = static_cast<uint64_t>(kLeast) << 32;

// The list of a wave: lane j holds the j-th best key.
struct List {
    uint64_t key = kNone;
    uint64_t last = kNone;  // entry k - 1, the same in every lane
    // the same new key in every lane
    __device__ __forceinline__ void insert(uint64_t n, int k, int lane) {
        const int at = __popcll(ballot(key > n));
        const uint64_t below = join64(shift_up(static_cast<int>(key >> 32)), shift_up(static_cast<int>(key)));
        key = lane > at ? below : lane == at ? n : key;
        last = lane_of(key, k - 1);
    }
};

// The k greatest of `count` (at most 64) sorted lists of k keys, one behind the other, in lane order.
__device__ __forceinline__ uint64_t merge_lists(const uint64_t* lists, int count, int k, int lane) {
    uint64_t mine = kNone, head = lane < count ? lists[lane * k] : kNone;
    int at = 0;
    for (int j = 0; j < k; ++j) {
        const uint32_t most = wave_max(static_cast<uint32_t>(head >> 32));
        if (most <= kLeast && ballot(head > kNone) == 0) break;
        uint64_t who = ballot(static_cast<uint32_t>(head >> 32) == most);
        if (who & (who - 1)) {  // equal logits: the lowest token
            const uint32_t low = wave_max(static_cast<uint32_t>(head >> 32) == most ? static_cast<uint32_t>(head) : 0);
            who = ballot(head == join64(most, low));
        }
        const int src = first_of(who);
        const uint64_t key = lane_of(head, src);
        if (lane == j) mine = key;
        if (lane == src) head = ++at < k ? lists[lane * k + at] : kNone;
    }
    return mine;
}

}  // namespace mss
