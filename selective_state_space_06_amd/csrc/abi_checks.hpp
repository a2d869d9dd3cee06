// abi_checks.hpp -- checks of tensor descriptors shared by the files of the extern "C" boundary.
// They look at descriptors alone: no HIP call, no device memory.
#pragma once

#include <initializer_list>
#include <stddef.h>
#include <stdint.h>

#include "mamba_scan.h"

namespace mss {
namespace abi {

inline int64_t numel(const mss_tensor_t& t) {
    int64_t n = 1;
    for (int i = 0; i < t.ndim; ++i) n *= t.shape[i];
    return n;
}

inline size_t elem_size(int32_t dtype) { return dtype == MSS_BF16 ? 2 : 4; }

inline bool shape_is(const mss_tensor_t& t, int ndim, int64_t s0, int64_t s1 = 0, int64_t s2 = 0, int64_t s3 = 0) {
    if (t.ndim != ndim) return false;
    const int64_t s[4] = {s0, s1, s2, s3};
    for (int i = 0; i < ndim; ++i)
        if (t.shape[i] != s[i]) return false;
    return true;
}

inline bool dense(const mss_tensor_t& t) {
    if (numel(t) == 0) return true;
    int64_t expect = 1;
    for (int i = t.ndim - 1; i >= 0; --i) {
        if (t.shape[i] != 1 && t.stride[i] != expect) return false;
        expect *= t.shape[i];
    }
    return true;
}

inline bool aligned(const mss_tensor_t& t, size_t a) {
    return (reinterpret_cast<uintptr_t>(t.data) % a) == 0;
}

struct Range {
    uintptr_t lo, hi;
};
inline Range range_of(const mss_tensor_t* t) {
    if (!t || !t->data) return {0, 0};
    const uintptr_t lo = reinterpret_cast<uintptr_t>(t->data);
    return {lo, lo + static_cast<uintptr_t>(numel(*t)) * elem_size(t->dtype)};
}
inline bool overlap(const mss_tensor_t* a, const mss_tensor_t* b) {
    const Range x = range_of(a), y = range_of(b);
    if (x.lo == x.hi || y.lo == y.hi) return false;
    return x.lo < y.hi && y.lo < x.hi;
}

// Status of one descriptor before its extents are compared: NULL descriptor or NULL data
// (for a non-empty tensor) -> NULL_ARG; ndim outside 1..4, a negative extent or an element count
// beyond 2^48 (so that no later size computation can overflow) -> SHAPE.
inline int check_desc(const mss_tensor_t* t, bool required) {
    if (!t) return required ? MSS_ERR_NULL_ARG : MSS_OK;
    if (t->ndim < 1 || t->ndim > 4) return MSS_ERR_SHAPE;
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] < 0) return MSS_ERR_SHAPE;
        if (__builtin_mul_overflow(n, t->shape[i], &n) || n > (int64_t{1} << 48)) return MSS_ERR_SHAPE;
    }
    if (!t->data && n != 0) return MSS_ERR_NULL_ARG;
    return MSS_OK;
}

template <size_t K>
int check_descs(const mss_tensor_t* const (&req)[K], std::initializer_list<const mss_tensor_t*> opt) {
    for (const mss_tensor_t* t : req)
        if (!t) return MSS_ERR_NULL_ARG;
    for (const mss_tensor_t* t : req) {
        const int s = check_desc(t, true);
        if (s != MSS_OK) return s;
    }
    for (const mss_tensor_t* t : opt) {
        const int s = check_desc(t, false);
        if (s != MSS_OK) return s;
    }
    return MSS_OK;
}

}  // namespace abi
}  // namespace mss
