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

inline size_t elem_size(int32_t dtype) { return dtype == MSS_F8E4M3 ? 1 : dtype == MSS_BF16 ? 2 : 4; }

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

using Ts = std::initializer_list<const mss_tensor_t*>;

inline bool act_dtype(int32_t d) { return d == MSS_F32 || d == MSS_BF16; }

inline bool all_dtype(Ts ts, int32_t d) {
    for (const mss_tensor_t* t : ts)
        if (t && t->dtype != d) return false;
    return true;
}

// Dense, element-aligned.
inline bool laid_out(Ts ts) {
    for (const mss_tensor_t* t : ts)
        if (t && (!dense(*t) || !aligned(*t, elem_size(t->dtype)))) return false;
    return true;
}

// No output overlaps an input or another output.
inline bool apart(Ts ins, Ts outs) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const mss_tensor_t* t : ins)
            if (overlap(*o, t)) return false;
        for (auto p = o + 1; p != outs.end(); ++p)
            if (overlap(*o, *p)) return false;
    }
    return true;
}

// Scratch of at least n floats, 16-byte aligned; may be NULL when n is 0.
inline int check_scratch(const mss_tensor_t* t, int64_t n) {
    if (n == 0 && !t) return MSS_OK;
    if (!t) return MSS_ERR_NULL_ARG;
    const int s = check_desc(t, true);
    if (s != MSS_OK) return s;
    if (t->ndim != 1 || t->shape[0] < n) return MSS_ERR_SHAPE;
    if (t->dtype != MSS_F32) return MSS_ERR_DTYPE;
    if (!dense(*t) || !aligned(*t, 16)) return MSS_ERR_LAYOUT;
    return MSS_OK;
}

template <class T>
T* ptr(const mss_tensor_t* t) {
    return t && numel(*t) > 0 ? static_cast<T*>(t->data) : nullptr;
}

inline bool whole_vectors(int64_t row, int32_t dtype, Ts ts) {
    if (row * static_cast<int64_t>(elem_size(dtype)) % 16 != 0) return false;
    for (const mss_tensor_t* t : ts)
        if (t && !aligned(*t, 16)) return false;
    return true;
}

}  // namespace abi
}  // namespace mss
