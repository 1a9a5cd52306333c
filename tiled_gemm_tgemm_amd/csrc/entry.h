// What the C entry points of the operators on 16-bit tiles share: types, byte
// ranges of arguments, workspaces.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm.h"

namespace tgemm {
namespace entry {

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t size_of(tgemm_dtype_t t) { return t == TGEMM_F32 ? 4 : 2; }
inline bool known(tgemm_dtype_t t) { return t == TGEMM_F32 || t == TGEMM_BF16 || t == TGEMM_F16; }

inline tgemm_status_t from_hip(hipError_t e) { return e == hipSuccess ? TGEMM_SUCCESS : TGEMM_ERROR_HIP; }

// A byte range that a call reads or writes.
struct Range {
    uintptr_t lo = 0, hi = 0;
};

// False if `rows` rows of `cols` elements, `ld` apart, are not at p: null,
// misaligned or past the end of the address space.  Nothing is at an empty one.
inline bool at(const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size, Range &r)
{
    r = Range();
    if (rows == 0 || cols == 0) return true;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p == nullptr || lo % size) return false;
    const unsigned __int128 end =
        (unsigned __int128)lo + ((unsigned __int128)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * size;
    if (end > (unsigned __int128)UINTPTR_MAX) return false;
    r.lo = lo;
    r.hi = (uintptr_t)end;
    return true;
}

inline bool apart(const Range &a, const Range &b) { return a.lo >= b.hi || b.lo >= a.hi; }

// `count` matrices of `rows` rows of `cols` elements, the rows ld and the matrices
// `stride` apart, that share none: one after another, or side by side.
inline bool separate(int64_t count, int64_t rows, int64_t cols, int64_t ld, int64_t stride)
{
    return count < 2 || stride >= (rows - 1) * ld + cols || (stride >= cols && ld >= (count - 1) * stride + cols);
}

// What is written overlaps nothing else.
inline bool disjoint(const Range *written, int n_written, const Range *read, int n_read)
{
    for (int i = 0; i < n_written; ++i) {
        for (int j = i + 1; j < n_written; ++j)
            if (!apart(written[i], written[j])) return false;
        for (int j = 0; j < n_read; ++j)
            if (!apart(written[i], read[j])) return false;
    }
    return true;
}

// The workspace's bytes and range; false if it is missing, misaligned or small.
inline bool room_at(void *workspace, size_t bytes, int64_t need, Range &r)
{
    if (need == 0) return true;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(workspace);
    if (workspace == nullptr || lo % 16 || bytes < (size_t)need || bytes > UINTPTR_MAX - lo) return false;
    r.lo = lo;
    r.hi = lo + (size_t)need;
    return true;
}

template <class T>
T *in(void *workspace, int64_t offset) { return offset < 0 ? nullptr : (T *)((char *)workspace + offset); }

}  // namespace entry
}  // namespace tgemm
