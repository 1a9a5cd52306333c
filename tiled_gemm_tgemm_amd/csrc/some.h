// Several adjacent values of a row at once, wherever it starts (device memory
// takes 16-byte accesses at any element's address) and ends.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tgemm {
namespace m16 {

template <class In, int N>
struct Some {
    typedef In type __attribute__((ext_vector_type(N), aligned(sizeof(In))));
};

// N adjacent values, `left` of them there, zero past those.
template <class In, int N>
__device__ __forceinline__ void load_some(const In *p, int64_t left, In (&v)[N])
{
    if (left >= N) {
        const typename Some<In, N>::type got = *(const typename Some<In, N>::type *)p;
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = got[e];
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = e < left ? p[e] : (In)0.0f;
    }
}

}  // namespace m16
}  // namespace tgemm
