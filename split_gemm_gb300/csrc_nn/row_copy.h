// Where one of a row's copies into shared memory reads, in plain C++ so that the host can check it.
#pragma once

#ifndef __CUDACC__
#define SGB_HOST_DEVICE
#else
#define SGB_HOST_DEVICE __host__ __device__ __forceinline__
#endif

namespace sgb {
namespace ln {

// A copy of `per` elements at column c of a row of `cols`: `at` elements from the row's start, of which `count` are read and the
// others come as zeros.  A copy with nothing to read takes an aligned address too, as an unaligned one is undefined
// whatever its size: that of the vector in which the row begins, `front` elements before it.
struct RowCopy {
    int at, count;
};

SGB_HOST_DEVICE RowCopy row_copy(int c, int per, int cols, int front)
{
    const int left = cols - c;
    return left <= 0 ? RowCopy{-front, 0} : RowCopy{c, left < per ? left : per};
}

}  // namespace ln
}  // namespace sgb
