// Where one of a row's copies into shared memory reads, in plain C++ so that the host can check it.
#pragma once

#ifndef __CUDACC__
#define SGB_HOST_DEVICE
#else
#define SGB_HOST_DEVICE __host__ __device__ __forceinline__
#endif

namespace sgb {
namespace ln {

// A copy of `per` elements at column c of a row of `cols` (`whole`: cols is a multiple of per): `at` elements from the row's start, of
// which `count` are read and the others come as zeros.  A copy with nothing to read takes an aligned address too, as an unaligned one is undefined
// whatever its size: that of the vector in which the row begins, `front` elements before it.
struct RowCopy {
    int at, count;
};

SGB_HOST_DEVICE RowCopy row_copy(int c, int per, int cols, int front, bool whole)
{
    // No columns leave nothing anyway, but are the same for all copies of a row (8192 x 16384 fp32 forward 180 us, 188 unasked).
    const int left = cols - c, count = cols == 0 || left <= 0 ? 0 : whole || left >= per ? per : left;
    return RowCopy{count ? c : -front, count};
}

}  // namespace ln
}  // namespace sgb
