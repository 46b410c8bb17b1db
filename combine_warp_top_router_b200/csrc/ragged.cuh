// ragged.cuh -- how an expert's rows are split into tiles (internal; plain integer
// arithmetic, also compiled for the host by the tests).
#pragma once

#ifdef __CUDACC__
#define MD_BOTH __host__ __device__ __forceinline__
#else
#define MD_BOTH inline
#endif

namespace md {

// Tiles of c rows, at most `most` rows each.  0 <= c < 2^31 - most.
MD_BOTH int ragged_tiles(int c, int most) { return (c + most - 1) / most; }

// Rows of each of them but the last: equal tiles, rounded up to a multiple of `gran`, which
// divides `most`.  c up to 2^31 - 1 - most: nothing here adds to c.
MD_BOTH int ragged_rows(int c, int most, int gran)
{
    const int nt = ragged_tiles(c, most);
    return nt ? ((c - 1) / nt + gran) / gran * gran : 0;
}

}  // namespace md
