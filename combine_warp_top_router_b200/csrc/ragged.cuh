// ragged.cuh -- how an expert's rows are split into tiles, and which kernel form takes
// them (internal; plain integer arithmetic, also compiled for the host by the tests).
#pragma once

#include <stdint.h>

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

// Row tiles of `most` rows that E ranges of `rows` rows make, at most: sum of ceil(c / most)
// <= rows / most + (experts with rows) (1 - 1 / most).
MD_BOTH int64_t ragged_most_tiles(int64_t rows, int E, int most) { return rows / most + (rows < E ? rows : E); }

// Whether a call takes k_expert_few.  With 64 rows to an expert and fewer it is bound by reading the
// weights, and that kernel's deeper ring of weights does that better; above, its narrow tiles
// read them again for every 64 rows (64 experts of 2048 x 2048, us, few / wide: 16 rows 83 / 90,
// 64 rows 98 / 94, 96 rows 159 / 96, 256 rows 377 / 119).  A call with no more wide tiles
// than there are SM pairs leaves SMs idle in the wide form, and takes the narrow tiles as long as
// those make one and a half rounds of the SMs at most.  1 to 32 experts, K and N of 256 to 4096, few / wide:
// 0.5 to 1.3 in one round and 0.6 to 1.3 in one and a half, below 1 but for K = 4096, 0.7 to 2.1 in
// two, 1.0 to 3.8 in more (1 expert of 4096 rows, 4096 x 1024: 110 / 29 us; 8 of 256 rows, 1024 x 1024:
// 19 / 13); short contractions at the low end.  `sub`: output columns of a wide tile, twice a narrow one's.
MD_BOTH bool ragged_few(int64_t rows, int E, int64_t columns, int sub, int sms)
{
    const int64_t wide = ragged_most_tiles(rows, E, 256) * ((columns + sub - 1) / sub);
    const int64_t few = ragged_most_tiles(rows, E, 64) * ((columns + sub / 2 - 1) / (sub / 2));
    return rows <= (int64_t)64 * E || (wide <= sms / 2 && 2 * few <= 3 * (int64_t)sms);
}

}  // namespace md
