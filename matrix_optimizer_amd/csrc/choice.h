// Which kernel a product takes: a rule on sizes alone, shared with the host's
// checks.
#pragma once
#include <stdint.h>

namespace muon {

// Single waves take time for each 16 to 64 rows of a run, tiles hardly any more for a longer run, but they
// take their whole time with CUs idle where there are few: the rows of the mean expert up to which waves are
// the faster fall with the number of tiles, tiles = experts with rows x tiles along n, and faster from where
// tiles take half of the card on.  Measured with as many rows for each expert, waves and tiles in us:
//   256 x 256 tiles (16-byte rows, bf16 results): 16 tiles (one [4096, 7168]) 128 rows 42 and 62; 32 ([8192,
//     28672]) 64 rows 155 and 203; 64 (four [4096, 7168]) 32 rows 46 and 54, 64 rows 77 and 57; 112 ([28672,
//     8192]) 16 rows 59 and 62, 24 rows 81 and 61; 128 (eight [4096, 7168]) 8 rows 50 and 55, 16 rows 62 and 56;
//     256 (32 [2048, 4096]) 4 rows 52 and 50; 1024 (64 [4096, 7168]) 2 rows 338 and 372, 4 rows 368 and 373, 8
//     rows 398 and 375.
//   128 x 128 tiles, 16-byte rows (fp32 results): 128 (two [8192, 7168]) 64 rows 85 and 120; 224 ([28672, 8192])
//     32 rows 110 and 132, 48 rows 152 and 133; 256 (eight [4096, 4096]) 16 rows 71 and 70, 32 rows 109 and 71;
//     512 (32 [2048, 4096]) 8 rows 88 and 94, 16 rows 102 and 96; 2048 (128 [2048, 4096]) 8 rows 370 and 390, 16
//     rows 412 and 396, 64 rows 794 and 401.
//   128 x 128 tiles, other rows, of which waves read the pieces slowly: 64 (two [4096, 4099]) 64 rows 71 and 84;
//     128 (eight [2048, 4099]) 16 rows 67 and 85, 32 rows 101 and 86; 224 ([28672, 8195]) 8 rows 133 and 130, 16
//     rows 160 and 130; 1024 (64 [2048, 2051]) 1 row 129 and 107.
// The runs' lengths are on the device.  Uneven ones favour tiles, which read a run's matrix once for 128 or 256
// rows: with every row in one run, 2 rows of the mean of 64 [4096, 7168] 131 and 62, 8 rows 288 and 81; to fp32 8
// rows 259 and 124, 64 rows 1165 and 298.  So the limit is at the lower end of what even runs bear.
constexpr int64_t most_rows_of_waves(int64_t tiles, bool large, bool pieces) {
  const int64_t half = pieces && !large ? 256 : 128, c = large ? 2048 : pieces ? 8192 : 4096, least = large ? 3 : pieces ? 8 : 1;
  const int64_t rows = c / (tiles < half ? 1 : 2) / (tiles < 1 ? 1 : tiles);
  return rows < least ? least : rows > 64 ? 64 : rows;
}

}  // namespace muon
