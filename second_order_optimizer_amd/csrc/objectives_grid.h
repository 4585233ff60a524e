// Workgroups of a launch over rows: plain host C++, so that the arithmetic can
// be checked without a GPU.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace kfac {

constexpr int kCus = 256;

// Workgroups for so many rows: as many as are resident, none for none.  Of
// workgroups with a row each at a time, fewer that all walk as many rows (4096 x
// 12000 bf16 47.5 -> 44.7 us); with four short rows at a time arithmetic counts
// and that loses (16384 x 500 17.2 -> 19.3 us).
inline int grid_of(int64_t rows, int teams, int per_cu) {
  const int64_t need = (rows + teams - 1) / teams, most = static_cast<int64_t>(kCus) * per_cu;
  if (need == 0) return 0;
  if (teams > 1) return static_cast<int>(std::min(need, most));
  const int64_t rounds = (need + most - 1) / most;
  return static_cast<int>((need + rounds - 1) / rounds);
}

}  // namespace kfac
