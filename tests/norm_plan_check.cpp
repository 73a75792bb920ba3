// awq_add_norm's launches (norm_waves and what follows from it in w4a16_weight_only_amd/csrc/awq_plan.h) on the CPU,
// for every row length: whatever plan_norm takes is launched within HIP's limits, with lanes for a whole row.  Prints
// "lengths checked: <n>" and exits 0, or prints the first failure and exits 1.
#include <cinttypes>
#include <cstdio>

#include "../include/awq_w4a16.h"
#include "../w4a16_weight_only_amd/csrc/awq_plan.h"

using namespace awq;

int main() {
  const int64_t counts[] = {1, 2, 3, 5, 4096, (int64_t(1) << 22) - 1, int64_t(1) << 22, int64_t(1) << 23, (int64_t(1) << 24) - 1,
                            int64_t(1) << 24};
  long checked = 0;
  for (int64_t H = 1; H <= kNormMaxH; ++H) {
    const int waves = norm_waves(H), threads = norm_threads(waves), rows = norm_rows(waves);
    const int64_t most = norm_launch_rows(waves);
    bool ok = threads <= 1024 && rows * waves * 64 == threads && most >= 1 && most % rows == 0;
    ok = ok && (int64_t)waves * 64 * (waves == 1 ? 16 : 32) >= H;  // two or four pieces of eight a lane
    for (const int64_t T : counts) {
      if (plan_norm(T, H, H, H, 0) != AWQ_OK) ok = false;
      int64_t covered = 0;
      int launches = 0;
      for (int64_t first = 0; first < T; first += most, ++launches) {
        const int64_t n = T - first < most ? T - first : most;
        const int64_t grid = (n + rows - 1) / rows;
        if (grid < 1 || grid * threads >= int64_t(1) << 32) ok = false;
        covered += n;
      }
      ok = ok && covered == T && launches <= 5 && (T > (1 << 20) || launches == 1);
      if (!ok) {
        std::fprintf(stderr, "H %" PRId64 " T %" PRId64 ": %d waves, %d threads, %" PRId64 " rows a launch\n", H, T, waves, threads, most);
        return 1;
      }
    }
    ++checked;
  }
  if (plan_norm(1, kNormMaxH + 1, kNormMaxH + 1, kNormMaxH + 1, 0) != AWQ_ERR_UNSUPPORTED) return 1;
  std::printf("lengths checked: %ld\n", checked);
  return 0;
}
