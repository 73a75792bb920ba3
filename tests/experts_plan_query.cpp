// Prints the plans of routed-expert calls (plan_experts in w4a16_weight_only_amd/csrc/awq_plan.cpp):
// one line "T topk E K inner N group_size cus halves" in (halves: 1 gate_up, 2 down, 3 mlp), one out:
// "status two_terms" and for either product "stream ranked rows tiles col_tiles splits grid".
#include <cinttypes>
#include <cstdio>
#include <initializer_list>

#include "../w4a16_weight_only_amd/csrc/awq_plan.h"

int main() {
  int64_t T, topk, E, K, inner, N, gs;
  int cus, halves;
  while (std::scanf("%" SCNd64 " %" SCNd64 " %" SCNd64 " %" SCNd64 " %" SCNd64 " %" SCNd64 " %" SCNd64 " %d %d", &T,
                    &topk, &E, &K, &inner, &N, &gs, &cus, &halves) == 9) {
    awq::ExpertsPlan p;
    const int st = awq::plan_experts(T, topk, E, K, inner, N, gs, cus, halves & 1, halves & 2, p);
    std::printf("%d %d", st, (int)p.two_terms);
    for (const awq::ExpertPlan* q : {&p.up, &p.down})
      std::printf(" %d %d %d %" PRId64 " %d %d %" PRId64, (int)q->stream, (int)q->ranked, q->rows, q->tiles, q->col_tiles,
                  q->splits, q->grid);
    std::printf("\n");
  }
  return 0;
}
