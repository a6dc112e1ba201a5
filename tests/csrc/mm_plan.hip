// Host program: which kernel a block-scaled product takes, and over how many workgroups k is spread. Arguments: T N K f32 for each
// call; prints "kernel shares" for each. No GPU is used.
#include <stdio.h>
#include <stdlib.h>

#include "../../activation_sparse_ffn_predictor_amd/csrc/mm.h"

int main(int n, char** a) {
  static const char* const names[] = {"few", "some32", "some64", "some128", "tile128", "tile256"};
  for (int i = 1; i + 3 < n; i += 4) {
    const sffn::MmPlan p = sffn::mm_plan(atoi(a[i]), atoi(a[i + 1]), atoi(a[i + 2]), atoi(a[i + 3]) != 0);
    printf("%s %d\n", names[p.how], p.ks);
  }
  return 0;
}
