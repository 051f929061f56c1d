// Host rules of the adapter pool's launches (no GPU needed): for each "m n_out k r n" read from standard input, whether the
// gradients are split over the CTAs of a cluster on a GPU of 148 SMs.
#include <cstdio>

#include "qlora_nf4.h"
#include "../../bit_nf4_quantized_27_b200/csrc/pool_kernels.cuh"

int main() {
  long long m, n_out, k;
  int r, n;
  while (std::scanf("%lld %lld %lld %d %d", &m, &n_out, &k, &r, &n) == 5)
    std::printf("%s\n", qlora::pool_grad_splits(qlora::pool_grad_units(n, r, k, n_out), m, n, 148) ? "split" : "whole");
  return 0;
}
