// Host program over the attention kernel's own cut of its work (kv_attention.cuh): reads lines "parts jobs cost ...", one
// cost per sequence in units (each with `jobs` jobs), and prints for each line "total n J M", then the parts' starts and then
// "part sequence job first last begun done" for every piece, found as the kernel's loop finds them.
#include <stdio.h>

#include <vector>

#include "../../nvfp4_block_scaled_11_b200/csrc/kv_attention.cuh"

using namespace nvfp4;

int main() {
  int most, jobs, count;
  while (scanf("%d %d %d", &most, &jobs, &count) == 3) {
    std::vector<int> cost(count);
    int64_t total = 0;
    for (int& c : cost) {
      if (scanf("%d", &c) != 1) return 1;
      total += (int64_t)c * jobs;
    }
    const KaParts parts(total, most);
    printf("%lld %d %d %d\n", (long long)total, parts.n, kKaJobUnits, kKaMinUnits);
    for (int c = 0; c <= parts.n; ++c) printf("%lld ", (long long)parts.start(c));
    printf("\n");
    for (int64_t u = 0; u < total; ++u) printf("%d ", parts.of(u));
    printf("\n");
    for (int c = 0; c < parts.n; ++c) {
      int64_t u = parts.start(c), seq_start = 0;
      const int64_t u_end = parts.start(c + 1);
      int b = 0;
      while (u - seq_start >= (int64_t)cost[b] * jobs) seq_start += (int64_t)cost[b++] * jobs;
      while (u < u_end) {
        if (u - seq_start >= (int64_t)cost[b] * jobs) seq_start += (int64_t)cost[b++] * jobs;
        const KaPiece piece(u, u_end, seq_start, cost[b]);
        if (!piece.mine) break;
        printf("%d %d %d %d %d %d %d\n", c, b, piece.job, piece.first, piece.last, piece.begun(), piece.done());
        u = piece.next;
      }
    }
    printf("end\n");
  }
  return 0;
}
