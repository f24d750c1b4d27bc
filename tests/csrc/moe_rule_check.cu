// The choice between the kernels of the experts' products (csrc/lk_moe.cuh), on the
// host: of each line "E k H F M mode op ..." of the input, 1 for the tensor-core kernel.
#include <cstdio>
#include <cstring>

#include "lk_moe.cuh"

int main() {
  int E, k, H, F, M;
  char mode[16], op[16];
  double single, rows;
  while (scanf("%d %d %d %d %d %15s %15s %lf %lf", &E, &k, &H, &F, &M, mode, op, &single, &rows) == 9) {
    const bool glu = !strcmp(op, "glu");
    printf("%d\n", lkmoe::rows_favoured(E, glu ? F : H, glu ? H : F, k, M, strcmp(mode, "int8act") ? 2 : 1, glu, 152));
  }
}
