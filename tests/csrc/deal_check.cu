// The deal of key units to blocks (csrc/lk_attn.cuh), on the host: every number
// of units that the calls accept, up to 2^31 - 1, is dealt whole, in order, to
// the n holders, and holder() finds each share's ends.  Prints the faults.
#include <cstdio>

#include "lk_attn.cuh"

using lkattn::deal_blocks;
using lkattn::Shares;

static long faults;

static void check(long T, int W, int least, bool one, int items) {
  const Shares s = deal_blocks((int)T, W, least, one, items);
  bool ok = s.n >= 1 && s.n <= W && s.k >= 1 && s.base >= 1;
  long at = 0;
  for (int c = 0; c < W && ok; ++c) {
    if (c >= s.n) break;  // what a block does
    const long b = s.begin(c), n = s.size(c);
    ok = b == at && n >= 1 && b + n <= T && s.holder((int)b) == c && s.holder((int)(b + n - 1)) == c;
    at = b + n;
  }
  if (!ok || at != T) {
    if (!faults++) printf("T %ld W %d least %d one %d items %d: n %d k %d, %ld dealt\n", T, W, least, one, items, s.n, s.k, at);
  }
}

int main() {
  const long most = 0x7fffffffL;
  const int widths[] = {1, 2, 148, 152, 192}, leasts[] = {1, 7, 12};
  for (int W : widths)
    for (int least : leasts) {
      for (long T : {1L, 2L, 11L, 12L, 13L, 150L, 151L, 5000L, 1L << 30, (1L << 30) + 1, most - 12, most - 1, most})
        check(T, W, least, false, 1);
      for (int items = 1; items <= W + 3; ++items)
        for (long G : {1L, 2L, 6L, 7L, 8L, 13L, 1000L, (1L << 30) / items, (1L << 30) / items + 1, most / items - 1, most / items})
          if (G > 0 && G * items <= most) check(G * items, W, least, true, items);
    }
  printf("%ld faults\n", faults);
  return faults != 0;
}
