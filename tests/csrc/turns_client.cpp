// Prints the rotation's frequencies (argv: "F" R scale theta), or how many tables a
// row of calls makes (argv: "N", then R scale theta of each call).
#include <stdio.h>
#include <stdlib.h>

#include "pod_turns.h"

int main(int argc, char** argv) {
  static pod::KeptTurns kept;
  for (int i = 2; i + 2 < argc; i += 3) {
    const int R = atoi(argv[i]);
    const pod::Turns& t = kept.of(R, strtof(argv[i + 1], nullptr), strtof(argv[i + 2], nullptr));
    if (argv[1][0] == 'F')
      for (int j = 0; j < R / 2; ++j) printf("%llu\n", (unsigned long long)t.f[j]);
  }
  if (argv[1][0] == 'N') printf("%u\n", kept.made());
  return 0;
}
