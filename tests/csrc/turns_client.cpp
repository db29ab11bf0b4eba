// Prints the rotation's frequencies (argv: "F" R scale theta).
#include <stdio.h>
#include <stdlib.h>

#include "pod_turns.h"

int main(int argc, char** argv) {
  if (argc != 5) return 1;
  const int R = atoi(argv[2]);
  pod::Turns t;
  pod::make_turns(R, strtof(argv[3], nullptr), strtof(argv[4], nullptr), &t);
  for (int j = 0; j < R / 2; ++j) printf("%llu\n", (unsigned long long)t.f[j]);
  return 0;
}
