// turns_check.cpp -- runs the library's rounding of frequencies to fractions of a turn
// (csrc/sp_turns.h) on the CPU.  Test infrastructure only: built by tests/test_turns.py.
// Input: frequencies, one a line (as C hexadecimal floats); output: their fractions.
#include <cstdio>
#include <cstdlib>

#include "sp_turns.h"

int main() {
    char line[128];
    while (std::fgets(line, sizeof line, stdin)) std::printf("%llu\n", (unsigned long long)sp::turn_of(std::strtod(line, nullptr)));
}
