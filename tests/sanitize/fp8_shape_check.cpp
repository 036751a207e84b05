// fp8_shape_check.cpp -- prints the form that a grouped product of e4m3 rows
// takes (csrc/fp8_shape.h), for "E N rows" lines on standard input; built with
// AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdio>

#include "fp8_shape.h"

int main()
{
    const char* const names[] = {"rows", "rows32", "32x64", "64x128", "128x128", "256x256"};
    int E, N, rows;
    while (std::scanf("%d %d %d", &E, &N, &rows) == 3) std::puts(names[(int)qmoe::fp8_tile(E, N, rows)]);
    return 0;
}
