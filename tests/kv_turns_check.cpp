// Prints the two doubles that kv_plan.h's kv_turns makes of each argument, as
// hexadecimal.
#include <stdio.h>
#include <stdlib.h>

#include "kv_plan.h"

int main(int n, char** v) {
    for (int i = 1; i < n; ++i) {
        double hi, lo;
        dq::kv_turns(strtod(v[i], nullptr), &hi, &lo);
        printf("%a %a\n", hi, lo);
    }
    return 0;
}
