// Command-line driver of the shares rule of csrc/q4_plan.h for the CPU tests: per
// line "<Hq> <Hkv> <D> <T> <sms>" -> shares of a token, warps of a CTA, bytes of
// shared memory that they take, the most there is.
#include <iostream>

#include "q4_plan.h"

int main() {
    int Hq, Hkv, D, sms;
    long long T;
    while (std::cin >> Hq >> Hkv >> D >> T >> sms) {
        const int parts = qa::q4_row_parts(Hq, Hkv, D, T, sms);
        std::cout << parts << " " << qa::kQ4RowWarps << " "
                  << (parts > 0 ? qa::q4_prefill_rows_smem(Hq, Hkv, D, parts) : 0) << " " << qa::kQ4RowSmemMost << "\n";
    }
    return 0;
}
