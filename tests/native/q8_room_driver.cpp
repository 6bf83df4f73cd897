// Command-line driver of csrc/q8_plan.h's room in an SM, one command per line:
//   room <bytes of an SM> <reserved a CTA> <bytes of a CTA>  -> CTAs
//   step <sms> <per SM> <Hkv> <most> <n> <work>*n            -> the largest number of splits, then each
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "q8_plan.h"

int main() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string cmd;
        in >> cmd;
        if (cmd == "room") {
            size_t sm, reserved, cta;
            in >> sm >> reserved >> cta;
            std::cout << qa::q8_ctas_per_sm(sm, reserved, cta) << "\n";
            continue;
        }
        int sms, per_sm, hkv, most, n;
        in >> sms >> per_sm >> hkv >> most >> n;
        std::vector<int> work(n), splits(n);
        for (int &w : work) in >> w;
        std::cout << qa::q8_plan_step(sms, hkv, most, n, work.data(), splits.data(), per_sm);
        for (int s : splits) std::cout << " " << s;
        std::cout << "\n";
    }
}
