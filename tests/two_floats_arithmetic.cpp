// The losses' arithmetic in two floats (two_floats.cuh), run on the host and measured against doubles.  Built without
// contraction, as the header writes its fused operations out.  Prints a line "name value" for each figure.
#include "../speculative_decoding_verification_14_gb300/csrc/two_floats.cuh"

#include <algorithm>
#include <cstdio>
#include <random>

using namespace sv;

static double value(Two x) { return (double)x.h + (double)x.l; }
static Two of(double x) { return Two{(float)x, (float)(x - (double)(float)x)}; }

int main() {
    std::mt19937_64 g(1);
    std::uniform_real_distribution<double> u(0, 1);
    double exp_off = 0, log_off = 0, sum_off = 0, product_off = 0, quotient_off = 0;
    for (int i = 0; i < 4000000; ++i) {
        const Two x = of(i % 5 ? -u(g) * (i & 1 ? 80 : 2) : 80 * u(g));
        exp_off = std::max(exp_off, std::fabs(value(two_exp(x)) / std::exp(value(x)) - 1));
        const Two y = of(std::exp((u(g) - 0.5) * (i & 1 ? 160 : 1)));
        log_off = std::max(log_off, std::fabs(value(two_log(y)) - std::log(value(y))));
        const Two a = of((u(g) - 0.5) * 100), b = of((u(g) + 1e-3) * 10);
        sum_off = std::max(sum_off, std::fabs(value(two_add(a, b)) - (value(a) + value(b))) /
                                        (std::fabs(value(a)) + std::fabs(value(b))));
        product_off = std::max(product_off, std::fabs(value(two_mul(a, b)) / (value(a) * value(b)) - 1));
        quotient_off = std::max(quotient_off, std::fabs(value(two_div(a, b)) / (value(a) / value(b)) - 1));
    }
    const float inf = INFINITY;
    const bool ends = two_exp(Two{-inf, NAN}).h == 0 && two_exp(Two{-90, 0}).h == 0 && two_exp(Two{89, 0}).h == inf &&
                      two_exp(Two{0, 0}).h == 1 && two_log(Two{1, 0}).h == 0 && two_mul(Two{-3e38f, 1e30f}, Two{2, 0}).h == -inf &&
                      two_mul(Two{-3e38f, 1e30f}, Two{2, 0}).l == 0;
    std::printf("exp_off %.17g\nlog_off %.17g\nsum_off %.17g\nproduct_off %.17g\nquotient_off %.17g\nends %d\n", exp_off, log_off,
                sum_off, product_off, quotient_off, (int)ends);
}
