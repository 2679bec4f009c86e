/* Host check of the KV cache's K codes (test infrastructure).
 *
 * The cache's writer forms clamp(rint(fl(x / sk)), -127, 127) without a
 * division: nr = -fl(1/sk), z = fl(x nr), r = fma(z, sk, x), y = fma(r, nr, z),
 * and the code is the low byte of fl(1.5 * 2^23 - y).  It takes this path for
 * sk in [2^-100, 2^125].  For each positive finite bf16 amax in the chosen set,
 * sk = fl(amax / 127), and every bf16 x with |x| <= amax this compares the two
 * and prints "pairs N differ D".
 *
 *   k_quotient_check sample   every amax mantissa at a spread of exponents
 *   k_quotient_check all      every positive finite bf16 amax (about 1e9 pairs)
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static float bf16_value(uint32_t bits) {
    uint32_t u = bits << 16;
    float f;
    memcpy(&f, &u, sizeof f);
    return f;
}

static int in_sample(uint32_t amax_bits) {
    static const int exps[] = {34, 35, 36, 60, 100, 120, 126, 127, 128, 131, 140, 160, 200, 250, 254};
    int e = (int)(amax_bits >> 7) & 0xFF;
    for (unsigned k = 0; k < sizeof exps / sizeof exps[0]; ++k)
        if (e == exps[k]) return 1;
    return 0;
}

int main(int argc, char **argv) {
    const int all = argc > 1 && strcmp(argv[1], "all") == 0;
    long long pairs = 0, differ = 0;
#pragma omp parallel for schedule(dynamic, 16) reduction(+ : pairs, differ)
    for (uint32_t ab = 0x0001; ab < 0x7F80; ++ab) {
        if (!all && !in_sample(ab)) continue;
        const float amax = bf16_value(ab);
        const float sk = amax / 127.0f;
        if (!(sk >= 0x1p-100f && sk <= 0x1p125f)) continue;
        const float nr = -(1.0f / sk);
        for (uint32_t xb = 0; xb < 0x10000; ++xb) {
            const float x = bf16_value(xb);
            if (!(fabsf(x) <= amax)) continue;
            volatile float z = x * nr;
            volatile float r = fmaf(z, sk, x);
            volatile float y = fmaf(r, nr, z);
            volatile float t = 12582912.0f - y;
            uint32_t bits;
            float tt = t;
            memcpy(&bits, &tt, sizeof bits);
            const int got = (int8_t)(bits & 0xFF);
            const int want = (int)fminf(fmaxf(rintf(x / sk), -127.0f), 127.0f);
            ++pairs;
            if (got != want) ++differ;
        }
    }
    printf("pairs %lld differ %lld\n", pairs, differ);
    return differ != 0;
}
