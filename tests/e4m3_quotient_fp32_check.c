/* Check behind the blockwise codes of the norm (fp32 values, any scale).
 *
 * A code is E4M3(RN(v / s)), all in fp32. The kernel forms the quotient by
 * Markstein's correction of the product with the rounded reciprocal (P.
 * Markstein, IBM J. Res. Dev. 34(1), 1990), r = RN(1 / s):
 *     y0 = RN(v r),  e = RN(v - s y0),  y1 = RN(y0 + r e).
 * y0 is within two steps of v / s, so e is a multiple of step(s) step(y0) of at
 * most 25 bits and e, r and their product each add at most 2^-24 of it: before
 * its last rounding y1 is within 2^-22 of a step of v / s. It can therefore
 * differ from RN(v / s) only that close to the middle of two neighbouring fp32
 * numbers, and the codes only where one of the two is a tie of two E4M3 codes.
 * All this needs e to be exact down to step(s) step(y0) >= 2^-149: for quotients
 * from 2^-11 on (smaller ones have code 0), s >= 2^-92.
 *
 * In integers, v = V 2^a and s = S 2^b of 24 bits each and N the number of half
 * steps next to the tie: V 2^j - S N = d with |d| <= 8. N is odd, so each d has
 * one S modulo 2^j. The program walks every tie (odd multiples 1 ... 31 of a
 * power of two), both sides, j and 0 < |d| <= 64, and compares the codes at the
 * binades of the quotient and of the scale from 2^LOW to 2^99. Prints the counts;
 * exits 1 on a difference. The argument is LOW (default -92).
 * Build with -ffp-contract=off. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

/* Nearest E4M3 value of y >= 0 (ties to the even mantissa), saturating at 448. */
static float e4m3_value(float y)
{
    if (y >= 448.0f) return 448.0f;
    if (y < 0x1p-6f) return nearbyintf(y * 512.0f) / 512.0f; /* subnormal step 2^-9 */
    uint32_t b;
    memcpy(&b, &y, 4);
    b = (b + 0x7FFFFu + ((b >> 20) & 1u)) & ~0xFFFFFu;      /* keep 3 mantissa bits */
    float r;
    memcpy(&r, &b, 4);
    return r;
}

/* Inverse of an odd number modulo 2^64 (Newton's iteration doubles the bits). */
static uint64_t inverse(uint64_t a)
{
    uint64_t x = a;
    for (int i = 0; i < 6; ++i) x *= 2 - a * x;
    return x;
}

static long long pairs, diff;

static void compare(uint32_t S, uint32_t V, int low)
{
    for (int b = low; b < 100; ++b) {
        const float s = ldexpf((float)S, b - 23), r = 1.0f / s;
        for (int q = -12; q <= 9; ++q) {
            const float v = ldexpf((float)V, b - 23 + q);
            if (v > 450.0f * s) break;
            const float y0 = v * r;
            const float y1 = fmaf(fmaf(-s, y0, v), r, y0);
            const float want = v / s;
            ++pairs;
            if (e4m3_value(y1) != e4m3_value(want)) {
                if (diff < 5) printf("difference: s=%a v=%a y1=%a v/s=%a\n", s, v, y1, want);
                ++diff;
            }
        }
    }
}

int main(int argc, char** argv)
{
    const int low = argc > 1 ? atoi(argv[1]) : -92;
    long long found = 0;
    for (uint64_t odd = 1; odd < 32; odd += 2) {
        uint64_t tie = odd;
        while (tie < (1u << 23)) tie <<= 1;              /* 24 bits */
        /* half steps above and below; below a power of two the steps are half as wide */
        const uint64_t beside[3] = {2 * tie + 1, 2 * tie - 1, 4 * tie - 1};
        for (int k = 0; k < (odd == 1 ? 3 : 2); ++k) {
            const uint64_t N = beside[k], inv = inverse(N);
            for (int j = 23; j <= 26; ++j) {
                const uint64_t mask = (1ull << j) - 1;
                for (int64_t d = -64; d <= 64; ++d) {
                    if (d == 0) continue;
                    for (uint64_t S = ((uint64_t)-d * inv) & mask; S < (1u << 24); S += mask + 1) {
                        if (S < (1u << 23)) continue;
                        const uint64_t V = (S * N + (uint64_t)d) >> j;   /* S N is below 2^50 */
                        if (V < (1u << 23) || V >= (1u << 24)) continue;
                        ++found;
                        compare((uint32_t)S, (uint32_t)V, low);
                    }
                }
            }
        }
    }
    printf("significands %lld, pairs %lld, E4M3 differences %lld\n", found, pairs, diff);
    return diff || !found;
}
