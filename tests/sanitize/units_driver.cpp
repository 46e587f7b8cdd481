// Host driver for the row sampler's constants (sample_units.hpp): they are the
// nearest whole numbers, also on a thread whose processor flushes subnormals.
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include <xmmintrin.h>

#include "../../top_search_resident_amd/csrc/sample_units.hpp"

static int bad = 0;
static void expect(uint64_t got, uint64_t want, const char *what, int shift) {
    if (got != want) {
        fprintf(stderr, "FAIL: %s at shift %d: got %llu want %llu\n", what, shift, (unsigned long long)got,
                (unsigned long long)want);
        bad = 1;
    }
}

// The whole number nearest to c 2^shift (0 < c < 1), from c's bits alone.
static uint64_t nearest(double c, int shift) {
    uint64_t bits;
    memcpy(&bits, &c, sizeof bits);
    const uint64_t mantissa = (bits & ((uint64_t(1) << 52) - 1)) | (uint64_t(1) << 52);
    const int down = 1075 - int(bits >> 52) - shift;  // c = mantissa 2^(exponent - 1075)
    return (mantissa + (uint64_t(1) << (down - 1))) >> down;
}

static void check_all() {
    for (volatile int s = 31; s <= 46; s = s + 1) {
        const int shift = s;
        const rt::SampleUnits u = rt::sample_units(shift);
        expect(u.c4, nearest(rt::kC4, shift), "c4", shift);
        expect(u.c3, nearest(rt::kC3, shift), "c3", shift);
        expect(u.c2, nearest(rt::kC2, shift), "c2", shift);
        expect(u.c1, nearest(rt::kC1, shift), "c1", shift);
        expect(u.one, uint64_t(1) << shift, "one", shift);
    }
    const struct {
        int64_t v;
        int shift;
    } rows[] = {{1, 46}, {2, 46}, {65536, 46}, {65537, 45}, {131072, 45}, {131073, 44}, {2147483647, 31}};
    for (const auto &row : rows) expect(uint64_t(rt::sample_shift(row.v)), uint64_t(row.shift), "shift", row.shift);
}

int main() {
    check_all();
    _mm_setcsr(_mm_getcsr() | 0x8040u);  // flush to zero, denormals are zero
    volatile double least = 2.2250738585072014e-308;
    if (least * 0.5 != 0.0) bad = 1, fprintf(stderr, "FAIL: the mode is not on\n");
    check_all();
    if (!bad) printf("ok\n");
    return bad;
}
