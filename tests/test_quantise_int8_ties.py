"""Why 127 x / m is rounded to the nearest integer exactly for bf16 x: how near it comes to a half integer, in integers, and
the f32 quotient by a rounded reciprocal and one fused correction for every x below every m, on the CPU."""
import subprocess

import numpy as np

X, M = np.arange(128, 256, dtype=np.int64)[:, None], np.arange(128, 256, dtype=np.int64)[None, :]


def distances(d):
    """127 X / (M 2^d) is a half integer, or n / (M 2^(d+1)) away from the nearest: the n, for X 2^-d <= M."""
    unit = M << d
    rest = (254 * X) % (2 * unit)                    # of 254 X = h unit, h odd
    n = np.abs(rest - unit)
    return np.where(X <= unit, n, -1)


def test_distance_from_half_integers():
    for d in range(12):
        n, unit = distances(d), M << d
        some = n > 0
        # relative to the quotient 254 X / (2 unit) itself
        rel = (n / (254.0 * X))[some]
        assert rel.min() >= 1 / (254 * 255) > 2.0 ** -16
    assert (distances(0) == 0).any() and (distances(1) == 0).any()                 # half integers occur
    # the distance itself gets small with the quotient: X = 255, M = 253, d = 8 is 1 / 64768 below a half
    n = distances(8)[255 - 128, 253 - 128]
    assert n == 2 and n / (2 * 253 * 2 ** 8) == 1 / 64768


PROGRAM = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
static float value(uint32_t b) { float x; memcpy(&x, &b, 4); return x; }
static uint32_t bits(float x) { uint32_t b; memcpy(&b, &x, 4); return b; }
int main(void) {
    const uint32_t exponents[] = {7, 8, 20, 127, 200, 254};
    long wrong = 0, all = 0;
    for (uint32_t mantissa = 0; mantissa < 128; ++mantissa)
        for (int i = 0; i < 6; ++i) {
            const float top = fmaxf(value(exponents[i] << 23 | mantissa << 16), 127.0f * 0x1p-126f);
            const float p = value(uint32_t(128 - int(bits(top) >> 23) + 127) << 23);
            const float by = 127.0f * p, m = top * p, r = 1.0f / m;
            for (uint32_t b = 0; b < 0x7F80; ++b) {
                const float x = value(b << 16);
                if (x > top) break;
                const double q = double(x) * 127.0 / double(top);      /* 2^-52 of itself off */
                const float y = x * by, t = y * r;
                const float sum = fmaf(fmaf(-t, m, y), r, t) + 0x1.8p23f;
                wrong += int8_t(bits(sum) & 255) != int(nearbyint(q));
                ++all;
            }
        }
    printf("%ld of %ld\n", wrong, all);
    return wrong != 0;
}
"""


def test_quotient(tmp_path):
    source, program = tmp_path / "quotient.cpp", tmp_path / "quotient"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-o", str(program), str(source)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("0 of "), r.stdout
    assert int(r.stdout.split()[2]) > 10_000_000
