"""The keys by which sampling orders logits, and the division of a range of keys (sample_keys.cuh): the
header's own code, compiled for the host."""
import os
import shutil
import subprocess

import pytest

from expert_select_gb300 import build as B

PROGRAM = r"""
#include "sample_keys.cuh"
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
using namespace moe::sample;
static float bits(uint32_t b) { float f; memcpy(&f, &b, 4); return f; }
static void need(bool ok, const char *what) { if (!ok) { printf("%s\n", what); exit(1); } }

static void order() {
    std::mt19937 g(3);
    const uint32_t low = key_of(-INFINITY), high = key_of(INFINITY);
    need(key_of(0.f) == key_of(-0.f), "0 and -0 have one key");
    for (int i = 0; i < 400000; ++i) {
        uint32_t k = low + g() % (high - low);
        if (i < 4000) k = key_of(0.f) - 2000 + i;
        need(key_of(value_of(k)) == k, "a key's value has the key");
        need(value_of(k) < value_of(k + 1), "the next key's value is larger");
    }
    need(value_of(low) == -INFINITY && value_of(high) == INFINITY, "the ends");
    for (uint32_t b = 0; b < 0x10000; ++b) {
        const float l = bits(b << 16);
        if (!std::isnan(l)) need(key_of(l) % 0x10000 == 0, "bf16 values' keys are multiples of 2^16");
    }
}

// The search as the kernel makes it: the n-th largest of x, which the row's values are compared with as values.
template <int kStep> static void search(const std::vector<float> &x, uint64_t target, float want) {
    float top = -INFINITY, least = INFINITY;
    for (float l : x) { top = std::fmax(top, l); least = std::fmin(least, l); }
    KeyRange<kStep> keys(key_of(least), key_of(top));
    for (bool more = keys.open(); more;) {
        const int shift = keys.shift();
        std::vector<uint64_t> bins(kRangeBins);
        const float lo = value_of(keys.min), hi = value_of(keys.max);
        for (float l : x)
            if (l >= lo && l <= hi) {
                const uint32_t bin = (keys.max - key_of(l)) >> shift;
                need(bin < kRangeBins, "a value's bin lies outside");
                ++bins[bin];
            }
        int bin = 0;
        for (; bin < kRangeBins && bins[bin] < target; ++bin) target -= bins[bin];
        need(bin < kRangeBins, "no bin");
        more = keys.narrow(bin, shift);
    }
    need(value_of(keys.max) == want, "another value than the n-th largest");
}

static float rounded(float l) { uint32_t b; memcpy(&b, &l, 4); return bits(b & 0xffff0000u); }

int main() {
    order();
    std::mt19937 g(1);
    std::normal_distribution<float> normal;
    for (int trial = 0; trial < 3000; ++trial) {
        // zeros of both signs between values of either sign, down to the smallest; the largest so that a range's
        // end falls beside zero's key
        const uint32_t n = (1u << trial % 23) * (1 + g() % 8) - 1;
        std::vector<float> x{bits(n)};
        const int kind = trial / 23 % 5;
        for (int i = 1; i < 400; ++i)
            x.push_back(i < 120 ? bits(i & 1 ? 0 : 0x80000000u)
                        : kind == 0 ? bits(0x80000000u | g() % 0x400000u)
                        : kind == 1 ? bits((g() & 0x80000000u) | g() % 64)
                        : kind == 2 ? normal(g) * 1e-38f
                        : kind == 3 ? normal(g) : bits(0x80000000u | g() % (n + 1)));
        for (int step = 0; step < 2; ++step) {
            std::vector<float> y(x);
            if (step) for (float &l : y) l = rounded(l);
            std::vector<float> s(y);
            std::sort(s.begin(), s.end(), [](float a, float b) { return a > b; });
            for (int q = 0; q < 6; ++q) {
                const int at = g() % s.size();
                if (step) search<16>(y, at + 1, s[at]); else search<0>(y, at + 1, s[at]);
            }
        }
    }
    printf("fine\n");
}
"""


def test_keys_and_ranges(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs a host compiler")
    src, exe = tmp_path / "keys.cpp", tmp_path / "keys"
    src.write_text("#include <algorithm>\n" + PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", B.CSRC, "-x", "c++", str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "fine\n", r.stdout


def test_the_kernels_use_these_keys():
    with open(os.path.join(B.CSRC, "sample.cu")) as f:
        text = f.read()
    assert "uint32_t key_of(" not in text and "KeyRange<kStep>" in text
