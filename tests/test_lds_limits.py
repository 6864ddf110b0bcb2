"""LDS that a launch reserves to limit its blocks per CU: with the kernel's own it stays within what a
block may have, and two blocks fit a CU.  Host arithmetic, compiled with g++; adamw.hip and
fused_adamw.hip assert theirs where they are compiled."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_sharded_mixed_amd", "csrc")
PROG = r'''
#include "zs_grid.h"
using namespace zs;
constexpr bool fits(unsigned own) {
    const int64_t all = int64_t(own) + two_blocks_lds(own);
    return all <= kBlockLdsMax && 2 * all <= kLdsPerCu && 3 * all > kLdsPerCu;
}
static_assert(fits(0) && fits(16) && fits(8208) && fits(24592) && fits(kTwoBlocksLds), "two blocks per CU");
static_assert(two_blocks_lds(kBlockLdsMax) == 0, "nothing is left to reserve");
static_assert(kBlockLdsMax == 64 * 1024, "the limit of a launch without an attribute");
int main() {}
'''


def test_a_reservation_counts_the_kernel_s_own_lds(tmp_path):
    subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-I", CSRC, "-x", "c++", "-"], input=PROG, text=True,
                   check=True)


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".hip")))
def test_a_kernel_with_lds_of_its_own_does_not_reserve_the_whole(name):
    text = open(os.path.join(CSRC, name)).read()
    assert "__shared__" not in text or "kTwoBlocksLds" not in text, name
