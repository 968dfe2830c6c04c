"""Outputs of the q/k norm that share elements with another tensor: the host's test
against an enumeration of the elements, and the refusals of the call."""
import os
import random
import subprocess

import pytest

from conftest import ROOT
from test_serving_ops_abi import ARG, lib, norm, view  # noqa: F401 (lib: fixture)

CSRC = os.path.join(ROOT, "recurrence_augmented_dilated_chunked_b200", "csrc")
MAIN = r"""
#include <cstdio>
#include "overlap.h"
int main() {
  long long a[4], b[4];
  int B, T, Dh, ha, hb;
  while (scanf("%d %d %d %lld %lld %lld %lld %d %lld %lld %lld %lld %d", &B, &T, &Dh, a, a + 1, a + 2, a + 3, &ha, b, b + 1,
               b + 2, b + 3, &hb) == 13) {
    const ratp_view x = {(void*)a[0], a[1], a[2], a[3], ha}, y = {(void*)b[0], b[1], b[2], b[3], hb};
    printf("%d\n", (int)ratp::views_overlap(x, y, 2, B, T, Dh));
  }
}
"""


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    (d / "main.cpp").write_text(MAIN)
    exe = str(d / "main")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(d / "main.cpp"),
                           "-o", exe])

    def run(cases):
        text = "\n".join(" ".join(str(x) for x in c) for c in cases)
        return [int(x) for x in subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()]

    return run


def elements(data, sb, st, sh, heads, B, T, Dh):
    """The 8-element pieces of a view (all its numbers are multiples of 8)."""
    return {data // 2 + b * sb + t * st + h * sh + c for b in range(B) for t in range(T) for h in range(heads)
            for c in range(0, Dh, 8)}


def test_against_an_enumeration(answers):
    r = random.Random(5)
    cases, want = [], []
    for _ in range(4000):
        B, T, Dh = r.randint(1, 3), r.randint(1, 4), r.choice([8, 16])
        vs = []
        for _ in range(2):
            heads = r.randint(1, 3)
            s = [8 * r.randint(0, 11) for _ in range(3)]
            if r.random() < 0.5:
                s[2] = Dh * r.randint(1, 2)
                s[1] = s[2] * heads * r.randint(1, 3)
                s[0] = s[1] * T
            vs.append([16 * r.randint(1, 30)] + s + [heads])
        if r.random() < 0.5:
            vs[1][1:3] = vs[0][1:3]
        cases.append([B, T, Dh] + vs[0] + vs[1])
        want.append(int(bool(elements(*vs[0], B, T, Dh) & elements(*vs[1], B, T, Dh))))
    assert answers(cases) == want
    assert 1000 < sum(want) < 3000


def test_layouts_of_real_use(answers):
    B, T, H, Dh = 4, 8192, 32, 128
    row, at = Dh * H, 1 << 20
    fused = lambda i: [at + 2 * i * row, 3 * row * T, 3 * row, Dh, H]
    flat = [at, row * T, row, Dh, H]
    head_major = [at + 2 * B * T * row, row * T, Dh, Dh * T, H]
    pairs = lambda i: [at + 2 * i * Dh, 2 * row * T, 2 * row, 2 * Dh, H]      # [B, T, H, 2, Dh]
    cases = [(fused(0), fused(1), 0), (fused(0), fused(2), 0), (flat, head_major, 0), (pairs(0), pairs(1), 0),
             (flat, [at + 2 * B * T * row] + flat[1:], 0), (flat, [at + 2 * row] + flat[1:], 1), (fused(0), fused(0), 1),
             (flat, [at] + head_major[1:], 1), ([at, 0, row, Dh, H], flat, 1),
             ([at, 2 * row * T, 2 * row, Dh, H], [at + 2 * row, 2 * row * T, 2 * row, Dh, 8], 0)]   # every second token
    assert answers([[B, T, Dh] + a + b for a, b, _ in cases]) == [w for _, _, w in cases]


def test_refusals(lib):  # noqa: F811
    q, far, k = view(), view(data=1 << 20), view(data=1 << 21)
    assert norm(lib, q=q, k=k, qo=k, ko=far) == ARG                          # onto the other input
    assert norm(lib, q=q, k=k, qo=far, ko=far) == ARG                        # both into one tensor
    assert norm(lib, q=q, k=k, qo=view(data=4096 + 1024), ko=far) == ARG     # its input a token on
    assert norm(lib, q=q, k=k, qo=view(sh=256), ko=far) == ARG               # its input in another order
    assert norm(lib, q=q, k=k, qo=far, ko=view(data=4096 + 256)) == ARG
