"""How cross attention cuts its units: the host's rules give the choices that stand starred beside their measurements
(152 SMs; fa2_cross_schedule.h is plain C++, compiled here by itself)."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_03_gb300", "csrc")
PROGRAM = r"""
#include "fa2_cross_schedule.h"
#include <cstdio>
#include <cstdlib>
int main(int, char** argv) {
  const bool bwd = argv[1][0] == 'b';
  const int D = std::atoi(argv[2]);
  const long long heads = std::atoll(argv[3]), rows = std::atoll(argv[4]), keys = std::atoll(argv[5]);
  const bool lengths = std::atoi(argv[6]) != 0;
  const int sms = std::atoi(argv[7]);
  const long long nkv = (keys + 127) / 128;
  int ctas;
  if (bwd) {
    const long long step = D <= 64 ? 128 : 64;
    ctas = fa2::cross_bwd_share_ctas(D, heads * nkv, (rows + step - 1) / step, lengths, heads * rows * D * 8, sms);
  } else {
    ctas = fa2::cross_share_ctas(D, fa2::split_keys(D, rows, nkv), heads * ((rows + 255) / 256), nkv, lengths, sms);
  }
  std::printf("%d\n", ctas);
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++")
    assert cxx, "a host compiler is needed to build the library anyway"
    d = tmp_path_factory.mktemp("schedule")
    (d / "main.cc").write_text(PROGRAM)
    exe = str(d / "main")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(d / "main.cc"), "-o", exe], check=True)

    def run(kind, D, heads, rows, keys, lengths=False, sms=152):
        args = [str(int(x) if isinstance(x, bool) else x) for x in (kind, D, heads, rows, keys, lengths, sms)]
        return int(subprocess.run([exe] + args, check=True, capture_output=True, text=True).stdout)

    return run


@pytest.mark.parametrize("D,heads,rows,keys,parts", [
    (64, 8, 128, 500, 1), (64, 8, 128, 1000, 1), (64, 8, 128, 1508, 3), (64, 8, 128, 2000, 4), (64, 8, 128, 4068, 4),
    (64, 8, 128, 16356, 10), (64, 32, 128, 16356, 4),
    (128, 8, 128, 500, 1), (128, 8, 128, 1000, 1), (128, 8, 128, 1508, 1), (128, 8, 128, 2000, 4), (128, 8, 128, 4068, 4),
    (128, 8, 128, 16356, 10),
])
def test_forward_parts(choose, D, heads, rows, keys, parts):
    assert choose("forward", D, heads, rows, keys) == (0 if parts == 1 else parts * heads)


def test_forward_over_counts_on_the_device(choose):
    assert choose("forward", 64, 96, 256, 4096, lengths=True) == 152
    # at least one unit per SM: by the most tiles a unit can have
    assert choose("forward", 64, 192, 256, 512, lengths=True) == 0 and choose("forward", 64, 192, 256, 768, lengths=True) == 152
    assert choose("forward", 128, 192, 128, 1024, lengths=True) == 0 and choose("forward", 128, 192, 128, 1536, lengths=True) == 152


@pytest.mark.parametrize("D,rows,parts", [(64, 256, 1), (64, 1024, 4), (64, 4096, 8), (64, 16384, 16),
                                          (128, 256, 1), (128, 1024, 4), (128, 4096, 8), (128, 16384, 16)])
def test_backward_parts(choose, D, rows, parts):
    assert choose("backward", D, 8, rows, 77) == (0 if parts == 1 else parts * 8)


def test_the_starred_choices_are_all_here(choose):
    # every star in the comments has a row above
    text = re.sub(r"\n//\s*", " ", open(os.path.join(CSRC, "fa2_cross_schedule.h")).read())
    assert len(re.findall(r"\d\* ", text)) == 13 + 8
    assert len(re.findall(r"all SMs\* ", text)) == 1


@pytest.mark.parametrize("sms", [1, 2, 7, 148, 152, 160])
def test_a_choice_is_between_the_units_and_the_sms(choose, sms):
    for kind in ("forward", "backward"):
        for D in (32, 128):
            for heads, rows, keys in ((1, 1, 1), (3, 700, 5000), (8, 100000, 77), (500, 40, 300), (1, 128, 10 ** 6)):
                for lengths in (False, True):
                    assert 0 <= choose(kind, D, heads, rows, keys, lengths, sms) <= sms
