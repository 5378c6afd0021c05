"""CTAs that an SM can hold together must fit its tensor memory together: an
allocation that has to wait holds up a cluster, and two clusters that wait for
each other's columns never end.  The host's sizes, compiled here without a GPU,
against an SM's 228 KB of shared memory and 512 columns."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_63_b200", "csrc")
SM, RESERVE, COLUMNS = 228 * 1024, 1024, 512

PROGRAM = r"""
#include <cstdio>
#include "dense_few_plan.h"
using namespace moe;
int main() {
  for (int cols = 32; cols <= 512; cols *= 2)
    for (size_t smem = 0; smem <= 220 * 1024; smem += 1000)
      std::printf("share %d %zu %zu\n", cols, smem, tmem_smem(smem, cols));
  const int64_t Ks[] = {1, 64, 200, 1411, 4096, 14336, 16384};
  const int Ns[] = {1, 130, 1000, 4096, 14336, 140000};
  for (int form = 0; form < 3; ++form)                       // one plane, two planes, gated
    for (int64_t M = 1; M <= (form == 1 ? 64 : 128); ++M)
      for (int64_t K : Ks)
        for (int N : Ns)
          for (int64_t sms : {148, 40}) {
            const FewPlan p = few_plan(M, K, N, form == 2, form == 1 ? 2 : 1,
                                       [&](int split, int per_sm) { return sms * per_sm / split * split; });
            const int nw = form == 2 ? 2 : 1, planes = form == 1 ? 2 : 1;
            const size_t used = 1024 + std::max((size_t)p.stages * (nw * kFewWBytes + (size_t)planes * p.tt * 128),
                                                (size_t)nw * p.tt * kFewBN * 4);
            std::printf("plan %d %lld %d %d %d %d %zu %zu\n", form, (long long)M, p.tt * nw * planes, p.tmem_cols,
                        p.stages, p.split, p.smem, used);
          }
}
"""


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("tmem")
    src, exe = d / "sizes.cpp", d / "sizes"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    rows = [ln.split() for ln in out]
    return ([tuple(map(int, r[1:])) for r in rows if r[0] == "share"],
            [tuple(map(int, r[1:])) for r in rows if r[0] == "plan"])


def least(sizes):
    """The least shared memory that a CTA with so many columns asks for."""
    out = {}
    for cols, _, got in sizes[0]:
        out[cols] = min(out.get(cols, got), got)
    return out


def test_a_kernel_gets_what_it_asked_for(sizes):
    assert all(got >= smem for _, smem, got in sizes[0])


def most_columns(smem):
    """Over any set of CTAs that an SM's shared memory holds (smem: columns ->
    dynamic bytes of a CTA), by dynamic programming in pieces of 64 bytes."""
    unit = 64
    need = {c: (s + RESERVE) // unit for c, s in smem.items()}
    most = [0] * (SM // unit + 1)
    for room in range(1, len(most)):
        most[room] = max([most[room - 1]] + [most[room - n] + c for c, n in need.items() if n <= room])
    return most[-1]


def test_ctas_that_fit_shared_memory_fit_tensor_memory(sizes):
    assert set(least(sizes)) == {32, 64, 128, 256, 512}
    assert most_columns(least(sizes)) <= COLUMNS


@pytest.mark.parametrize("smem", [{256: 87040, 128: 54272}, {256: 87040, 32: 37888}, {512: 120 * 1024, 32: 37888},
                                  {512: 120 * 1024, 256: 87040}])
def test_sizes_of_the_buffers_alone_do_not(smem):
    """Two gated CTAs of 80 rows and one of a linear layer; a router CTA of 120
    KB and a decoding one: they fit the shared memory, not the columns."""
    assert most_columns(smem) > COLUMNS


def test_few_row_plans(sizes):
    """Every plan has its columns' share, whole stages, and what it uses."""
    low = least(sizes)
    for form, M, used_cols, cols, stages, split, smem, used in sizes[1]:
        what = (form, M, stages, split)
        assert cols >= used_cols and cols in low and smem >= low[cols], what
        assert stages >= 2 and split in (1, 2, 4, 8) and used <= smem <= 220 * 1024, what


def test_every_allocation_takes_its_share():
    """Each kernel that allocates tensor memory sizes its launch by the rule."""
    found = set()
    for f in os.listdir(CSRC):
        text = open(os.path.join(CSRC, f)).read()
        if "tcgen05.alloc" in text:
            found.add(f)
            assert "tmem_smem(" in text or "kAllTmemSmem" in text or "few_plan(" in text, f
    assert found
