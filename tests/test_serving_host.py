"""Host-side checks of the serving operators' arithmetic and of refusals at the largest sizes (no GPU)."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import test_serving_abi as abi
from test_serving_abi import lib  # noqa: F401  (a fixture)
from transformer_decode_step_weight_gb300 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "transformer_decode_step_weight_gb300", "csrc")

def _run(tmp_path, source):
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()

def test_pages_wanted_by_the_largest_extensions(tmp_path):
    # the plan's own arithmetic: needs of every sequence, summed as the planning kernel sums them
    cases = [(2048, 1 << 20, 0, 1, 0), (2048, 1 << 30, 0, 1, 0), (1, 1 << 30, 0, 1, 0), (2, 1 << 30, 0, 1, 0),
             (2048, (1 << 30) - 7, 7, 16, 1), (2048, 5, 3, 16, 1), (2048, 0, 3, 16, 0), (3, 33, 16, 16, 0)]
    lines = "".join(f"  one({n}, {new}, {length}, {ps}, {copy});\n" for n, new, length, ps, copy in cases)
    got = [int(x) for x in _run(tmp_path, f"""#include <stdio.h>
#include "page_plan.h"
using namespace qd;
static void one(int seqs, int n_new, int len, int ps, bool copy) {{
  PageSum sum = 0;
  for (int s = 0; s < seqs; ++s) {{
    const PageNeed x = page_need(len, n_new, ps, copy);
    if (x.copy() != copy) sum -= 1;
    sum += x.pages();
  }}
  printf("%lld\\n", (long long)sum);
}}
int main() {{
{lines}  return 0;
}}
""")]
    want = [n * (-(-(length + new) // ps) - -(-length // ps) + copy) for n, new, length, ps, copy in cases]
    assert got == want and max(want) == 2 ** 41


@pytest.mark.parametrize("n_pages", [2 ** 30 + 1, 2 ** 31 - 1])
def test_more_pages_than_the_walk_over_their_counts_takes_are_refused(lib, n_pages):  # noqa: F811
    c = C.byref(abi._cache(n_pages=n_pages, workspace_bytes=1 << 40))
    fake = abi.FAKE
    assert lib.qd_pages_fork(c, fake, fake, 1, None) == -2
    assert lib.qd_pages_extend(c, fake, None) == -2
    assert lib.qd_pages_trim(c, fake, None) == -2
    assert lib.qd_pages_compact(c, fake, None) == -2
    assert b"n_pages" in lib.qd_last_error()


def test_a_stream_of_another_device_is_refused():
    # entering it would make its device current, and the call would then run on the tensors' own stream
    class Tensor:
        def get_device(self):
            return 1

    class Stream:
        device = torch.device("cuda", 0)

    with pytest.raises(ValueError, match="cuda:0"):
        api._elsewhere(Tensor(), Stream())


def test_the_binding_zeroes_the_head_that_the_header_names():
    header = open(os.path.join(ROOT, "include", "qd.h")).read()
    assert int(header.split("#define QD_ATTN_WORKSPACE_HEAD")[1].split()[0]) == api._ATTN_HEAD
