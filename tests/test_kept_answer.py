"""The number of a kernel's registers that the 4-bit decode asks for before its first launch
(kept_answer.h): a question that fails is asked again, an answer is kept."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_paged_attention_gb300", "csrc")

MAIN = r"""
#include "kept_answer.h"
#include <cstdio>
enum Status { OK = 0, FAILED = 2 };
int asked = 0;
int main() {
  std::atomic<int> kept{0};
  // two failures (which may have written something), then an answer, then a question that would fail again
  auto ask = [](int* n) { *n = 7 + asked; return ++asked == 3 ? OK : FAILED; };
  for (int i = 0; i < 5; ++i) {
    int v = -1;
    const Status st = qpa::kept_answer(kept, ask, v);
    printf("%d %d %d\n", (int)st, st == OK ? v : 0, asked);
  }
}
"""


def test_a_failed_question_is_not_kept(tmp_path):
    src, exe = str(tmp_path / "k.cpp"), str(tmp_path / "k")
    with open(src, "w") as f:
        f.write(MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, src, "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    assert out[:5] == ["2 0 1", "2 0 2", "0 9 3", "0 9 3", "0 9 3"]


def test_the_decode_asks_through_it():
    with open(os.path.join(CSRC, "pa_nvfp4.cu")) as f:
        text = f.read()
    assert text.count("cudaFuncGetAttributes") == 1 and "kept_answer(kept, " in text
