"""Host-side checks that stand between a call and a kernel that could not end."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "qwen3_decoder_block_b200", "csrc")


def test_a_failed_check_fails_every_call(tmp_path):
    """A kernel that may not be launched is refused each time, not only the first one."""
    gxx, cuda = shutil.which("g++"), "/usr/local/cuda/include"
    if gxx is None or not os.path.isdir(cuda):
        pytest.skip("no host compiler or CUDA headers")
    src = tmp_path / "ready.cpp"
    src.write_text('''#include "internal.h"
int main() {
  q3::ReadyKernels r;
  int calls = 0, a = 0, b = 0;
  auto bad = [&] { ++calls; return -6; };
  auto good = [&] { ++calls; return 0; };
  if (r.once(&a, 0, bad) != -6 || r.once(&a, 0, bad) != -6 || calls != 2) return 1;
  if (r.once(&a, 0, good) != 0 || r.once(&a, 0, bad) != 0 || calls != 3) return 2;
  if (r.once(&a, 1, bad) != -6 || r.once(&b, 0, bad) != -6 || calls != 5) return 3;
  return 0;
}
''')
    exe = str(tmp_path / "ready")
    subprocess.run([gxx, "-std=c++17", "-I", cuda, "-I", CSRC, str(src), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_warpgroup_splits_fit_the_registers_at_launch():
    """setmaxnreg.inc takes from what the block was launched with: the shares of a kernel's warpgroups
    must not add up to more than its threads times the registers the compiler gave them."""
    import __graft_entry__
    __graft_entry__.build()
    log = os.path.join(ROOT, "qwen3_decoder_block_b200", "lib", "libqwen3blk.so.ptxas.log")
    if not os.path.exists(log):
        pytest.skip("the library was built elsewhere, without the compiler's report")
    regs = dict(re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", open(log).read(), flags=re.S))

    def used(word):
        found = [int(v) for k, v in regs.items() if word in k]
        assert len(found) == 1, (word, found)
        return found[0]

    # shares of the warpgroups (128 threads each), as the sources state them
    paged = open(os.path.join(CSRC, "attention_paged.cu")).read()
    s8, s16, c8, c16, widen = map(int, re.search(
        r"kRegsSoftmax = FP8 \? (\d+) : (\d+), kRegsCtl = FP8 \? (\d+) : (\d+), kRegsWiden = (\d+)", paged).groups())
    assert used("attn_paged_chunk_kernelILb0E") * 384 >= (2 * s16 + c16) * 128
    assert used("attn_paged_chunk_kernelILb1E") * 512 >= (2 * s8 + c8 + widen) * 128
    flat = open(os.path.join(CSRC, "attention.cu")).read()
    softmax, ctl = (int(re.search(rf"constexpr int kPrefillRegs{n} = (\d+)", flat).group(1)) for n in ("Softmax", "Ctl"))
    assert used("attn_prefill_kernel") * 384 >= (2 * softmax + ctl) * 128
