"""Launches that may begin under the end of the one before them: what the
operators' sources have to keep to, by reading them (no GPU)."""
import glob
import os
import re
import shutil
import subprocess

import pytest

OPS = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "adamw_optimizer_step_persistent_gb300", "csrc", "ops")


def _close(text, at, pair):
    """Behind the bracket that closes the one before `at`."""
    depth = 1
    while depth:
        depth += {pair[0]: 1, pair[1]: -1}.get(text[at], 0)
        at += 1
    return at


def _functions():
    """{(file, name): (is a kernel, body)} of the kernels, and of the functions
    that are one kind of their CTAs."""
    found = {}
    for path in sorted(glob.glob(os.path.join(OPS, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\bvoid\s+", text):
            at = m.end()
            while attribute := re.compile(r"__\w+__\(").match(text, at):
                at = re.compile(r"\s*").match(text, _close(text, attribute.end(), "()")).end()
            name = re.compile(r"(\w+)\(").match(text, at)
            if not name:
                continue
            at = re.compile(r"[\s\w]*").match(text, _close(text, name.end(), "()")).end()
            kernel = text[:m.start()].rstrip().endswith("__global__")
            if text[at] == "{" and (kernel or name[1].endswith("_cta")):
                found[os.path.basename(path), name[1]] = (kernel, text[at:_close(text, at + 1, "{}")])
    return found


FUNCTIONS = _functions()
KERNELS = sorted(k for k, (kernel, _) in FUNCTIONS.items() if kernel and k[1] != "take_status_kernel")


def _waits(at):
    body = FUNCTIONS[at][1]
    if re.search(r"\n  chain_wait\(\);", body):
        return True
    # a kernel of several kinds of CTAs: each of them
    kinds = re.findall(r"\b(\w+_cta)\b", body)
    return bool(kinds) and all(_waits((at[0], k)) for k in kinds)


def test_kernels_are_found():
    sources = "".join(re.sub(r"//[^\n]*", "", open(p).read()) for p in glob.glob(os.path.join(OPS, "*.cu*")))
    assert len(KERNELS) == sources.count("__global__") - 1


@pytest.mark.parametrize("at", KERNELS, ids=lambda at: at[1])
def test_every_thread_waits_for_the_launch_before(at):
    """What earlier launches wrote is visible behind a kernel's own wait only:
    it stands in the kernel's (or its CTAs') outermost block, behind no condition."""
    assert _waits(at)
    assert not re.search(r"if \([^\n]*\)\s*chain_wait\(\)", FUNCTIONS[at][1])


NVCC = "/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else shutil.which("nvcc")


@pytest.mark.skipif(NVCC is None, reason="no nvcc")
def test_a_failed_question_for_a_kernels_registers_is_asked_again(tmp_path):
    """With a runtime call of the test's own that fails once: the second call of
    the operator is not refused for the first one's failure."""
    src = tmp_path / "ask.cu"
    src.write_text("""
#include <stdarg.h>
#include <stdio.h>
#include "ops/attention.cuh"
static int asked = 0, registers = 96;
extern "C" int answer(cudaFuncAttributes* f) {
  if (++asked == 1) return cudaErrorMemoryAllocation;
  f->numRegs = registers;
  return cudaSuccess;
}
namespace fadam_ops {
fadam_status fail(fadam_status st, const char* fmt, ...) { return st; }
fadam_status cuda_fail(cudaError_t, const char*) { return FADAM_ECUDA; }
}
template <int N> __global__ void kernel() {}
int main() {
  using fadam_ops::launched_with;
  const int first = launched_with<kernel<0>>("it"), second = launched_with<kernel<0>>("it");
  const int third = launched_with<kernel<0>>("it"), known = asked;
  registers = 95;
  const int other = launched_with<kernel<1>>("it"), again = launched_with<kernel<1>>("it");
  printf("%d %d %d %d %d %d", first, second, third, known, other, again);
}
""")
    own = tmp_path / "own.cpp"
    own.write_text("""
extern "C" int answer(void*);
extern "C" int cudaFuncGetAttributes(void* f, const void*) { return answer(f); }
""")
    root = os.path.dirname(os.path.dirname(os.path.dirname(OPS)))
    exe = str(tmp_path / "ask")
    subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-cudart", "shared",
                    "-I", os.path.dirname(OPS), "-I", os.path.join(root, "include"), str(src), str(own), "-o", exe],
                   check=True, capture_output=True)
    env = dict(os.environ, LD_LIBRARY_PATH=os.path.join(os.path.dirname(os.path.dirname(NVCC)), "lib64"))
    out = subprocess.run([exe], check=True, capture_output=True, text=True, env=env).stdout
    failed = 4      # FADAM_ECUDA
    assert out == f"{failed} 0 0 2 {failed} {failed}"


def test_waits_of_whole_warps_have_one_answer():
    """Elected lanes, loads of tensor memory and group barriers take all lanes of a
    warp: a wait that gives up does so for all of them.  (One thread alone waits in
    the warp that loads.)"""
    for kind in ("keys_cta", "queries_cta"):
        assert not re.search(r"\bbar_wait\(", FUNCTIONS["attention_backward.cuh", kind][1])
    body = FUNCTIONS["attention_forward.cuh", "attention_forward_kernel"][1]
    _, others = body.split("} else if (warp == kMultiply || warp == kMultiply2) {")
    assert not re.search(r"\bbar_wait\(", others) and "warp_wait(" in others
