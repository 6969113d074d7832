"""Which kernel the dense products of each tested shape take, by the host's own rule (gemm.cuh) for 152 SMs: a changed
estimate that leaves a kernel without a test on the GPU shows here. Needs nvcc, no GPU."""
import os
import subprocess

import pytest

from w4a16_moe_decode_gb300.build import ARCH, CSRC, INCLUDE, nvcc

import test_gpu_dense_overlap
import test_gpu_ffn
import test_gpu_orthogonalize
import test_gpu_orthogonalize_elements
from _dense_shapes import LONG, UPDATES_BY_PAIRS

PROGRAM = r"""
#include <cstdio>
#include "gemm.cuh"
using namespace flint::gemm;
struct Plain { static constexpr bool PAIR = false, SMALL = false; };
struct Gated { static constexpr bool PAIR = true, SMALL = false; };
struct Few { static constexpr bool PAIR = false, SMALL = true; };
static void put(const char* what, const Choice& c) { printf("%s:%s%d ", what, c.kind == 0 ? "pairs" : c.kind == 1 ? "one" : "half", c.S); }
static int blocks(int k) { return (k + BK - 1) / BK; }
int main() {
  char op;
  int a, b, c;
  while (scanf(" %c %d %d %d", &op, &a, &b, &c) == 4) {
    if (op == 'o') {  // matrices, rows, columns: the operands' sizes of orthogonalize.cu
      const int m = std::min(b, c), k = std::max(b, c), segs = m <= 32 ? 3 : m <= 64 ? 2 : 1;
      const int halves = m <= 32 ? 3 : 1;
      const Args gram = {{{m, m, blocks(k), halves, 0, 0, 0, 0, 1, a}}, 1, 1, nullptr, 0}, poly = {{{m, m, blocks(m), halves, 0, 0, 0, 0, 1, a}}, 1, 1, nullptr, 0};
      put("gram", m <= 32 ? choose<Few>(gram) : choose<Plain>(gram));
      put("poly", m <= 32 ? choose<Few>(poly) : choose<Plain>(poly));
      put("update", choose<Plain>({{{b, c, blocks(m), segs, 0, 0, 0, 0, 0, a}}, 1, 1, nullptr, 0}));
    } else {  // tokens, hidden, inter: those of ffn.cu
      put("glu", choose<Gated>({{{a, c, blocks(b), 1, 0, 0, 0, 0, 0, 1}}, 1, 0, nullptr, 0}));
      put("down", choose<Plain>({{{a, b, blocks(c), 1, 0, 0, 0, 0, 0, 1}}, 1, 0, nullptr, 0}));
      put("dglu", choose<Plain>({{{a, c, blocks(b), 1, 0, 0, 0, 0, 0, 1}}, 1, 0, nullptr, 0}));
      const Problem px = {a, b, blocks(c), 2, 0, 0, 0, 0, 0, 1}, pw = {c, b, blocks(a), 1, 0, 0, 0, 0, 0, 1}, pd = {b, c, blocks(a), 1, 0, 0, 0, 0, 0, 1};
      int64_t cycles[3];
      const Choice all = choose<Plain>({{px, pw, pw, pd}, 4, 0, nullptr, 0}, &cycles[0]);
      const Choice dx = choose<Plain>({{px}, 1, 0, nullptr, 0}, &cycles[1]), dw = choose<Plain>({{pw, pw, pd}, 3, 0, nullptr, 0}, &cycles[2]);
      if (cycles[0] <= cycles[1] + cycles[2]) {
        put("grads", all);
      } else {
        put("dx", dx);
        put("dw", dw);
      }
    }
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cu").write_text(PROGRAM)
    exe = str(d / "choice")
    subprocess.run([nvcc(), *ARCH, "-std=c++17", "-I", INCLUDE, "-I", CSRC, str(d / "choice.cu"), "-o", exe], check=True, capture_output=True)

    def run(op, shapes):
        """[{product: kernel}] of each shape."""
        text = "".join(f"{op} {a} {b} {c}\n" for a, b, c in shapes)
        # (no device, so that the rule is asked for the SMs that it was made for)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}).stdout
        return [dict(w.split(":") for w in line.split()) for line in out.splitlines()]

    return run


def test_updates_by_pairs(chosen):
    for shape, c in zip(UPDATES_BY_PAIRS, chosen("o", UPDATES_BY_PAIRS)):
        assert set(c.values()) == {"pairs1"}, (shape, c)


def test_updates_of_every_kernel(chosen):
    """Each product of an update by each kernel that the rule has for it, over the shapes that the cluster kernel leaves."""
    shapes = [s for s in test_gpu_orthogonalize.SHAPES + test_gpu_orthogonalize_elements.OTHERS + UPDATES_BY_PAIRS if min(s[1:]) > 128]
    got = chosen("o", shapes + [(1, 256, 2048), (1, 20, 9001), (1, 9001, 20)])
    for product in ("gram", "poly", "update"):
        kinds = {c[product][:-1] for c in got}
        assert kinds == {"pairs", "one", "half"}, (product, kinds)
    assert {c["gram"][-1] for c in got} >= {"1", "4", "8"}  # clusters along K


def test_blocks_of_every_kernel(chosen):
    forward = chosen("f", test_gpu_ffn.SHAPES + test_gpu_ffn.LARGE + LONG)
    for product, kinds in (("glu", {"pairs", "one"}), ("down", {"pairs", "half"}), ("dglu", {"pairs", "half"}),
                           ("dx", {"pairs", "half", "one"}), ("dw", {"pairs", "half"}), ("grads", {"pairs", "half"})):
        assert {c[product][:-1] for c in forward if product in c} >= kinds, product
    assert test_gpu_ffn.LONG == LONG
    first, second = chosen("f", LONG)
    assert first["down"] == "half1" and second["dw"] == "pairs1" and second["dx"][-1] != "1"  # one tile a CTA, and clusters


def test_calls_side_by_side_take_clusters_and_pairs(chosen):
    steps = [a[1:4] for pair in test_gpu_dense_overlap.PAIRS for a in pair if a[0] is test_gpu_dense_overlap.Step]
    kinds = {v for c in chosen("f", steps) for v in c.values()}
    assert any(k[-1] != "1" for k in kinds) and "pairs1" in kinds
