"""Which shape of tiles a product of given sizes takes (CPU: the library's rule,
compiled by itself), so that the GPU tests' sizes reach every one."""
import os
import subprocess

from _product_shapes import GRADIENTS, PRODUCTS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "message_fp16_all_amd", "csrc")

PROGRAM = """
#include <cstdio>
#include "product_shape.h"
using namespace hr;
int main() {
    const char *shapes[] = {"Large", "Half", "Middle", "Some", "Low", "Few", "FewAcross", "Tiny", "AnyMiddle", "AnyFew"};
    const char *gradients[] = {"Large", "Middle", "Deep", "AnyMiddle"};
    char what;
    size_t experts, rows, a, b, any;
    while (std::scanf(" %c %zu %zu %zu %zu %zu", &what, &experts, &rows, &a, &b, &any) == 6) {
        if (what == 'g')
            std::puts(gradients[int(gradient_shape(int(experts), a, b, any))]);
        else
            std::puts(shapes[int(product_shape(rows, int(experts), b, what == 't', any))]);
    }
    std::printf("%d %d\\n", int(ProductShape::AnyFew), int(GradientShape::AnyMiddle));
}
"""


def test_the_sizes_reach_every_shape(tmp_path):
    source = tmp_path / "shapes.cc"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(source), "-o", str(tmp_path / "shapes")], check=True)
    asked, want = [], []
    for along, across, experts, rows, k, n in PRODUCTS:
        odd = int(n % 16 != 0)
        asked += [f"p {experts} {rows} {k} {n} {odd}", f"t {experts} {rows} {k} {n} {odd}"]
        want += [along, across]
    for shape, experts, rows, n, k in GRADIENTS:
        asked.append(f"g {experts} {rows} {n} {k} {int(n % 8 != 0)}")
        want.append(shape)
    out = subprocess.run([str(tmp_path / "shapes")], input="\n".join(asked), check=True, capture_output=True, text=True).stdout
    *got, counts = out.split("\n")[:-1]
    assert got == want
    assert counts == "9 3"
    assert len({s for p in PRODUCTS for s in p[:2]}) == 10 and len({g[0] for g in GRADIENTS}) == 4
