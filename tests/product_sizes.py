"""The products' host arithmetic (csrc/zero_product_sizes.h) compiled by itself."""
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_optimizer_step_gb300", "csrc")


def run(body: str, *args) -> str:
    """What a program with this main() prints."""
    program = ('#include <cstdio>\n#include <cstdlib>\n#include <initializer_list>\n#include "zero_product_sizes.h"\n'
               "using namespace zgb;\nusing namespace zgb::product;\n"
               "int main(int argc, char **argv)\n{\n" + body + "\n}\n")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "sizes.cpp"), os.path.join(d, "sizes")
        with open(src, "w") as f:
            f.write(program)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, src, "-o", exe],
                       check=True)
        return subprocess.run([exe, *map(str, args)], check=True, capture_output=True,
                              text=True).stdout


def pair_shape(m: int, n: int, sms: int, gated: bool) -> dict:
    """How the pair kernel goes over an m by n result."""
    names = ("half", "cut", "tiles_m", "tiles_n", "whole", "steps")
    out = run("    const PairShape g = pair_shape(atoll(argv[1]), atoll(argv[2]), atoi(argv[3]), "
              "atoi(argv[4]));\n" + "".join('    printf("%%lld ", (long long)g.%s);\n' % x
                                            for x in names) + "    return 0;", m, n, sms,
              int(gated))
    return dict(zip(names, map(int, out.split())))
