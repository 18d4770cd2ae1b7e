"""The tests' copy of the adapters' split rules against the header itself."""
import os
import random
import subprocess

from delayed_scaling_linear_amd import build
from tests import adapter_splits as splits

PROGRAM = r"""
#include <cstdio>
#include "adapter.h"
using namespace fp8dsl;
int main() {
    long rows, adapters, rank, in, out;
    while (scanf("%ld %ld %ld %ld %ld", &rows, &adapters, &rank, &in, &out) == 5) {
        const AdapterPlanShape p(rows, adapters);
        printf("%ld %d %d %ld %ld %ld\n", (long)p.tiles_max, adapter_parts(p.tiles_max, in, rank),
               adapter_parts(p.tiles_max, out, rank),
               (long)adapter_expand_chunk(p.tiles_max, in, rank),
               (long)adapter_expand_chunk(p.tiles_max, out, rank),
               (long)adapter_chunk(p.tiles_max, rank, in, out));
    }
}
"""


def test_the_copy_follows_the_header(tmp_path):
    (tmp_path / "splits.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "splits")
    subprocess.run([build.hipcc(), "--offload-host-only", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
                    "-x", "hip", str(tmp_path / "splits.cpp"), "-o", exe],
                   check=True, capture_output=True, env={**os.environ, "TMPDIR": str(tmp_path)})
    rng = random.Random(0)
    sizes = [(rng.choice([1, 40, 1500, 4200, 8300, rng.randrange(1, 1 << 20)]), rng.randrange(1, 60),
              8 * rng.randrange(1, 17), 8 * rng.randrange(1, 1300), 8 * rng.randrange(1, 1300))
             for _ in range(4000)]
    text = "\n".join(" ".join(map(str, s)) for s in sizes)
    lines = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout.split("\n")
    for (rows, count, rank, n_in, n_out), line in zip(sizes, lines):
        t = splits.tiles(rows, count)
        assert line.split() == [str(v) for v in (
            t, splits.parts(t, n_in, rank), splits.parts(t, n_out, rank),
            splits.expand_chunk(t, n_in, rank), splits.expand_chunk(t, n_out, rank),
            splits.gradient_chunk(t, rank, n_in, n_out))]
