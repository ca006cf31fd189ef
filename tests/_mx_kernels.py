"""Which kernel a product of microscaled tensors runs in: the library's own rule (mx_route of csrc/pkv_internal.h) in a small host
program, and shapes for each kernel."""
import functools
import os
import shutil
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_qk_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "pkv_internal.h"
int main()
{
    for (int row, tokens, out, sms; scanf("%d %d %d %d", &row, &tokens, &out, &sms) == 4;) {
        const pkv::MxRoute r = pkv::mx_route(row, tokens, out, sms);
        printf("%d %d %d\n", (int)r.pairs, r.tile, r.splits);
    }
    return 0;
}
"""
SMS = 152
PAIRS = "pairs"


@functools.lru_cache(None)
def _program():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    d = tempfile.mkdtemp(prefix="mx_route")
    src, exe = os.path.join(d, "route.cu"), os.path.join(d, "route")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-I", CSRC, "-o", exe, src], check=True, capture_output=True)
    return exe


def route(kind, tokens, n_in, n_out, sms=SMS):
    """PAIRS, or (tokens a tile, CTAs of a cluster)."""
    row = n_in if kind == "mx8" else n_in // 2
    out = subprocess.run([_program()], input=f"{row} {tokens} {n_out} {sms}\n", capture_output=True, text=True, check=True).stdout
    pairs, tile, splits = map(int, out.split())
    return PAIRS if pairs else (tile, splits)


# (tokens, input features, output features) and where they run, in either kind, on 152 SMs
FEW = [
    ((9, 4224, 1024), (16, 8)), ((9, 4096, 6144), (16, 4)), ((9, 1152, 12800), (16, 2)), ((9, 640, 20480), (16, 1)),
    ((27, 4224, 1024), (32, 8)), ((27, 4096, 6144), (32, 4)), ((27, 1152, 12800), (32, 2)), ((27, 640, 20480), (32, 1)),
    ((50, 4224, 1024), (64, 8)), ((50, 4096, 4096), (64, 4)), ((50, 1152, 6144), (64, 2)), ((50, 640, 12800), (64, 1)),
    ((1, 4096, 20480), (16, 1)), ((20, 4096, 20480), (32, 1)), ((40, 4096, 20480), (64, 1)),  # a ring used again, more tiles than SMs
    ((300, 4096, 1280), (64, 2)),
    ((1, 12288, 4096), (16, 4)), ((20, 4096, 24576), (32, 1)),  # an MLP's widths
]
MANY = [
    ((49, 640, 19584), PAIRS),      # the odd CTA of a pair wholly beyond the tokens; a 4-bit row of two stages and a half
    ((70, 1152, 20480), PAIRS),     # a 4-bit row that ends in half a stage
    ((129, 4096, 10240), PAIRS),    # one token beyond half a tile; more stages than the rings hold
    ((257, 1152, 6144), PAIRS),     # one token beyond a tile
    ((700, 128, 2048), PAIRS),      # less than a stage in 4 bits
    ((1025, 4096, 3200), PAIRS),    # features of a tile and a third
    ((700, 16512, 2048), PAIRS),    # a long row
    ((2048, 8192, 1280), PAIRS),
    ((64, 4096, 24576), PAIRS), ((300, 12288, 4096), PAIRS),  # an MLP's widths
    ((5000, 384, 384), PAIRS),      # many tiles a pair, a stage and a half each in 4 bits
]
