"""The rotating decode in a process of its own, under the tuning variables that
the parent set (they are read once per process).  Exit status 0: it passed."""

import sys

import torch

from tests.test_gpu_rotary_decode import LENS, case16, check16, step16


def main() -> int:
    dev = torch.device("cuda", 0)
    for dtype, d, heads in (("bf16", 128, (32, 8)), ("f16", 64, (8, 8))):
        lens, tables, kc, vc, q, k, v, slots, rot, w = case16(dev, LENS, *heads, d, dtype, 21)
        out, where = step16(dev, lens, tables, kc, vc, q, k, v, slots, rot)
        check16(out, where, w, rot, lens, tables, kc, vc, q, dtype)
    return 0


if __name__ == "__main__":
    sys.exit(main())
