"""Shapes of the layer for one token by the form its down product takes (T, H,
I, E, K, the parts of the form with shared rows; 0: the other form), shared by
the tests of the choice and of the results."""
import torch

BF, FP = torch.bfloat16, torch.float16
TYPES = [(BF, BF), (FP, FP), (BF, torch.int8), (FP, torch.int8)]

# Repeated ids of one expert (K = 2 E) count as much to read whatever its
# size; the last two are 24 MiB of weights and more.
ONE_TOKEN = {
    2: [(1, 4096, 4101, 1, 2, 4), (1, 4112, 4101, 1, 2, 0), (1, 80, 4099, 1, 2, 4),
        (1, 4096, 3203, 3, 1, 3), (1, 4112, 3203, 3, 1, 0)],
    1: [(1, 4096, 4101, 1, 2, 4), (1, 4112, 4101, 1, 2, 4), (1, 80, 4099, 1, 2, 4),
        (1, 4096, 6407, 3, 1, 6), (1, 4112, 6407, 3, 1, 6)],
}


def one_token(wdtype):
    return ONE_TOKEN[1 if wdtype == torch.int8 else 2]
