"""Helper of the tests of the operators around the mixer (not collected)."""
import numpy as np


def half_step(v):
    """Half of bf16's step at |v| (eight significant bits): what a rounding to
    nearest is off by at most."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 8)
