"""Which sizes take which kernel of the 8-bit operators, and the comparison that the product's tests share.

tests/test_int8_launches.py holds the tables against the library's own choice (on the host, through the
recorded launches), tests/test_gpu_int8_paths.py runs them.
"""
import numpy as np

U = 2.0 ** -24
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -126}  # half a subnormal step (fp32: flush)
TYPES = ("f16", "bf16", "f32")


def product_errors(got, want, mag, dt):
    """Where an output of the product is not what its definition allows; a NaN never is.

    want: the outputs in 64 bits; mag: |scaled sum| + |bias|, which the fp32 roundings go by (the sum's, two
    products', the addition's: below 5 U).  fp16 outputs from 65520 on round to the infinity of their sign.
    """
    off = 5 * U * mag
    ok = np.abs(got - want) <= UNIT[dt] * np.abs(want) + off + TINY[dt]  # False for NaN and infinities
    if dt == "f16":
        ok &= np.abs(want) - off < 65520
        ok |= (np.abs(want) + off >= 65520) & (got == np.copysign(np.inf, want))
    return ~ok


# tile (channels x tokens, stages in LDS) -> its instance's parameters, (tokens, channels) that take it at any
# k from `least_k` on, columns per stage
TILES = {
    "16x16": ("8", (5, 300), 1, 256),
    "32x32": ("32, 32, 1, 1, 4, 256, 4, 2", (17, 4243), 1, 256),
    "64x32": ("64, 32, 2, 1, 2, 256, 3, 4", (7, 13843), 1, 256),
    "32x64": ("32, 64, 1, 2, 2, 256, 4, 4", (39, 4236), 1, 256),
    "64x64": ("64, 64, 2, 2, 1, 128, 4, 4", (38, 8651), 1, 128),
    "64x128": ("64, 128, 2, 4, 1, 128, 4, 4", (71, 8500), 1, 128),
    "128x128": ("128, 128, 2, 4, 1, 128, 4, 2", (69, 16489), 1, 128),
    "128x128 of two stages": ("128, 128, 2, 4, 1, 128, 2, 2", (137, 24863), 1, 128),
    "256x256": ("256, 256, 2, 4, 1, 128, 2, 1", (524, 20483), 760, 128),  # the rule takes it for long k only
}


def tile_ks(tile):
    """For 1 to 6 stages (16 x 16, which has none: blocks of a wave) a k with no tail, with a tail of whole
    16-byte pieces and with one inside a piece; for the largest tile 6 to 9 stages."""
    least, kb = TILES[tile][2:]
    first = -(-least // kb)
    return [s * kb - cut for s in range(first, first + (6 if least == 1 else 4)) for cut in (0, 16, kb - 37)
            if s * kb - cut >= least]


# name -> (rows, vocab, the rows kernel's parameters behind the type, splits, slices of a workgroup)
PLANS = {
    "one wave": (2000, 500, "true, 64", 1, 1),                          # up to 32 alternatives only
    "a short row": (1500, 2000, "true, 256", 1, 1),
    "short splits": (3, 40001, "true, 256", 20, 1),
    "a row in registers": (40, 32751, "false, 1024", 1, 1),
    "wide splits": (64, 131072, "false, 256", 16, 1),
    "wide splits of two slices": (40, 262147, "false, 256", 22, 2),
    "a workgroup over four slices": (1100, 32001, "false, 256", 1, 4),
    "a workgroup over seven slices": (600, 50003, "false, 256", 1, 7),
}


def plan_top_ks(plan):
    return (1, 5, 32) if plan == "one wave" else (1, 20, 64)
