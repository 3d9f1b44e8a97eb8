"""Sizes that reach every kernel of the products of include/tsenor_ops.h, with the form that each takes:
tests/test_ops_forms.py holds the library's rule to it without a GPU, tests/test_gpu_ops_forms.py compares
the results.  A rule that sends a size elsewhere, or a form without a size, fails the former."""
import numpy as np

# columns, rows, buffers of the ring and workgroups at once of each tile fed by direct loads; weight gradients
# of 64 x 64 have a ring of 4, and a workgroup for each tile
TILES = {"256x256": (256, 256, 4, 256), "256x128": (256, 128, 6, 256), "128x128": (128, 128, 8, 256),
         "64x64": (64, 64, 8, 512)}

# rows, experts, m, k; the form of the product, of the transposed one, of 8-bit integers
PRODUCTS = [
    (10, 4, 200, 520, "few16", "64x64", "few16"),
    (5, 64, 1024, 264, "few32", "64x64", "few32"),
    (40, 5, 2048, 712, "few64", "64x64", "few64"),
    (64, 1, 1000, 712, "few32x32", "64x64", "few32x32"),
    (1000, 16, 520, 712, "64x64", "64x64", "64x64"),
    (1660, 13, 1032, 712, "64x64", "64x64", "64x64"),        # more tiles than workgroups
    (2900, 6, 1000, 712, "128x128", "128x128", "128x128"),
    (20000, 540, 120, 712, "128x128", "128x128", "128x128"),  # more tiles than workgroups
    (3000, 5, 2048, 712, "256x128", "256x128", "256x128"),
    (5000, 4, 2824, 712, "256x128", "256x128", "256x128"),    # more tiles than workgroups
    (4100, 3, 2056, 712, "256x256", "256x256", "256x256"),
    (9000, 5, 2304, 712, "256x256", "256x256", "256x256"),    # more tiles than workgroups
    (8300, 4, 8200, 72, "256x256", "256x256", "256x256"),     # so many that half tiles keep their places
    (3000, 2, 4097, 517, "staged256x128", "any", "256x256"),  # rows that are not 16-byte aligned
    (200, 3, 333, 517, "any", "any", "64x64"),
]

# rows, experts, m, k; the form
GRADIENTS = [
    (1001, 4, 1032, 1032, "64x64"),
    (3000, 2, 1288, 1032, "64x64"),
    (2600, 1, 1792, 2056, "128x128"),
    (8000, 8, 1024, 1024, "128x128"),  # more tiles than workgroups
    (2500, 5, 1800, 2056, "256x256"),
    (9000, 8, 1288, 2056, "256x256"),  # more tiles than workgroups
    (4000, 70, 520, 520, "256x256"),   # more than 64 experts
    (3000, 5, 511, 1001, "any"),
]


def counts_of(rows, experts):
    """Rows of each expert: uneven, some without any (of more than two experts), five rows of none."""
    rng = np.random.default_rng(rows + experts)
    share = rng.random(experts) + 0.1
    if experts > 2:
        share[rng.integers(experts)] = 0.0
    return rng.multinomial(rows - 5, share / share.sum()).tolist()


def tiles_of(form, counts, m):
    """Tiles of a product that hold rows of an expert."""
    columns, rows = TILES[form][:2]
    return -(-m // columns) * sum(-(-n // rows) for n in counts)
