"""Sizes that reach every kernel of the products of two MXFP4 operands, and in the tiled ones every height of
a last row tile.  test_mx_select_host.py asserts that each case takes the kernel it is listed under;
test_gpu_mx_tiles.py runs them."""
from collections import namedtuple

# The names of csrc/wq_mx_select.hpp, in its order.
KERNELS = ("MX_STREAM_16", "MX_STREAM_32", "MX_TILES_64", "MX_TILES_128", "MX_TILES_128x256", "MX_TILES_128x256_ONE",
           "MX_TILES_256")

Dense = namedtuple("Dense", "kernel m n k")
# n that no 16-byte piece divides, k whose last step or stage (512, 256) ends inside; the last row tile has at
# most 64 rows, 65 to 128, or more
DENSE = [Dense("MX_STREAM_16", 9, 77, 576), Dense("MX_STREAM_16", 300, 77, 192), Dense("MX_STREAM_32", 40, 2101, 1088),
         Dense("MX_TILES_64", 513, 900, 1088), Dense("MX_TILES_128", 1300, 1701, 832),
         Dense("MX_TILES_128", 1380, 1700, 448), Dense("MX_TILES_128x256", 1440, 4100, 1344),
         Dense("MX_TILES_128x256", 1500, 4099, 320), Dense("MX_TILES_128x256_ONE", 4111, 4097, 576),
         Dense("MX_TILES_128x256_ONE", 4170, 4096, 832), Dense("MX_TILES_256", 3100, 4097, 2112),
         Dense("MX_TILES_256", 3172, 4100, 2368), Dense("MX_TILES_256", 3250, 4096, 2112)]

# counts: every expert's rows, empty experts among them; the rest of the t * topk pairs are dropped
Experts = namedtuple("Experts", "kernel gate_up t topk n k counts")
_FEW, _EIGHT, _THREE, _LONG = (0, 17, 1, 16, 3), (1, 64, 65, 128, 0, 100, 30, 5), (180, 326, 64), (300, 356, 0, 700)
EXPERTS = [Experts("MX_STREAM_16", True, 20, 2, 65, 576, _FEW), Experts("MX_STREAM_16", False, 20, 2, 130, 576, _FEW),
           Experts("MX_STREAM_16", True, 300, 2, 150, 192, (300, 280)),
           Experts("MX_STREAM_16", False, 300, 2, 300, 192, (300, 280)),
           Experts("MX_TILES_128", True, 165, 2, 350, 832, (64, 161, 65)),
           Experts("MX_TILES_128", False, 165, 2, 701, 832, (64, 161, 65)),
           Experts("MX_TILES_128x256", True, 100, 4, 1501, 1088, _EIGHT),
           Experts("MX_TILES_128x256", False, 100, 4, 2972, 1088, _EIGHT),
           Experts("MX_TILES_128x256_ONE", True, 300, 2, 2350, 704, _THREE),
           Experts("MX_TILES_128x256_ONE", False, 300, 2, 4701, 1856, _THREE),
           Experts("MX_TILES_256", True, 700, 2, 7201, 2112, _LONG),
           Experts("MX_TILES_256", False, 700, 2, 14401, 2112, _LONG)]


def rows_of_last_tiles(counts, height):
    """The heights of every expert's last row tile, in the classes at most 64, 65 to 128, more."""
    last = [(c - 1) % height + 1 for c in counts if c]
    return {0 if r <= 64 else 1 if r <= 128 else 2 for r in last}
