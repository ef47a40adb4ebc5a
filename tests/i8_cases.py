"""Sizes that reach every kernel of the products of two int8 operands, and in the tiled ones every height of
a last row tile.  test_i8_host.py asserts that each case takes the kernel it is listed under; test_gpu_i8.py
runs them."""
from collections import namedtuple

# The names of csrc/wq_i8_select.hpp, in its order.
KERNELS = ("I8_STREAM_16", "I8_STREAM_32", "I8_NARROW", "I8_TILES_64", "I8_TILES_128", "I8_TILES_128x256", "I8_TILES_256")

Dense = namedtuple("Dense", "kernel m n k")
# n that no 16-byte piece divides, k whose last step or stage (256, 128) ends inside; the last row tile of the
# large tiles has at most 64 rows, 65 to 128, 129 to 192, or more
DENSE = [Dense("I8_STREAM_16", 1, 1, 64), Dense("I8_STREAM_16", 9, 77, 576), Dense("I8_STREAM_16", 300, 77, 192),
         Dense("I8_STREAM_32", 100, 1001, 1088), Dense("I8_STREAM_32", 32, 4095, 64),
         Dense("I8_NARROW", 33, 2100, 64), Dense("I8_NARROW", 100, 1101, 320), Dense("I8_NARROW", 64, 4099, 576),
         Dense("I8_NARROW", 127, 1053, 832), Dense("I8_NARROW", 128, 1701, 1088), Dense("I8_NARROW", 1500, 129, 192),
         # every number of stages modulo the four that are on their way
         Dense("I8_TILES_64", 20, 24600, 64), Dense("I8_TILES_64", 250, 3105, 192), Dense("I8_TILES_64", 100, 2601, 320),
         Dense("I8_TILES_64", 64, 6000, 512), Dense("I8_TILES_64", 70, 8190, 576), Dense("I8_TILES_64", 333, 1111, 704),
         Dense("I8_TILES_64", 32, 6145, 832), Dense("I8_TILES_64", 17, 4130, 960), Dense("I8_TILES_64", 513, 3000, 1088),
         Dense("I8_TILES_64", 9, 8177, 1152), Dense("I8_TILES_64", 3, 24577, 448),
         Dense("I8_TILES_128", 1300, 1701, 832), Dense("I8_TILES_128", 1380, 1700, 448),
         Dense("I8_TILES_128x256", 1440, 4100, 1344), Dense("I8_TILES_128x256", 1500, 4099, 320),
         Dense("I8_TILES_256", 3100, 4097, 1088), Dense("I8_TILES_256", 3172, 4100, 1152),
         Dense("I8_TILES_256", 3250, 4096, 64), Dense("I8_TILES_256", 3300, 4096, 192)]

# counts: every expert's rows, empty experts among them; the rest of the t * topk pairs are dropped
Experts = namedtuple("Experts", "kernel gate_up t topk n k counts")
_FEW, _EIGHT, _THREE, _LONG = (0, 17, 1, 16, 3), (1, 64, 65, 128, 0, 100, 30, 5), (180, 326, 64), (300, 356, 0, 230, 444)
EXPERTS = [Experts("I8_STREAM_16", True, 20, 2, 65, 576, _FEW), Experts("I8_STREAM_16", False, 20, 2, 130, 576, _FEW),
           Experts("I8_TILES_128", True, 165, 2, 350, 832, (64, 161, 65)),
           Experts("I8_TILES_128", False, 165, 2, 701, 832, (64, 161, 65)),
           Experts("I8_TILES_128", True, 300, 2, 2350, 704, _THREE),
           Experts("I8_TILES_128", False, 300, 2, 4701, 64, _THREE),
           Experts("I8_TILES_128x256", True, 100, 4, 8201, 448, _EIGHT),
           Experts("I8_TILES_128x256", False, 100, 4, 16301, 448, _EIGHT),
           Experts("I8_TILES_256", True, 700, 2, 7201, 1088, _LONG),
           Experts("I8_TILES_256", False, 700, 2, 14401, 1088, _LONG)]


def heights_of_last_tiles(counts, height):
    """The kernels' heights of every expert's last row tile, in 64 rows."""
    return {(c - 1) % height // 64 + 1 for c in counts if c}
