"""Shapes (n, k, f) of the gated block that reach each tile of its products, held to the rules by a host test and run by a
GPU test."""

FORWARD = {"few": [(16, 72, 130), (32, 136, 200)], "k64x32": [(40, 136, 200), (130, 72, 600)], "k128x32": [(100, 72, 4200), (300, 64, 2700)],
           "k64x128": [(200, 72, 5000)], "k128x128": [(1000, 72, 3000)], "k256x128": [(2000, 64, 3000)]}
# by tile, whether the sum is split and whether it goes over two terms of dg and du
DX = {("k64x64", False, True): (10, 72, 33), ("k64x64", True, True): (10, 72, 130), ("k128x256", False, True): (20000, 72, 1), ("k64x64", False, False): (16, 2056, 257),
      ("k64x64", True, False): (16, 264, 2000), ("k64x256", False, False): (1000, 264, 33), ("k64x256", True, False): (10, 4104, 1000),
      ("k128x128", False, False): (20000, 72, 33), ("k128x128", True, False): (70, 4104, 1000),
      ("k128x256", False, False): (20000, 136, 33), ("k128x256", True, False): (70, 2056, 5000),
      ("k256x256", False, False): (20000, 264, 33), ("k256x256", True, False): (3000, 136, 3000)}
DW = {("k64x64", False, True): (10, 72, 33), ("k64x64", True, True): (520, 72, 33), ("k128x256", False, True): (2, 72, 9000), ("k64x64", False, False): (129, 520, 130),
      ("k64x64", True, False): (1000, 264, 33), ("k64x256", False, False): (16, 264, 2000), ("k64x256", True, False): (1500, 4104, 33),
      ("k128x128", False, False): (16, 72, 9000), ("k128x128", True, False): (1000, 72, 3000),
      ("k128x256", False, False): (10, 136, 9000), ("k128x256", True, False): (2100, 136, 3000),
      ("k256x256", False, False): (10, 72, 20000), ("k256x256", True, False): (1500, 72, 9000)}
