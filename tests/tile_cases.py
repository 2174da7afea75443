"""Shapes that take each product tile of the library: what test_gpu_tiles.py runs, and what
test_tile_rules_host.py holds against the rules that choose the tiles.  Whoever changes a rule moves
the shapes with it."""

# swz_gemm_f8: (m, n) by the tile it takes, rows x columns of C; fp32 results with fp32 scales of both
# operands' rows take 128 x 256 where the others take 256 x 256.
GEMM = {(64, 64): (130, 200), (64, 128): (1000, 1100), (128, 128): (1500, 1500), (256, 256): (2100, 2200)}
# one block of 128, two, an odd count, a count with a tail, a tail alone
GEMM_K = [128, 256, 384, 1000, 40]

# Losses: (n, v, k) by the rows of the forward call's tiles, of the gradient's logits' tiles (each piece of
# the vocabulary) and of dW's tiles.
LOSS = {(300, 16500, 200): (128, [128], [128]),
        (600, 33000, 136): (256, [256, 256], [128, 64]),
        (600, 33000, 1032): (256, [256, 256], [256, 256])}
