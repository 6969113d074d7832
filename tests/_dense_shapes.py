"""Shapes of the dense products' tests that are there for one kernel each: what test_dense_choice_cpu.py says of their
choice is what the tests on the GPU then run."""

# n, rows, cols: the products of S, of P and the update all by pairs of CTAs. Batches of one tile, of tiles off the
# diagonal, of sides that are no multiple of 8 or of a tile, both ways round.
UPDATES_BY_PAIRS = [(20, 512, 512), (76, 200, 264), (76, 264, 200), (152, 129, 131), (10, 1001, 1003), (10, 1003, 1001), (12, 777, 1030),
                    (12, 1030, 777)]
# T, H, I: long runs of k-blocks, one tile a CTA and SM
LONG = [(1024, 832, 2600), (100, 2600, 8000)]
