"""Sizes that send the vocabulary loss to its main kernels: the streamed tiles with more
tiles than the 256 workgroups, so that some take two, and the large tiles of the
gradients' products over one piece of the vocabulary and over several.  The CPU test
holds the rule to these choices; the GPU test runs them."""
import collections

# T, H, V; the tiles of the loss and of dz, and how many of them; pieces; whether the gradients take the tiles for few
# rows, else the pair of tiles; slices of dx
Case = collections.namedtuple("Case", "T H V loss tiles dz pieces few pair slices")

TILES = {0: (256, 256), 1: (256, 128), 2: (128, 128), 3: (128, 64), 4: (64, 64), 5: (32, 32), 6: (64, 512), 7: (128, 256)}

CASES = [
    Case(40, 64, 140000, 6, 274, 6, 1, True, None, 220),
    Case(33, 72, 140008, 6, 274, 6, 1, True, None, 220),   # a masked last stage
    Case(100, 64, 70000, 7, 274, 7, 1, True, None, 183),
    Case(128, 200, 70008, 7, 274, 7, 1, True, None, 110),
    Case(300, 64, 30000, 7, 354, 7, 1, False, 6, 16),      # three row tiles
    Case(380, 72, 30008, 7, 354, 7, 1, False, 5, 16),
    Case(150, 72, 70000, 1, 547, 1, 1, False, 5, 16),
    Case(1000, 64, 20000, 1, 628, 1, 1, False, 6, 8),
    Case(4100, 2056, 16392, 0, 1105, 0, 2, False, 0, 1),
    Case(2100, 512, 33000, 0, 1161, 0, 2, False, 1, 8),
    Case(2100, 1032, 24584, 0, 873, 0, 1, False, 2, 2),
    Case(2100, 2056, 4104, 0, 153, 0, 1, False, 3, 1),
    Case(20000, 264, 9000, 0, 2844, 0, 3, False, 5, 1),
]
