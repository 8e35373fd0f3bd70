"""Sizes that send the vocabulary loss to its main kernels: the streamed tiles with more
tiles than the 256 workgroups, so that some take two, and the large tiles of the
gradients' products over one piece of the vocabulary and over several.  The CPU test
holds the rule to these choices; the GPU test runs them."""
import collections

# T, H, V; the tiles of the loss, and how many of them; pieces; both gradients' pair of tiles and slices of dx; whether dx
# alone takes the tiles for few rows
Case = collections.namedtuple("Case", "T H V loss tiles pieces pair slices few")

TILES = {0: (256, 256), 1: (256, 128), 2: (128, 128), 3: (128, 64), 4: (64, 64), 5: (32, 32), 6: (128, 256)}

CASES = [
    Case(40, 64, 70000, 6, 274, 1, 7, 16, False),
    Case(33, 72, 70008, 6, 274, 1, 6, 16, False),     # a masked last stage
    Case(100, 64, 70000, 6, 274, 1, 7, 16, False),
    Case(128, 200, 70008, 6, 274, 1, 5, 16, False),
    Case(65, 4104, 70000, 6, 274, 1, 0, 6, True),
    Case(100, 2056, 124000, 6, 485, 1, 0, 12, True),
    Case(300, 64, 30000, 6, 354, 1, 6, 16, False),    # three row tiles
    Case(380, 72, 30008, 6, 354, 1, 5, 16, False),
    Case(150, 72, 70000, 1, 547, 1, 5, 16, False),
    Case(1000, 64, 20000, 1, 628, 1, 6, 8, False),
    Case(4100, 2056, 16392, 0, 1105, 2, 0, 1, False),
    Case(2100, 512, 33000, 0, 1161, 2, 1, 8, False),
    Case(2100, 1032, 24584, 0, 873, 1, 2, 2, False),
    Case(2100, 2056, 4104, 0, 153, 1, 3, 1, False),
    Case(18000, 264, 9000, 0, 2556, 3, 5, 1, False),
]
