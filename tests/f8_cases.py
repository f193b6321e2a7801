"""Calls of the E4M3 products that between them reach every kernel and every part of their loops on a device of 256 CUs:
which one takes them is checked without a GPU (test_f8_cut_cpu.py), what they compute on one (test_gpu_f8_ways.py)."""

CUS = 256
WAYS = ["T64x32", "T64x64", "T128x64", "T128x128", "G256x32Wide", "G256x64Wide", "G256x64", "G256x128", "T64x32Wide", "T64x64Wide",
        "T128x128Wide", "T256x256", "G256x256"]

# tokens, n, k of products: the way, and the parts of K.  A wave holds the weights' scales of 64 blocks of 128 at a time, so
# parts of more than that load them again.
PRODUCTS = [
    (20, 144, 16400, "T64x32", 7),
    (32, 1936, 262144, "T64x32", 5),       # 410 blocks a part
    (40, 144, 272, "T64x64", 1),
    (70, 16, 262144, "T64x64", 29),        # 71
    (1003, 2064, 8336, "T64x64", 1),       # 66
    (510, 6160, 144, "T128x64", 1),
    (130, 6160, 8336, "T128x64", 3),
    (61, 16400, 8336, "T128x64", 1),       # 66
    (1003, 6160, 400, "T128x128", 1),
    (200, 4112, 8336, "T128x128", 3),
    (510, 6160, 8336, "T128x128", 1),      # 66
    (2040, 6160, 528, "T256x256", 1),      # an odd number of blocks, ragged last tiles
    (4090, 8176, 400, "T256x256", 1),      # two tiles for each workgroup
    (1003, 6160, 8336, "T256x256", 1),     # 66
]
# tokens, inter, hidden: the way of gate and up, and the parts of hidden
GATED = [
    (20, 400, 2064, "G256x32Wide", 3),
    (20, 1152, 262144, "G256x32Wide", 10),  # 205 blocks a part
    (40, 272, 1040, "G256x64Wide", 2),
    (50, 1168, 262144, "G256x64Wide", 16),  # 128
    (70, 144, 272, "G256x64", 1),
    (70, 272, 2064, "G256x64", 3),
    (70, 2064, 66048, "G256x64", 7),        # 74
    (1003, 6160, 16, "G256x128", 1),
    (3000, 272, 4112, "G256x128", 3),
    (1280, 400, 66048, "G256x128", 6),      # 86
    (510, 8208, 272, "G256x256", 1),        # an odd number of blocks, ragged last tiles
    (2040, 2064, 8336, "G256x256", 1),      # 66
    (2040, 8176, 528, "G256x256", 1),       # two tiles for each workgroup
]
# The same of plans with exact products.
EXACT_PRODUCTS = [
    (20, 144, 16400, "T64x32Wide", 10),
    (32, 1936, 262144, "T64x32Wide", 8),    # 256 blocks a part
    (33, 144, 272, "T64x64Wide", 1),
    (300, 4112, 2064, "T64x64Wide", 2),
    (1003, 2064, 8336, "T64x64Wide", 1),    # 66
    (510, 2064, 8336, "T128x128Wide", 3),
    (1003, 6160, 8336, "T128x128Wide", 1),  # 66
]
EXACT_GATED = [
    (65, 272, 1040, "G256x64Wide", 2),
    (70, 2064, 66048, "G256x64Wide", 7),    # 74
    (2040, 2064, 528, "G256x64Wide", 1),
]
# Up to 16 tokens, whose codes a workgroup holds 512 blocks at a time (all tokens' together).
FEW_PRODUCTS = [(3, 48, 262144), (16, 144, 66048)]
FEW_GATED = [(16, 272, 4240), (1, 272, 66048), (5, 144, 13328), (3, 272, 22160), (16, 4240, 272), (1, 66048, 272), (7, 9616, 9616)]
