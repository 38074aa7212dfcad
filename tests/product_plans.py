"""Sizes that bring the dense product through every kernel of its plans, K split over workgroups and not, with the last
band, block, column tile and part incomplete. Shared by the CPU test that holds them against the plan and the GPU test
that runs them."""

# (N, M): one more token than whole tiles, and most of a tile more; rows that fill neither their band nor their tile
ONE = [(1, 1), (25, 9), (4097, 1), (4123, 9), (4097, 42), (4143, 41), (2721, 33), (49, 2092), (4161, 66), (4145, 74), (33, 4231),
       (50, 4107), (65, 5530), (5480, 73), (257, 3657), (161, 5707), (513, 3715), (321, 5661), (769, 5255), (5470, 650),
       (4609, 1671), (1415, 5434), (1, 4131), (16, 4100)]
# one column tile, less than one, an odd and an even number of them, more than any ring has stages
COLUMNS = [5, 64, 130, 449, 1000]

# (N, M, K): K split (with a workspace), the last part shorter than the others
SPLIT = [(1, 1, 18792), (1, 1, 18575), (168, 81, 38736), (83, 169, 39681), (165, 328, 39801), (180, 325, 41361),
         (129, 231, 29432), (161, 194, 29316), (305, 199, 20337), (181, 349, 20273), (261, 249, 21343), (276, 244, 20244),
         (325, 393, 15589), (297, 411, 15497), (387, 616, 12486), (520, 501, 11545), (852, 635, 9590), (682, 742, 9099),
         (1098, 959, 9084), (750, 1428, 9018), (2204, 1315, 37727), (1209, 2413, 38176)]

# at most 4 tokens and weights of 32 MB and more
STREAM = [(1, 4090, 8200), (3, 4090, 8200), (4, 391, 90000), (2, 8210, 8330), (1, 14498, 2346), (4, 14490, 2400)]

KERNELS = ["k_w8_stream<16, 2>", "k_w8_stream<8, 4>", "k_w8_ring<1, 1, 4, 2>", "k_w8_ring<1, 1, 16, 2>", "k_w8_ring<2, 1, 8, 2>",
           "k_w8_ring<2, 2, 8, 2>", "k_w8_ring<4, 1, 4, 3>", "k_w8_ring<2, 4, 6, 2>", "k_w8_ring<4, 2, 6, 2>",
           "k_w8_tiles<2, 2, 2, 2, 4, 3>", "k_w8_tiles<2, 2, 4, 2, 2, 3>", "k_w8_tiles<2, 4, 4, 2, 1, 4>",
           "k_w8_tiles<2, 4, 8, 2, 1, 4>", "k_w8_tiles<2, 4, 8, 4, 1, 3>"]
NEVER_SPLIT = KERNELS[:3]
