"""(tokens, cols, rows, with an activation) that together run every form of the linear layer's tiled product (each product by
each kind of tiles, with its contraction whole and split) for every number of steps, modulo the steps after which
a kind's images repeat; and dx and dW by one launch too, in either kind of tiles; eight steps and more, so that its steady loop runs.  tests/test_linear_plan.py holds them to that."""

SHAPES = [
    (1368, 1856, 264, True), (1224, 512, 1256, True), (288, 2792, 1808, True), (263, 1360, 1024, True),
    (1784, 912, 272, True), (35, 7424, 2248, False), (3430, 3680, 69, True), (360, 704, 328, True),
    (1149, 520, 1864, False), (960, 664, 2248, False), (3672, 536, 3608, True), (362, 5480, 328, True),
    (1537, 1480, 1336, False), (1349, 1616, 1504, False), (3323, 2848, 648, True), (131, 8576, 5872, False),
    (408, 8352, 408, True), (750, 3296, 608, False), (138, 9688, 5680, False), (535, 7000, 520, True),
    (577, 7336, 576, False), (767, 648, 5624, False), (847, 5384, 728, False), (4914, 848, 832, False),
    (131, 9928, 5552, True), (1153, 3280, 3408, True), (4560, 1896, 1088, True), (3916, 7056, 528, True),
    (4952, 2312, 880, True), (3172, 8528, 392, True), (837, 9760, 792, False), (4153, 1000, 4176, True),
    (925, 9632, 876, False), (1073, 7224, 1120, False), (1015, 8608, 1008, False), (262, 9984, 1102, True),
    (1091, 9984, 984, False), (322, 9896, 1088, True), (1283, 528, 5936, False), (1141, 9912, 1096, False),
    (391, 8304, 1360, True), (2446, 648, 3208, False), (4234, 976, 3544, True), (1350, 8184, 3136, False),
    (2055, 720, 3881, True), (2206, 776, 3611, False), (1305, 832, 5936, False), (4902, 648, 2328, True),
    (2107, 704, 5630, False), (2756, 7664, 1576, False), (2565, 784, 4441, True), (4957, 848, 2320, False),
    (837, 8320, 4736, False), (600, 1000, 776, True), (777, 1237, 1001, True), (700, 904, 971, False),
    (1150, 2168, 1324, False), (1106, 1872, 913, False)]
