"""(tokens, cols, rows, experts, top, alike) that together run every form of the experts' products: each number of waves that share
a tile and of tiles a wave takes, on aligned rows and on rows that are not, with Wg and Wu starting alike between two multiples
of 16 bytes and (alike false) differently.  The ends are odd: numbers of rows that are no multiple of 16 or of a group of tiles,
odd numbers of those groups.  tests/test_moe_plan.py holds them to that."""

SHAPES = [
    # one token: 16, 8, 4, 2 and 1 waves for each of its experts
    (1, 136, 72, 5, 1, True), (1, 264, 520, 9, 2, True), (1, 1100, 104, 9, 4, True), (1, 200, 136, 12, 6, True),
    (1, 520, 264, 12, 8, True), (1, 72, 200, 40, 17, True),
    (1, 137, 71, 5, 1, True), (1, 130, 262, 9, 2, False), (1, 1101, 99, 9, 3, True), (1, 203, 131, 12, 5, False),
    (1, 523, 250, 12, 7, True), (1, 77, 204, 40, 20, False),
    # choices in the first product, in 4, 8 and 16 waves a tile
    (8, 1032, 264, 64, 8, True), (8, 2072, 136, 64, 8, True), (8, 264, 72, 64, 8, True),
    (8, 1001, 300, 64, 8, True), (8, 261, 300, 64, 8, False), (8, 2065, 140, 64, 8, False), (8, 130, 90, 64, 8, True),
    (5, 67, 34, 12, 3, False), (8, 131, 120, 64, 8, False), (8, 259, 140, 64, 8, True),
    # and not: the second product in 1 (by two tiles at once too), 2, 4, 8 and 16 waves a tile
    (128, 1032, 136, 64, 8, True), (128, 520, 72, 64, 8, True), (128, 264, 40, 64, 8, True), (64, 264, 200, 64, 8, True),
    (40, 200, 24, 20, 4, True), (16, 72, 264, 5, 2, True), (96, 1560, 40, 64, 8, True),
    (128, 1100, 135, 64, 8, True), (128, 1270, 37, 64, 8, False), (128, 1036, 140, 64, 8, False), (128, 1034, 126, 64, 8, False), (128, 500, 133, 64, 8, False),
    (128, 250, 130, 64, 8, True), (128, 133, 70, 64, 8, True), (64, 130, 138, 64, 8, False), (40, 131, 45, 20, 4, True),
    (16, 70, 150, 5, 2, False), (100, 1290, 36, 64, 8, True), (20, 259, 1290, 64, 2, False), (150, 65, 130, 3, 2, True),
]
