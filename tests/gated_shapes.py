"""(tokens, cols, rows) that together run every form of the gated block's tiled product (each
product by each kind of tiles, with its contraction whole and split) for every number of steps, modulo
the steps after which a kind's images repeat, that the form takes; eight steps and more, so
that its steady loop runs.  tests/test_gated_plan.py holds them to that."""

SHAPES = [
    (256, 520, 128), (320, 576, 200), (1024, 704, 520), (384, 640, 520), (1024, 776, 170), (320, 4160, 392),
    (1100, 2048, 128), (256, 2304, 1032), (777, 776, 2311), (448, 1000, 4100), (513, 1024, 4100), (1800, 2304, 200),
    (1800, 2304, 256), (2304, 904, 2304), (777, 704, 2311), (1800, 704, 4096), (2048, 4160, 128), (777, 832, 2311),
    (384, 904, 4100), (2048, 4160, 200), (1800, 576, 2304), (2048, 4160, 256), (1800, 640, 2304), (1800, 776, 2304),
    (1800, 832, 2304), (513, 2304, 4096)]
