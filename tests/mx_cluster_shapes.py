"""Products (rows of x, rows of weights, K, two weights, fp16 rows) whose blocks, in clusters or
by themselves, work on several tiles, one after the other."""

# clusters that share K, with K of whole steps and not: (the blocks of a cluster, product)
SHARED = [(8, (4, 4695, 4672, 0, 1)), (8, (6, 4908, 4736, 0, 1)), (4, (7, 9798, 2656, 0, 1)), (2, (8, 19534, 1184, 0, 1)),
          (2, (7, 19668, 1280, 0, 1)), (8, (7, 4639, 11840, 0, 0)), (8, (5, 4906, 11904, 0, 0)), (4, (387, 2573, 15264, 0, 0)),
          (4, (507, 939, 14752, 1, 0)), (4, (500, 960, 14752, 1, 0))]
# pairs with two accumulators for every other step, and an odd number of steps: the two warps that
# issue products change places from tile to tile
PAIRS_ODD = [(207, 4893, 384, 0, 0), (199, 4893, 896, 0, 0), (16, 39080, 384, 0, 0), (200, 4096, 384, 1, 0), (133, 4869, 1152, 1, 0)]
# blocks by themselves with several tiles each; all but the first have a K that fits no step
ALONE = [(3, 45000, 128, 0, 1), (5, 40000, 160, 0, 1), (700, 4000, 96, 0, 0), (2100, 1300, 160, 0, 0), (300, 8000, 160, 1, 0),
         (130, 21001, 96, 1, 0), (16, 40000, 224, 1, 0)]
# fp16 rows of an odd number of steps and several tiles a block: the warps that issue products change
# places from tile to tile, while the rows are still being taken apart
ROWS_ODD = [(7, 29719, 128, 0, 1), (8, 60000, 128, 0, 1), (8, 40000, 96, 0, 1), (8, 30000, 384, 0, 1), (6, 25000, 640, 0, 1)]
