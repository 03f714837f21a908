"""Products (rows of x, rows of weights, K, two weights, fp16 rows) whose blocks work in clusters
on several tiles, one after the other."""

# clusters that share K, with K of whole steps and not: (the blocks of a cluster, product)
SHARED = [(8, (4, 4695, 4672, 0, 1)), (8, (6, 4908, 4736, 0, 1)), (4, (7, 9798, 2656, 0, 1)), (2, (8, 19534, 1184, 0, 1)),
          (2, (7, 19668, 1280, 0, 1)), (8, (7, 4639, 11840, 0, 0)), (8, (5, 4906, 11904, 0, 0)), (4, (387, 2573, 15264, 0, 0)),
          (4, (507, 939, 14752, 1, 0)), (4, (500, 960, 14752, 1, 0))]
# pairs with two accumulators for every other step, and an odd number of steps: the two warps that
# issue products change places from tile to tile
PAIRS_ODD = [(207, 4893, 384, 0, 0), (199, 4893, 896, 0, 0), (16, 39080, 384, 0, 0), (200, 4096, 384, 1, 0), (133, 4869, 1152, 1, 0)]
