"""Calls of the operators on windows, pages and caches made shorter whose work lists are long: the kernels' larger arguments, and
lists of several launches.  What launches a call makes is tested without a GPU, what it gives on one."""

# name: (query rows, key rows, query heads, kv heads, window, sinks, a view per sequence, launches: (entries of the type, views of it))
KEY_WEIGHTS = {
    "256 entries": ([100], [20000], 8, 2, 0, 0, False, [(256, 1)]),
    "256 entries, a window": ([333, 1], [30000, 500], 4, 1, 20000, 300, False, [(256, 1)]),
    "1152 entries": ([100], [80000], 8, 2, 0, 0, False, [(1152, 1)]),
    "1152 entries, a window": ([700, 3], [120000, 9000], 4, 1, 70000, 40, False, [(1152, 1)]),
    "two launches": ([100], [350000], 4, 1, 0, 0, False, [(1152, 1)] * 2),
    "two launches, ragged": ([97, 25, 60], [200000, 60001, 130003], 4, 1, 0, 0, False, [(1152, 1)] * 2),
    "two launches of views": ([100, 30], [120000, 90000], 4, 1, 0, 0, True, [(768, 64)] * 2),
}
# more than 4096 blocks of query rows over the same keys: what they receive is added to what an earlier launch left
MANY_ROWS = dict(L=50000, window=64, sinks=200, hq=8, hkv=1)

# name: (query rows, key rows, query heads, kv heads, window, sinks, a view per sequence or pages, launches as above)
ATTENTION = {
    "views in one": ([800] * 64, [800] * 64, 8, 1, 300, 3, "view", [(1536, 1)] * 2),
    "views in one, one cut": ([800] * 63 + [60], [800] * 63 + [40000], 8, 1, 0, 0, "view", [(1536, 1)] * 2),
    "a view each": ([310] * 64, [310 + 7 * s for s in range(64)], 8, 1, 200, 5, "views", [(576, 65)] * 2),
    "pages": ([800] * 64, [800] * 64, 8, 1, 500, 3, "pages", [(1536, 1)] * 2),
    "pages, one cut": ([800] * 63 + [60], [800] * 63 + [40000], 8, 1, 0, 0, "pages", [(1536, 1)] * 2),
}
