"""Calls of the latent tree operator whose results are counts.

Queries are 0 but for one rotary element, so that each key weighs 1 or nothing
(a score of thousands below 0: every odd row does without the keys of every odd
group), and a latent column is 1 for the keys of one group of 64 (every
`latent`-th group), else 0.  A row's output is then, column by column, the
number of such keys that it sees over the number of all that it sees.  Sums of
up to 2^24 ones are exact in float32, and so is a weight of 1 in bf16; what is
left is the reciprocal, the product and the rounding of the output.  A tile
that is lost, taken twice, or taken for another row changes a column by a
whole group."""
import numpy as np

GROUP = 64

CASES = {
    # name: lengths, nodes, heads, latent, page, kernel, mode, form of the join
    # 80 units of 128 and 7 rows in 76 parts: parts that end a unit, hold whole ones and begin another
    "pairs 512, more units than parts": ([(i * 397) % 1500 for i in range(40)], 5, 27, 512, 128, "pairs", "cut", 0),
    "pairs 256, more units than parts": ([(i * 397) % 1500 for i in range(40)], 5, 27, 256, 0, "pairs", "cut", 0),
    "pairs 512, many units and refused ones": ([None if i % 11 == 5 else (i * 211) % 900 for i in range(90)], 3, 41, 512, 0,
                                               "pairs", "cut", 0),
    "pairs 512, ragged trees": ([512 + 1097 * i for i in range(8)], 60, 32, 512, 128, "pairs", "cut", 0),
    "pairs 256, ragged trees": ([100 + 1097 * i for i in range(8)], 61, 31, 256, 0, "pairs", "cut", 0),
    "pairs 512, a few units": ([5000, 70, 1900], 9, 33, 512, 128, "pairs", "cut", 1),
    "pairs 256, a few units": ([5000, 70, 1900], 9, 33, 256, 0, "pairs", "cut", 1),
    "pairs 512, one unit": ([30000], 3, 11, 512, 128, "pairs", "cut", 8),
    "pairs 256, one unit": ([30000], 2, 9, 256, 0, "pairs", "cut", 8),
    "pairs 512, short units": ([0] * 30 + [4000], 2, 64, 512, 0, "pairs", "cut", 1),
    "pairs 512, halves": ([32768] * 4, 4, 128, 512, 0, "pairs", "halves", 1),
    "pairs 256, halves": ([82000] * 2, 3, 90, 256, 0, "pairs", "halves", 1),
    "pairs 512, halves of one sequence": ([93000], 5, 67, 512, 128, "pairs", "halves", 1),
    "pairs 512, whole": ([1000] * 70, 1, 64, 512, 128, "pairs", "whole", 0),
    "pairs 256, several whole": ([500 + i % 7 for i in range(100)], 7, 19, 256, 0, "pairs", "whole", 0),
    "few 512, more units than parts": ([(i * 397) % 1500 for i in range(230)], 1, 16, 512, 128, "few", "cut", 1),
    "few 256, more units than parts": ([(i * 397) % 1500 for i in range(300)], 1, 13, 256, 0, "few", "cut", 1),
    "few 512, refused ones": ([None if i % 13 == 2 or 50 < i < 90 else (i * 211) % 900 for i in range(210)], 1, 16, 512, 0, "few",
                              "cut", 1),
    "few 512, one token": ([20000], 1, 16, 512, 128, "few", "cut", 8),
    "few 256, one token of one head": ([20000], 1, 1, 256, 0, "few", "cut", 8),
    "few 512, rows of several units": ([700, 90], 3, 37, 512, 128, "few", "cut", 8),
}


def group_column(at, latent):
    return at // GROUP % latent


def tree_column(node, latent):
    return latent - 1 - node % 16


def odd(at):
    return at // GROUP % 2 == 1


def expected(length, nodes, heads, latent, mask, groups=None):
    """out [nodes, heads, latent] in float64; `groups`: how often each of the
    prefix's groups of keys is taken (once each)."""
    at = np.arange(length)
    weigh = np.ones(length) if groups is None else np.repeat(groups, GROUP)[:length]
    out = np.zeros((nodes, heads, latent))
    for parity in (0, 1):
        see = weigh * ~(odd(at) & (parity == 1))
        prefix = np.bincount(group_column(at, latent), weights=see, minlength=latent)
        for i in range(nodes):
            own = np.bincount(tree_column(np.arange(nodes), latent), weights=mask[i].astype(float), minlength=latent)
            rows = [h for h in range(heads) if (i * heads + h) % 2 == parity]
            out[i, rows] = (prefix + own) / (prefix.sum() + own.sum())
    return out


def tolerance(ref, half_step):
    """A reciprocal and a product in float32, and the output's rounding."""
    return ref * (half_step + 2.0 ** -22)
