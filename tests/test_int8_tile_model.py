"""The constants by which gemm_a8w8 chooses its kernel, from the times they were fitted to, and what the choice costs on
the times of every kernel (no GPU: both tables are in profiles/, us per call)."""
import csv
import math
import os
import re

import numpy as np

from mxfp4_block_scaled_02_amd import build, ops

NAMES = list(ops.A8W8_PATHS.values())


def table(name):
    """[((M, N, K), {kernel: us}, row)]"""
    with open(os.path.join(build.ROOT, "profiles", name)) as f:
        return [(tuple(int(r[c]) for c in "MNK"), {n: float(r[n]) for n in NAMES if r[n]}, r) for r in csv.DictReader(f)]


def constants():
    """[(rows, columns, start, tile, step, tile_step)] of the kernels' source."""
    with open(os.path.join(build.CSRC, "gemm_int8.hip")) as f:
        rows = re.findall(r"^    \{(\d+), (\d+), ([-\d.]+)f, ([-\d.]+)f, ([-\d.]+)f, ([-\d.]+)f\},", f.read(), re.M)
    assert len(rows) == len(NAMES)
    return [(int(r[0]), int(r[1]), *map(float, r[2:])) for r in rows]


def terms(shape, bm, bn):
    M, N, K = shape
    n, t = -(-(-(-M // bm) * -(-N // bn)) // 256), K / 128
    return [1, n, t, n * t]


def test_constants_are_the_fit_of_the_times():
    times = table("int8_tile_fit.csv")
    assert len(times) == 255
    for name, (bm, bn, *c) in zip(NAMES, constants()):
        here = [(terms(shape, bm, bn), us[name]) for shape, us, _ in times if name in us]
        X, y = np.array([x for x, _ in here], float), np.array([t for _, t in here])
        fit, *_ = np.linalg.lstsq(X / y[:, None], np.ones(len(y)), rcond=None)  # least squares of the relative error
        assert np.allclose(fit, c, rtol=0, atol=6e-4), (name, fit, c)


def loss(rows):
    """(geometric mean, largest) of the chosen kernel's time over the fastest one's."""
    q = [us[r["chosen"]] / min(us.values()) for _, us, r in rows]
    return math.exp(sum(map(math.log, q)) / len(q)), max(q)


def test_cost_of_the_choice():
    rows = table("int8_tile_check.csv")
    assert all(ops.a8w8_path(*shape) == r["chosen"] for shape, _, r in rows)
    inside = [r for r in rows if max(r[0][1:]) <= 7168]
    wide = [r for r in rows if max(r[0][1:]) > 7168]
    assert len(inside) == 255 and len(wide) == 36
    mean, worst = loss(inside)
    assert mean < 1.0085 and worst < 1.235
    mean, worst = loss(wide)
    assert mean < 1.0105 and worst < 1.115


def test_the_model_ranks_and_does_not_predict():
    """Its figure for the chosen kernel over the measured time: the range that the comment at the constants states."""
    by_name = dict(zip(NAMES, constants()))

    def ratios(rows):
        out = []
        for shape, us, r in rows:
            bm, bn, *c = by_name[r["chosen"]]
            out.append(np.dot(c, terms(shape, bm, bn)) / us[r["chosen"]])
        return min(out), float(np.median(out)), max(out)

    rows = table("int8_tile_check.csv")
    low, mid, high = ratios([r for r in rows if max(r[0][1:]) <= 7168])
    assert 0.62 < low < 0.64 and 0.97 < mid < 0.99 and 1.26 < high < 1.28
    low, mid, high = ratios([r for r in rows if max(r[0][1:]) > 7168])
    assert 0.45 < low < 0.47 and 0.65 < mid < 0.67 and 1.12 < high < 1.14
