"""The training products' schedule on the CPU (tests/train_schedule.cpp walks
csrc/tg_plan.h, the code that the kernels and their launches use): every k step
of every tile once, parts and boxes within their buffers, joins of just the parts
that were stored, nothing at all for a piece that the device's row count leaves
out."""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import pytest

from flash_mixed_chunk_gb300 import _buildlib

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def schedule(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("schedule") / "schedule.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_buildlib.nvcc())), "include")
    # an overflow of signed arithmetic ends the process
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-ftrapv", "-w", "-I",
                    _buildlib.CSRC, "-isystem", cuda, os.path.join(HERE, "train_schedule.cpp"),
                    "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.check_vocab_gradients.restype = ctypes.c_char_p
    lib.check_projection_gradients.restype = ctypes.c_char_p
    return lib


def vocab(lib, cg, M, V, d, count, workers, cap=0):
    return lib.check_vocab_gradients(cg, M, V, d, count, workers, cap).decode()


# more rows and a longer vocabulary than the pieces of 256 columns, and few rows
# with a target: the queued pieces go far beyond the ones that are there
@pytest.mark.parametrize("M,V,d,count", [
    (300000, 5000000, 64, 1000), (300000, 4300000, 384, 1024), (300000, 5000000, 64, 0),
    (1 << 24, 1 << 24, 8, 5), (262145, 4200000, 64, 1000), (300000, 5000000, 64, 9000),
    (1 << 22, 40000000, 48, 70), ((1 << 24) - 1, (1 << 24) - 1, 8, 1 << 12)])
@pytest.mark.parametrize("workers", [76, 74])
def test_pieces_that_are_not_there(schedule, M, V, d, count, workers):
    assert vocab(schedule, 2, M, V, d, count, workers) == ""


# the sizes at which the kernels run, in one piece and several
@pytest.mark.parametrize("cg,M,V,d", [
    (2, 16384, 32000, 768), (2, 8192, 32000, 768), (2, 2048, 50001, 512), (1, 37, 8191, 256),
    (2, 4200, 40100, 64), (2, 8200, 33000, 64), (2, 70000, 2100, 16), (1, 1, 1, 8),
    (1, 100, 530000, 8), (1, 100, 530000, 64), (2, 300, 263000, 8), (2, 512, 300000, 64)])
def test_listed_sizes(schedule, cg, M, V, d):
    for count in {M, M // 7, 1, 0}:
        for workers in (152 // cg, 148 // cg, 3):
            assert vocab(schedule, cg, M, V, d, count, workers) == ""


def log_int(r, lo, hi):
    return int(round(lo * (hi / lo) ** r.random()))


@pytest.mark.parametrize("seed", range(8))
def test_random_vocabularies(schedule, seed):
    r = random.Random(seed)
    for _ in range(200):
        cg = r.choice((1, 2))
        M = log_int(r, 1, 128) if cg == 1 else log_int(r, 129, 60000)
        V, d = log_int(r, 1, 60000), 8 * log_int(r, 1, 256)
        count = r.choice((M, r.randint(0, M), r.randint(0, min(M, 300))))
        one = schedule.vocab_boxes(M, 256)
        cap = r.choice((0, one, one + r.randint(0, 5000), one * r.randint(1, 6)))
        cap = min(cap, schedule.vocab_boxes(M, V))
        workers = r.choice((152 // cg, 148 // cg, r.randint(1, 152 // cg)))
        got = vocab(schedule, cg, M, V, d, count, workers, cap)
        assert got == "", (cg, M, V, d, count, workers, cap, got)


@pytest.mark.parametrize("seed", range(4))
def test_random_projections(schedule, seed):
    r = random.Random(100 + seed)
    for _ in range(200):
        cg = r.choice((1, 2))
        M = log_int(r, 1, 128) if cg == 1 else log_int(r, 129, 60000)
        N, d = 64 * log_int(r, 1, 64), 8 * log_int(r, 1, 256)
        workers = r.choice((152 // cg, 148 // cg, r.randint(1, 152 // cg)))
        for blocked in (0, 1):
            got = schedule.check_projection_gradients(cg, M, N, d, blocked, workers).decode()
            assert got == "", (cg, M, N, d, blocked, workers, got)
