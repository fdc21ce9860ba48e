"""The kernels' own reading of a tree's masks (``tree_bits`` in ``internal.h``), compiled for the host, against the
definition (no GPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import _trees as tr
from mixed_attention_quantized_gb300 import build

SOURCE = """
#include "internal.h"
extern "C" void read_masks(const uint32_t* masks, int rows, int words, int n, int rel0, int rels, uint32_t* out) {
  for (int i = 0; i < rows; ++i)
    for (int r = 0; r < rels; ++r) out[i * rels + r] = mixattn::tree_bits(masks + (long)i * words, words, n, rel0 + r);
}
"""


@pytest.fixture(scope="module")
def read(tmp_path_factory):
    d = tmp_path_factory.mktemp("tree_bits")
    (d / "bits.cc").write_text(SOURCE)
    lib = str(d / "libbits.so")
    subprocess.run([build._cxx(), "-O1", "-std=c++17", "-fPIC", "-shared", "-I", build.CSRC, str(d / "bits.cc"), "-o", lib],
                   check=True)
    f = ctypes.CDLL(lib).read_masks
    f.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 5 + [ctypes.c_void_p]

    def call(masks, n, rels):
        """uint32 [rows, rels] of packed masks [rows, words], which end at the end of their memory's words."""
        out = np.zeros((masks.shape[0], len(rels)), dtype=np.uint32)
        f(masks.ctypes.data, *masks.shape, n, rels[0], len(rels), out.ctypes.data)
        return out

    return call


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 70, 1023, 1024])
@pytest.mark.parametrize("more", [0, 1, 3])
@pytest.mark.parametrize("stray", [False, True])
def test_every_window_of_32_keys(read, n, more, stray):
    rng = np.random.default_rng(n)
    m = rng.random((min(n, 40), n)) < 0.5
    m[0], m[-1] = True, False
    words = (n + 31) // 32 + more
    bits = np.full((len(m), 32 * words), stray)
    bits[:, :n] = m
    packed = (bits.reshape(len(m), words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    rels = range(-70, n + 70)
    got = read(np.ascontiguousarray(packed), n, rels)
    # keys -102 .. n + 101 behind the context: all of the context, the mask's, none past the row
    line = np.concatenate([np.ones((len(m), 102), bool), m, np.zeros((len(m), 102), bool)], 1)
    for i, rel in enumerate(rels):
        want = (line[:, 102 + rel:134 + rel].astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
        assert np.array_equal(got[:, i], want.astype(np.uint32)), rel


def test_the_tests_packing_is_what_it_reads(read):
    masks = [tr.random_tree(n, np.random.default_rng(n), 2) for n in (5, 40, 70)]
    packed = np.ascontiguousarray(tr.pack(masks, stray=True).view(np.uint32))
    at = 0
    for m in masks:
        n = len(m)
        got = read(packed[at:at + n].copy(), n, range(0, 96))
        assert np.array_equal((got[:, ::32][:, :, None] >> np.arange(32) & 1).reshape(n, -1)[:, :n].astype(bool), m)
        at += n
