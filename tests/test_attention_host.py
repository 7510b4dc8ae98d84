"""The attention kernel's own source on the CPU (hip_on_host/), with so few
workgroups that each one takes many tiles, items and requests: the refill of
its buffers, cuts inside and at the borders of items, the second look-up of
pages, and the counted waits. Every access is checked, the scratch has the size
that its workgroups use, and results are held against sums in 64 bits (attention_host.cpp)."""
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests import host_kernel

# query heads a key head, rows of a request: blocks of 16, 32, 64, 128 and 256 queries
BLOCKS = {16: (2, 2, 8), 32: (5, 4, 6), 64: (8, 5, 8), 128: (8, 9, 16), 256: (8, 17, 36)}
TYPES = [(b, d) for b in (0, 1) for d in (64, 128, 256) if b or d < 256]
KERNELS = [(b, d, m) for b, d in TYPES for m in BLOCKS if d < 256 or m < 256]
TREE, CHAIN, RISING, MALFORMED = range(4)


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    scratch = "  __shared__ AttnScratch<E, D, QT, WQ, WK> s;\n"
    return host_kernel.program(tmp_path_factory.mktemp("attention"), "attention.hip", "attention_host.cpp",
                               ((scratch, scratch + "  emu_tiles(&s, sizeof(s), s.tile, sizeof(s.tile));\n"),
                                ("kJoinGroups = 2048", "kJoinGroups = 3")))


def _run(program, bf16, D, block, kv, page, cus, B, lens, kind, seed):
    G, lo, hi = BLOCKS[block]
    out = host_kernel.run(program, bf16, D, G * kv, kv, page, cus, B, lo, hi, lens[0], lens[1], kind, seed, block)
    assert "ok" in out


def _all(program, cases):
    with ThreadPoolExecutor(4) as pool:
        for done in [pool.submit(_run, program, *c) for c in cases]:
            done.result()


@pytest.mark.parametrize("block", BLOCKS)
def test_long_spans(program, block):
    # one or two workgroups: spans of several requests, empty contexts among them
    _all(program, [(b, d, m, kv, page, cus, B, lens, kind, m + d + kind) for b, d, m in KERNELS if m == block
                   for kind, kv, page, cus, B, lens in ((TREE, 2, 16, 1, 3, (0, 300)), (CHAIN, 1, 2, 3, 2, (300, 500)),
                                                        (RISING, 1, 8, 1, 2, (200, 400)))])


def test_pages_are_looked_up_again(program):
    # pages of one token: more of them in a span than fit at a time
    _all(program, [(b, d, m, 1, 1, 1, 1, (2100, 2400), TREE, m) for b, d, m in KERNELS if d == 64 or m == 32])


def test_random_batches(program):
    for_seed = lambda s: KERNELS[s * 7 % len(KERNELS)]
    _all(program, [(*for_seed(s), 1 + s % 3, 1 << s % 6, 1 + s % 4, 1 + s % 7, (0, 60 + 15 * s), TREE, s) for s in range(16)])


def test_cuts_near_the_borders_of_items(program):
    # items several times as long as the reach within which a cut moves to a border
    _all(program, [(s // 4 % 2, 64, (16, 32, 64, 256)[s % 4], 1 + s % 3, 16, (2, 3, 5)[s % 3], 1 + s % 4, (900, 2200), CHAIN, s)
                   for s in range(15) if s not in (3, 7, 11)] + [(1, 64, 256, 1, 16, 3, 1, (1500, 2200), CHAIN, 3)])


def test_malformed_batches_stay_inside(program):
    # lengths, pages, offsets and parents out of range: nothing beyond the arrays is touched
    for_seed = lambda s: KERNELS[s * 5 % len(KERNELS)]
    _all(program, [(*for_seed(s), 2, 4, 1 + s % 3, 6, (0, 150), MALFORMED, s) for s in range(24)])
