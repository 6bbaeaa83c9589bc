"""Host-side checks of the operators around a layer's products at the ends of their arguments' ranges (no
GPU)."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from test_layer_host import B, P, _forward, _orthogonalize

far = pytest.mark.skipif(torch.cuda.is_available(), reason="no work may be queued with these addresses")


@pytest.mark.parametrize("over", [dict(ldo=1 << 39, os=1 << 39), dict(os=1 << 39), dict(ldg=1 << 39), dict(gs=1 << 39)])
def test_matrix_strides_that_no_memory_has(over):
    """2^39 values of 2 bytes is what a tensor map's stride cannot hold."""
    assert _orthogonalize({**dict(rows=30, cols=48), **over}) == B.ERR_SHAPE


@far
@pytest.mark.parametrize("over", [dict(ldo=1 << 33, os=1 << 38), dict(ldg=1 << 38, gs=1 << 38),
                                  dict(batch=1, gs=1 << 50, os=1 << 50), dict(batch=1, rows=1, ldg=1 << 50, ldo=1 << 50)])
def test_matrix_strides_that_are_accepted(over):
    assert _orthogonalize({**dict(rows=30, cols=48), **over}) in (B.ERR_DEVICE, B.ERR_CUDA)


@pytest.mark.parametrize("over", [
    # token 1's first head is token 0's third: what lies between the tokens, in values, passes 2^63
    dict(T=1 << 30, positions=P, out_strides=(1 << 34, 1 << 33)),
    dict(T=1 << 30, positions=P, out_strides=(1 << 38, 64)), dict(T=1 << 30, positions=P, q_strides=(1 << 38, 64)),
    dict(T=1 << 20, positions=P, k_strides=(1 << 32, 64)), dict(out_strides=(1 << 39, 64)),
    dict(out_strides=(64, 1 << 39)), dict(hq=1 << 20, out_strides=(1 << 20, 1 << 36))])
def test_head_strides_that_no_memory_has(over):
    assert _forward(over) == (B.ERR_SHAPE, B.ERR_SHAPE)


@far
@pytest.mark.parametrize("over", [dict(T=1 << 20, positions=P, out_strides=(1 << 28, 64)),
                                  dict(q_strides=(1 << 38, 1 << 37), out_strides=(1 << 38, 1 << 30))])
def test_head_strides_that_are_accepted(over):
    assert all(st in (B.ERR_DEVICE, B.ERR_CUDA) for st in _forward(over))


SHIM = """
#include "heads_overlap.h"
extern "C" int meet(const int64_t* a, const int64_t* b)
{
    auto runs = [](const int64_t* v) {
        return nvfp4::Runs(reinterpret_cast<const void*>(v[0]), v[1], v[2], v[3], v[4], v[5]);
    };
    return nvfp4::runs_meet(runs(a), runs(b));
}
"""


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    """meet(a, b) of views (address, heads, tokens, bytes of a head, bytes from head to head, from token to token)."""
    folder = tmp_path_factory.mktemp("overlap")
    (folder / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover=all", "-static-libubsan", "-I",
                    os.path.join(os.path.dirname(B.__file__), "csrc"), "-o", str(folder / "shim.so"),
                    str(folder / "shim.cpp")], check=True)
    f = ctypes.CDLL(str(folder / "shim.so")).meet
    view = ctypes.c_int64 * 6
    return lambda a, b: bool(f(view(*a), view(*b)))


def _bytes(at, heads, tokens, run, head, token):
    return {at + t * token + h * head + i for t in range(tokens) for h in range(heads) for i in range(run)}


def test_views_that_share_a_byte(meet):
    rng = random.Random(0)
    shared = 0
    for _ in range(30000):
        def view(near):
            run, heads, tokens = rng.choice((1, 2, 3, 4, 6)), rng.randint(1, 4), rng.randint(1, 5)
            head = rng.choice((0, run, run, run + 1, 2 * run, rng.randint(0, 40)))
            token = rng.choice((0, heads * head, heads * head + run, rng.randint(0, 40)))
            if rng.random() < 0.3:
                token, head = run, tokens * run + rng.randint(0, 3)
            if near and rng.random() < 0.6:  # as the other one
                heads, tokens, head, token = near[1], near[2], near[4], near[5]
            return (1000 + rng.randint(0, 60), heads, tokens, run, head, token)
        a = view(None)
        b = view(a)
        want = not _bytes(*a).isdisjoint(_bytes(*b))
        shared += want
        assert meet(a, b) == want and meet(b, a) == want, (a, b)
    assert 3000 < shared < 27000


def test_views_as_calls_have_them(meet):
    """Parts of a product's rows, arrays by head, and what would take long to tell."""
    T, D = 1 << 20, 256
    row = 48 * D
    q, k, v = (0, 32, T, D, D, row), (32 * D, 8, T, D, D, row), (40 * D, 8, T, D, D, row)
    for a, b in ((q, k), (q, v), (k, v)):
        assert not meet(a, b) and meet(a, a)
        assert meet(a, (b[0] - 16, *b[1:])) or a is q and b is v
    by_head = (1 << 40, 32, T, D, T * D, D)
    assert not meet(q, by_head) and meet((1 << 40, 1, T, D, 0, D), by_head)
    # every second head, and the others
    assert not meet((0, 16, T, D, 2 * D, row), (D, 16, T, D, 2 * D, row))
    assert meet((0, 16, T, D, 2 * D, row), (16, 16, T, D, 2 * D, row))
    # FP32 results over bf16 values at the same address
    assert meet((0, 32, T, 2 * D, 2 * D, 64 * D), (0, 32, T, D, D, 32 * D))
    # rows of unlike strides that never meet, too many to try: they count as apart
    assert not meet((0, 1, T, 16, 0, 64), (32, 1, T, 16, 0, 128))


def test_ways_of_orthogonalize_refusals():
    f = B.lib().nvfp4_selftest_orthogonalize_ways
    ways = (ctypes.c_int * 3)()
    assert f(1, 4, 4, None) == B.ERR_NULL
    for bad in ((0, 4, 4), (1, 0, 4), (1, 4, (1 << 18) + 1)):
        assert f(*bad, ways) == B.ERR_SHAPE
