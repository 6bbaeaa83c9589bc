"""Every way to spread a product of the orthogonalisation (tiles by pairs, by single CTAs, by clusters) with every
way to store its result, on gradients of every kind, against the steps in 64 bits; every test through both
libraries."""
import pytest
import torch

from nvfp4_testlib import need_gpu
from test_gpu_orthogonalize import _check, _gradient

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["release", "checked"], autouse=True)
def _library(request):
    need_gpu()
    if request.param == "release":
        yield
    else:
        with B.bounds_checked():
            yield


# batch, rows, cols of X (a fresh output is written by tensor copies or 16 bytes at a time where its columns are a
# multiple of 8, otherwise value by value; that of a G with more rows than columns is written turned).  How many
# clusters of 4 a GPU holds at once differs between GPUs; none of these sizes is near the number.
CASES = [(1, 800, 1104), (1, 801, 1101), (2, 96, 160), (1, 300, 1000), (1, 304, 1001), (1, 264, 304), (1, 257, 303),
         (1, 640, 2048), (1, 636, 2047), (3, 904, 1000), (1, 2304, 2312), (1, 2300, 2301)]
CASES = [(b, *size) for b, rows, cols in CASES for size in ((rows, cols), (cols, rows))]


def test_the_cases_reach_every_kernel_and_store():
    reached = set()
    for batch, rows, cols in CASES:
        gram, square, update = B.selftest_orthogonalize_ways(batch, rows, cols)
        reached |= {("gram", gram), ("square", square), ("update", update),
                    ("last", update, "turned" if rows > cols else "straight", "whole" if cols % 8 == 0 else "by value")}
    ways = (1, 2, 4, 128, 256)
    wanted = {(p, w) for p in ("gram", "square", "update") for w in ways} | {
        ("last", w, t, s) for w in ways for t in ("turned", "straight") for s in ("whole", "by value")}
    assert reached == wanted, sorted(map(str, wanted ^ reached))


@pytest.mark.parametrize("batch,rows,cols", CASES)
def test_every_way(batch, rows, cols):
    g = _gradient((batch, rows, cols), seed=rows)
    g = g[0] if batch == 1 else g
    _check(B.orthogonalize(g), g, (batch, rows, cols))


def _kind(kind, shape):
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    batch, rows, cols = shape
    g = randn(*shape)
    if kind == "low rank":
        return randn(batch, rows, 8) @ randn(batch, 8, cols) + 1e-2 * g
    if kind == "rows":
        return g * torch.logspace(-2, 0, rows, device="cuda")[:, None]
    if kind == "columns":
        return g * torch.logspace(-2, 0, cols, device="cuda")
    if kind == "one row":
        g[:, 1:] = 0
        return g
    if kind == "orthogonal":
        q = torch.linalg.qr(g.mT if rows < cols else g)[0]
        return (q.mT if rows < cols else q).contiguous()
    if kind == "rank one":
        return randn(batch, rows, 1) @ randn(batch, 1, cols)
    if kind == "few nonzero":
        return g * (torch.rand(shape, generator=gen, device="cuda") < 0.01)
    # singular values that fall off over four decades
    u, v = (torch.linalg.qr(randn(batch, n, min(rows, cols)))[0] for n in (rows, cols))
    return (u * torch.logspace(0, -4, min(rows, cols), device="cuda")) @ v.mT


# the kinds on every kernel: clusters of 2 and single narrow tiles, single CTAs for update, single CTAs and pairs, pairs
@pytest.mark.parametrize("batch,rows,cols", [(1, 800, 1104), (1, 636, 2047), (3, 904, 1000), (1, 2304, 2312),
                                             (1, 2301, 2300)])
@pytest.mark.parametrize("kind", ["low rank", "rows", "columns", "one row", "orthogonal", "rank one", "few nonzero",
                                  "falling off"])
def test_kinds_of_gradients(kind, batch, rows, cols):
    g = _kind(kind, (batch, rows, cols))
    _check(B.orthogonalize(g), g, (kind, batch, rows, cols))


@pytest.mark.parametrize("batch,rows,cols", [(1, 640, 2047), (2, 904, 1001), (1, 2047, 300), (1, 2301, 2300)])
def test_what_the_workspace_and_its_surroundings_hold(batch, rows, cols):
    need = B.lib().nvfp4_orthogonalize_workspace_bytes(batch, rows, cols)
    room = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    g = _gradient((batch, rows, cols))
    want = B.orthogonalize(g)
    for fill in (0xFF, 0, 0x7C):
        room.fill_(fill)
        assert torch.equal(B.orthogonalize(g, workspace=room[256:256 + need]), want)
        assert (room[:256] == fill).all() and (room[256 + need:] == fill).all()
    # parts of a larger matrix, on 16 bytes and off them
    for first in (8, 3):
        buf = torch.full((batch, rows + 2, -(-(cols + 16) // 8) * 8), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, 1:-1, first:first + cols]
        B.orthogonalize(g, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert (buf == 7.0).all()
