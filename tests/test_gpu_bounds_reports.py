"""The debug build's reports of calls that were made without a status word."""
import pytest
import torch

from nvfp4_testlib import need_gpu

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

pytestmark = pytest.mark.gpu


def test_a_refused_access_without_a_status_word_ends_the_block_with_an_error():
    need_gpu()
    with pytest.raises(B.NVFP4Error, match="outside its buffer"):
        with B.bounds_checked():
            B.selftest_bounds(None)
    with B.bounds_checked():  # the report is not left behind
        B.route(torch.zeros(3, 4, device="cuda"), 2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with B.bounds_checked():  # a call with a word of its own reports there only
        B.selftest_bounds(st)
        torch.cuda.synchronize()
    assert int(st) == B.DEVSTAT_BOUNDS
    assert not B.is_bounds_checked()


def test_other_errors_of_the_block_come_first_and_other_bits_do_not_raise():
    need_gpu()
    with pytest.raises(KeyError):
        with B.bounds_checked():
            B.selftest_bounds(None)
            raise KeyError("the caller's")
    with B.bounds_checked():  # the next block does not answer for that one
        B.route(torch.zeros(3, 4, device="cuda"), 2)
    with B.bounds_checked():
        e, w = B.route(torch.full((3, 4), float("nan"), device="cuda"), 2)
    assert (e == -1).all()


def test_a_report_made_while_capturing_is_seen_after_the_replay():
    need_gpu()
    x = torch.zeros(3, 4, device="cuda")
    with pytest.raises(B.NVFP4Error, match="outside its buffer"):
        with B.bounds_checked():
            B.route(x, 2)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                B.selftest_bounds(None)
            graph.replay()


def test_a_block_may_lie_inside_a_capture():
    need_gpu()
    x = torch.randn(3, 4, device="cuda")
    with B.bounds_checked():
        ref = B.route(x, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with B.bounds_checked():
            got = B.route(x, 2)
    graph.replay()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    with pytest.raises(B.NVFP4Error, match="outside its buffer"):
        with B.bounds_checked():
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                with B.bounds_checked():
                    B.selftest_bounds(None)
            graph.replay()
