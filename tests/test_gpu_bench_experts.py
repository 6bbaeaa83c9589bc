"""The benchmark's mixture-of-experts step at a small size: it runs clean and reproducibly, and every
operator is timed."""
import pytest
import torch

import synth
from nvfp4_testlib import need_gpu

pytest.importorskip("nvfp4_bit_quantized_03_b200")
import bench  # noqa: E402

pytestmark = pytest.mark.gpu


def test_experts_step_runs_and_is_timed():
    need_gpu()
    wl = synth.ExpertsLayer("small", 3, 200, 256, 384, 6, 2)
    step = bench.ExpertsStep(wl, torch.device("cuda"))
    first = step.run()
    step.events = []
    again = step.run()
    torch.cuda.synchronize()
    assert int(step.dev_status) == 0
    assert [n for n, _, _ in step.events] == [
        "route", "plan", "up fprop", "down fprop", "combine", "combine backward", "down dgrad",
        "down wgrad", "up dgrad", "up wgrad", "gather backward", "route backward"]
    for name in first:
        assert torch.equal(first[name], again[name]), name
        assert torch.isfinite(first[name].float()).all(), name
    assert first["dw1"].shape == (6 * 384, 256) and first["dw2"].shape == (6 * 256, 384)
