"""The benchmark's DRAM traffic belongs to the kernel source that is there (CPU only)."""
import itertools

import pytest

import bench


@pytest.mark.parametrize("causal,full", list(itertools.product(bench.ALL_SCHEDS, repeat=2)))
def test_every_pair_of_schedules_has_its_traffic(causal, full):
    """Null means that csrc/bwd.cu changed after the captures: capture again (the
    command is in profiles/bwd_main_per_schedule_b1h16s8192d128_b4h16s2048d64.md)."""
    got = bench.traffic_for_current_kernel({"causal": causal, "full": full})
    # at least the inputs and outputs of a launch, 12 bytes an element
    assert got is not None and got > 12 * bench.B * bench.H * bench.S * bench.D / 2
