"""The committed traffic profile is that of the present kernel sources (CPU), so
that the benchmark reports its figure.  After a change to them: profile again,
or, where the assembly of the GEMM's kernels is the same instruction for
instruction, say so in the profile beside the new hash."""
import bench


def test_the_benchmark_has_its_traffic_figure():
    assert bench.measured_traffic() == 1885745164
