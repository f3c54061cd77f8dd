"""The committed DRAM captures are of the kernels' present sources: bench.py reports a traffic only
then, and would leave it out without a word."""
import pytest


@pytest.mark.parametrize("source,summary,algorithmic", [("combine.cu", "combine_dsv3_prefill.md", 4.230e9),
                                                        ("dispatch.cu", "scatter_dsv3_prefill.md", 2.412e9)])
def test_a_capture_of_the_present_source(source, summary, algorithmic):
    import bench
    traffic = bench.profile_traffic(source, summary)
    assert traffic is not None, f"{source} changed: take the DRAM capture of profiles/{summary} again"
    assert 0.8 * algorithmic < traffic < 1.1 * algorithmic
