"""Passes whose work items hold a single streamed tile: few positions over a large
table (item-owned pass) and a table of few tiles over several position tiles
(position-owned pass), with more work items than SMs."""
import pytest

from vocabulary_label_bce_b200 import workloads as W

from gpu_util import check_against_oracle, run_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,D", [(64, 40000, 64), (128, 25000, 128), (60, 30000, 256), (513, 5000, 64), (600, 8000, 64)])
def test_one_tile_per_work_item(T, V, D):
    p = W.draw(T=T, V=V, D=D, K=4, dtype="bf16", seed=3, ids="zipf", zipf_s=1.1, mask="none")
    for _ in range(3):
        check_against_oracle(p, run_gpu(p, "mean"), "mean")
