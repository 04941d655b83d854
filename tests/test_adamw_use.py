"""LoraAdamW as a program holds it: what it may be made from, and when."""
import pytest
import torch

import rank_gemm_lora_amd as rg
from tests.test_adamw import DEV, say


@pytest.mark.gpu
def test_an_optimizer_is_not_made_during_a_capture():
    """Made during one, its zero moments, its masters and its table would be work of the graph: every replay would
    start it anew. The refused call leaves the capture usable."""
    say("adamw made during a capture")
    p, g = torch.ones(300, device=DEV), torch.ones(300, device=DEV)
    other = torch.zeros(1, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captur"):
            rg.LoraAdamW([p], [g])
        other += 1
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert float(other) == 3 and bool((p == 1).all())
