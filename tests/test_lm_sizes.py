"""Host-side checks (no GPU) of the workspace queries from Python."""
import pytest
import torch

import selective_state_space_85_amd as ss

QUERIES = (ss.glu_workspace_bytes, ss.glu_bwd_workspace_bytes, ss.xent_workspace_bytes, ss.xent_bwd_workspace_bytes)


@pytest.mark.parametrize("query", QUERIES, ids=lambda q: q.__name__)
def test_types_and_sizes(query):
    assert query(100, 63, 96, torch.bfloat16) > 0 and query(100, 63, 96, torch.float32) >= 0
    with pytest.raises(TypeError):
        query(100, 63, 96, torch.float16)
    with pytest.raises(ValueError):
        query(100, 0, 96, torch.float32)
