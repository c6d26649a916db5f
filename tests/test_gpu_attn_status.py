"""The status word of the attention calls' workspaces."""
import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("streams", [0, 3])
def test_decode_clears_the_word(streams):
    """Also a call without a sequence, on a workspace that holds anything."""
    q = torch.ones((streams, 2, 64), dtype=torch.float16, device="cuda")
    cache = torch.ones((2, 16, 1, 64), dtype=torch.float16, device="cuda")
    need = rnn._lib.load().rnn_attn_decode_workspace_size(streams, 2, 1, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = rnn.attn_decode(q, cache, cache, ints([[0, 1]] * streams).view(streams, 2),
                          ints([20] * streams), workspace=ws)
    rnn.workspace_status(ws)
    assert (out == 1).all()


@pytest.mark.parametrize("tokens,cu", [(0, [0, 0]), (5, [0]), (5, [0, 5]), (5, [5, 5])])
def test_prompt_clears_the_word(tokens, cu):
    x = torch.ones((tokens, 2, 64), dtype=torch.float16, device="cuda")
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    out = rnn.attn_prompt(x, x, x, ints(cu), out=x.clone(), workspace=ws)
    rnn.workspace_status(ws)
    assert (out == 1).all()
