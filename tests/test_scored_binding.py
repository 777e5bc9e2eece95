"""Host-side refusals of the binding of the calls with scores, without a GPU."""
import pytest
import torch

from test_kv_abi import spv  # noqa: F401  (a fixture)


@pytest.mark.parametrize("scores", [None, 30.0, {"cap": 30.0}])
def test_scores_have_to_be_scores(spv, scores):  # noqa: F811
    x, i = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    cache, q = spv.KVCache(x, x), torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    calls = [lambda: spv.spv_paged_attention_scored(q, cache, i[None], i, scores),
             lambda: spv.spv_attention_mass_scored(q, torch.zeros(1, 1, 4), cache, i[None], i, i, scores)]
    if scores is not None:
        calls.append(lambda: spv.spv_prompt_attention(q, cache, i[None], i, scores))
    for call in calls:
        with pytest.raises(ValueError, match="scores must be"):
            call()
