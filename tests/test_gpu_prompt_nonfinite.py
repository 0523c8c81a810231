"""GPU checks of mkv_prompt_attention with non-finite values of v whose weight is as good as none."""
import pytest
import torch

from test_gpu_prompt_attention import make, pool_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("hot", [3, 700, 767])
def test_visible_values_without_weight_stay_nonfinite(D, hot, value):
    """Scores up to 2^20 apart: the weight of the key with the non-finite value underflows for most
    rows, or is rescaled to nothing by a later key.  Every row that sees it has an infinity or NaN in
    that channel, near the row's end and far before it; no other element changes."""
    lens = (5, 768)
    q, k, v = make(lens, 2, 1, D, seed=42)
    q[:, :, 0] = 1024.0
    k[:, 0, 0] = 0.0
    k[5:, 0, 0] = torch.arange(768, device="cuda").bfloat16()    # later keys outweigh earlier ones ...
    k[5 + 740:, 0, 0] = -900.0                                   # ... but the last ones weigh nothing themselves
    pool = pool_for(1, D)
    want = pool.prompt_attention(q, k, v, lens, sm_scale=1.0)
    assert bool(torch.isfinite(want).all())
    v[5 + hot, 0, 7] = value
    out = pool.prompt_attention(q, k, v, lens, sm_scale=1.0)
    pool.device_status()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[5 + hot:, :, 7] = True
    assert torch.equal(~torch.isfinite(out), bad)
    assert torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_visible_key_with_score_minus_infinity(D):
    """Its own weight is 0 and 0 times infinity is NaN: its channel is non-finite for every row that
    sees it, the other channels are those of the other keys."""
    lens = (300,)
    q, k, v = make(lens, 2, 1, D, seed=43)
    q[:, :, 0] = 1.0
    pool = pool_for(1, D)
    for hot in (2, 290):
        k2, v2 = k.clone(), v.clone()
        k2[hot, 0, 0] = float("-inf")
        want = pool.prompt_attention(q, k2, v2, lens)
        v2[hot, 0, 9] = float("inf")
        out = pool.prompt_attention(q, k2, v2, lens)
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[hot:, :, 9] = True
        assert torch.equal(~torch.isfinite(out), bad)
        assert torch.equal(out[~bad], want[~bad])
    pool.device_status()
