"""GPU checks of mkv_prompt_attention where a CTA works through many items: more than eight per SM, of
several tokens per tile, with prompts whose last item leaves its second tile empty; and outputs of any 16-byte alignment."""
import pytest
import torch

from test_gpu_prompt_attention import check, make, pool_for, reference

pytestmark = pytest.mark.gpu

SMS = 148
# (their sum, and with it the number of items, is what counts; lengths from one token on, some ending
# just behind a tile's first, a tile's last, an item's last token)
LENS = (2100, 1, 1563, 64, 65, 0, 1299, 32, 33, 1180, 7, 1025, 96, 97, 900, 128, 800, 511, 700, 640, 420, 385, 31, 222)


def items(D, Hq, Hkv):
    unit = 128 // (Hq // Hkv) * (1 if D == 256 else 2)
    return sum(-(-n // unit) for n in LENS) * Hkv


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 32, 8), (64, 24, 8), (128, 40, 8), (256, 24, 4)])
def test_many_items_per_cta(D, Hq, Hkv):
    assert items(D, Hq, Hkv) >= 8 * SMS
    q, k, v = make(LENS, Hq, Hkv, D, seed=31, qs=2.0)
    pool = pool_for(Hkv, D)
    out = pool.prompt_attention(q, k, v, LENS)
    pool.device_status()
    check(out, *reference(q, k, v, LENS, D ** -0.5))
    assert torch.equal(out, pool.prompt_attention(q, k, v, LENS))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 32, 8), (256, 24, 4)])
def test_infinite_values_of_late_items(D, Hq, Hkv):
    """The rows that see a non-finite value, in that channel of its heads, and no other element: the
    flag that asks for a row's repair belongs to one item of the many that a CTA works on."""
    q, k, v = make(LENS, Hq, Hkv, D, seed=32)
    pool = pool_for(Hkv, D)
    want = pool.prompt_attention(q, k, v, LENS)
    first = [sum(LENS[:i]) for i in range(len(LENS))]
    g, bad = Hq // Hkv, torch.zeros_like(want, dtype=torch.bool)
    # (prompt, token, KV head, channel): first, middle and last tokens of long and of the shortest prompts
    for i, t, h, c in ((1, 0, 0, 0), (10, 6, Hkv - 1, D - 1), (7, 31, 1, 5), (22, 3, 2, 9), (0, 2099, 1, 1), (2, 777, 3, 17),
                       (14, 0, 0, 33), (20, 200, 2, 40), (4, 64, 1, 63), (9, 1179, 0, 2)):
        v[first[i] + t, h, c] = float("-inf") if t % 2 else float("inf")
        bad[first[i] + t:first[i] + LENS[i], h * g:(h + 1) * g, c] = True
    out = pool.prompt_attention(q, k, v, LENS)
    pool.device_status()
    assert torch.equal(~torch.isfinite(out), bad)
    assert torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("offset", [8, 16, 24])
def test_outputs_of_any_16_byte_alignment(D, offset):
    lens = (70, 1, 300)
    q, k, v = make(lens, 6, 2, D, seed=41)
    pool, rows = pool_for(2, D), sum(lens)
    want = pool.prompt_attention(q, k, v, lens)
    flat = torch.full((offset + rows * 6 * D + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    assert flat.data_ptr() % 32 == 0
    out = flat[offset:offset + rows * 6 * D].view(rows, 6, D)
    pool.prompt_attention(q, k, v, lens, out=out)
    pool.device_status()
    assert torch.equal(out, want)
    assert bool((flat[:offset] == 3.0).all()) and bool((flat[offset + rows * 6 * D:] == 3.0).all())
