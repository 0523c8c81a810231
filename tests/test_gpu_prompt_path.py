"""The operators of a prompt's path together, as a program uses them: rotary positions, prompt
attention, the prefill write, branches of the cached prompts, decode steps on them (each rotated,
appended and attended), rollback, release and compaction -- against the oracle's pool and float64
attention at every step."""
import numpy as np
import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool
from oracle import attention as A
from oracle import formats as F
from oracle import pool as P

from harness import assert_close
from test_gpu_pages import compare_pages
from test_gpu_prompt_attention import check as check_attention
from test_gpu_prompt_attention import reference as attention_reference
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu


def f64(t):
    return F.bf16_bits_to_f64(t.cpu().view(torch.int16).numpy().view(np.uint16))


@pytest.mark.parametrize("D,Hq,Hkv,axes", [(64, 4, 4, 1), (128, 8, 2, 3), (256, 12, 2, 2)])
def test_prompt_path(D, Hq, Hkv, axes):
    g = torch.Generator(device="cuda").manual_seed(D)
    lens, window = (333, 1, 150), 48
    shape = (Hkv, D, 12, 40, 120, 120)
    lp, op = Pool(*shape), P.RefPool(*shape)
    inv = torch.tensor([10000.0 ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float32, device="cuda")
    axis = [i * axes // (D // 2) for i in range(D // 2)]

    def draw(rows):
        q, k, v = (torch.randn((rows, h, D), generator=g, device="cuda").to(torch.bfloat16)
                   for h in (Hq, Hkv, Hkv))
        return q, k, v

    def rotated(q, k, pos):
        qr, kr = lp.rope(q, k, pos, inv, axes=axis)
        check_rope(qr, q, pos, inv, axis, False)
        check_rope(kr, k, pos, inv, axis, False)
        return qr, kr

    # ---- the prompts: rotate, attend, write
    q, k, v = draw(sum(lens))
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    pos = torch.stack([pos // (i + 1) for i in range(axes)]).contiguous()
    q, k = rotated(q, k, pos)
    out = lp.prompt_attention(q, k, v, lens)
    check_attention(out, *attention_reference(q, k, v, lens, D ** -0.5))
    lp.prefill([0, 1, 2], lens, k, v, window=window)
    op.prefill([0, 1, 2], lens, f64(k), f64(v), window)

    # ---- branches, a few decode steps on them, rollback
    src, dst, at = [0, 0, 2, 1], [3, 4, 5, 6], [333, 320, 149, 1]
    lp.fork(src, dst, at)
    op.fork(src, dst, at)
    compare_pages(lp, op, range(12))
    live = [3, 4, 5, 6, 0]
    for step in range(6):
        q, k, v = draw(len(live))
        ctx = torch.tensor([op.ctx[s] for s in live], dtype=torch.int32, device="cuda")
        q, k = rotated(q, k, torch.stack([ctx // (i + 1) for i in range(axes)]).contiguous())
        ones = [1] * len(live)
        lp.append(live, ones, k, v)
        op.append(live, ones, f64(k), f64(v))
        assert lp.demote(live, window) == len(op.demote(live, window))
        got = lp.decode(live, q.unsqueeze(1)).cpu().numpy()
        qd = f64(q)
        for i, s in enumerate(live):
            K, V = op.dequant_seq(s)
            assert_close(got[i], A.attention(K, V, qd[i:i + 1], D ** -0.5), what=f"step {step} seq {s}")
        if step == 2:
            cut = [op.ctx[s] - c for s, c in zip((3, 5, 6), (2, 3, 1))]
            lp.truncate([3, 5, 6], cut)
            op.truncate([3, 5, 6], cut)
        if step == 3:
            lp.free([0, 2])
            op.free([0, 2])
            live.remove(0)
            assert lp.compact() == op.compact()
        compare_pages(lp, op, range(12))
    lp.device_status()
