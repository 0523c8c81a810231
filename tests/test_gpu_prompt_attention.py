"""GPU checks of mkv_prompt_attention against the formula in float64.

Tolerance, element by element.  With A = softmax(scores) . |V| (so |out| <= A):
  * the result is rounded to bf16: 2^-8 |out|;
  * each probability is rounded to bf16 before it multiplies V: 2^-8 A;
  * a score sums D products in fp32, each step off by at most 2^-23 of the magnitudes summed (a
    tensor core may truncate): E = D 2^-23 scale max(sum |q k|); the exponent's products and the
    2^x function add less than 8 2^-23 (max |scaled score| + 1).  Both act on numerator and
    denominator: 2 (E + ...) A;
  * the sums over n keys of probabilities and of products: 2 n 2^-23 A.
"""
import numpy as np
import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool

pytestmark = pytest.mark.gpu


def make(lens, Hq, Hkv, D, seed=0, extra=0, qs=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens) + extra
    def draw(h, s=1.0):
        return (torch.randn((n, h, D), generator=g, device="cuda") * s).to(torch.bfloat16)
    return draw(Hq, qs), draw(Hkv), draw(Hkv)


def pool_for(Hkv, D):
    return Pool(Hkv, D, 1, 1, 1, 1)


def reference(q, k, v, lens, scale):
    """(out, tolerance) in float64."""
    T, Hq, D = sum(lens), q.shape[1], q.shape[2]
    g = Hq // k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    a = 0
    for n in lens:
        for h in range(Hq if n else 0):
            Q, K, V = (x[a:a + n].double() for x in (q[:, h], k[:, h // g], v[:, h // g]))
            s = Q @ K.t() * scale
            mask = torch.ones_like(s, dtype=torch.bool).triu(1)
            E = D * 2.0 ** -23 * scale * (Q.abs() @ K.abs().t()).masked_fill(mask, 0).max()
            E += 8 * 2.0 ** -23 * (s.masked_fill(mask, 0).abs().max() * 1.4427 + 1)
            w = torch.softmax(s.masked_fill(mask, float("-inf")), -1)
            o, A = w @ V, w @ V.abs()
            out[a:a + n, h] = o
            tol[a:a + n, h] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * E + 2 * n * 2.0 ** -23) * 1.01 * A
        a += n
    return out, tol


def check(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), float((err / tol).nan_to_num(9e9).max()))


LENS = [(1,), (2, 1), (16,), (37,), (64,), (127, 129), (128,), (256, 1, 0, 255), (257,), (0, 300, 5), (513, 640),
        (1000, 3, 700)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(D, lens):
    q, k, v = make(lens, 4, 2, D, seed=sum(lens))
    pool = pool_for(2, D)
    out = pool.prompt_attention(q, k, v, lens)
    pool.device_status()
    check(out, *reference(q, k, v, lens, D ** -0.5))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 1), (6, 2), (7, 1), (8, 1), (16, 1), (48, 1), (65, 1), (128, 1),
                                    (4, 4), (24, 4)])
def test_head_groups(D, Hq, Hkv):
    lens = (150, 1, 290)
    q, k, v = make(lens, Hq, Hkv, D, seed=Hq)
    pool = pool_for(Hkv, D)
    out = pool.prompt_attention(q, k, v, lens)
    pool.device_status()
    check(out, *reference(q, k, v, lens, D ** -0.5))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prompt_and_large_scores(D):
    """Scores that keep climbing move the reference and rescale the output many times."""
    lens = (2300, 4100)
    q, k, v = make(lens, 2, 1, D, seed=3, qs=8.0)
    ramp = torch.linspace(0.05, 3, sum(lens), device="cuda")[:, None, None]
    k = (k.float() * ramp).to(torch.bfloat16)
    pool = pool_for(1, D)
    out = pool.prompt_attention(q, k, v, lens)
    pool.device_status()
    check(out, *reference(q, k, v, lens, D ** -0.5))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_strided_rows_of_a_fused_projection(D):
    """q, k and v as parts of one [rows, (Hq + 2 Hkv) D] tensor, at offsets within each row."""
    lens, Hq, Hkv = (70, 200, 33), 6, 2
    q, k, v = make(lens, Hq, Hkv, D, seed=5)
    rows = sum(lens)
    fused = torch.full((rows + 3, (Hq + 2 * Hkv) * D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    a, b = Hq * D + 8, (Hq + Hkv) * D + 16
    parts = [fused[:, o:o + h * D].unflatten(1, (h, D)) for o, h in ((0, Hq), (a, Hkv), (b, Hkv))]
    for part, x in zip(parts, (q, k, v)):
        part[:rows] = x
    pool = pool_for(Hkv, D)
    out = torch.full((rows + 3, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = pool.prompt_attention(*parts, lens, out=out)
    pool.device_status()
    assert got is out and (out[rows:] == 7.0).all()      # rows behind the last prompt stay
    check(out[:rows], *reference(q, k, v, lens, D ** -0.5))
    assert torch.equal(out[:rows], pool.prompt_attention(q, k, v, lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq", [1, 3, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 3.3e38])
def test_masked_values_never_reach_an_output(D, Hq, value):
    """Tokens that a row does not see may hold anything: the rows before them keep the outputs
    that finite values there give, bit for bit; the prompts before and after are untouched."""
    lens, hot = (90, 300, 41), (13, 127, 128, 200, 299)
    q, k, v = make(lens, Hq, 1, D, seed=11)
    pool = pool_for(1, D)
    want = pool.prompt_attention(q, k, v, lens)
    for t in hot:
        k2, v2 = k.clone(), v.clone()
        v2[90 + t, 0, ::7] = value
        k2[90 + t, 0, 5] = value
        out = pool.prompt_attention(q, k2, v2, lens)
        assert torch.equal(out[:90 + t], want[:90 + t]), t
        assert torch.equal(out[390:], want[390:]), t
    pool.device_status()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_visible_nonfinite_values_propagate(D, value):
    lens = (5, 260)
    q, k, v = make(lens, 4, 2, D, seed=12)
    v[5 + 130, 1, 3] = value
    v[5 + 7, 0, D - 1] = value
    pool = pool_for(2, D)
    out = pool.prompt_attention(q, k, v, lens).float()
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[5 + 130:, 2:, 3] = True
    want[5 + 7:, :2, D - 1] = True
    assert torch.equal(bad, want)
    if value == value:  # an infinity keeps its sign where it has been seen in the same pass
        assert (out[5 + 130:, 2:, 3] == value).all()
    v[5 + 131, 1, 3] = -value
    out = pool.prompt_attention(q, k, v, lens).float()
    assert torch.isnan(out[5 + 131:, 2:, 3]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_and_infinite_scores(D):
    lens = (33, 200)
    q, k, v = make(lens, 3, 1, D, seed=13)
    pool = pool_for(1, D)
    check(pool.prompt_attention(q, k, v, lens, sm_scale=0.0), *reference(q, k, v, lens, 0.0))
    check(pool.prompt_attention(q, k, v, lens, sm_scale=1.7), *reference(q, k, v, lens, 1.7))
    # a first key whose score is -inf: later keys decide, the first row has no weight at all
    k2 = k.clone()
    k2[33, 0, 0] = float("-inf")
    q2 = q.clone()
    q2[33:, :, 0] = 1.0
    out = pool.prompt_attention(q2, k2, v, lens)
    assert torch.isnan(out[33]).all()
    want, tol = reference(q2, k2.clamp(min=-1e30), v, lens, D ** -0.5)
    check(out[34:], want[34:], torch.full_like(want[34:], 2.0 ** -7 * float(v.abs().max()) * 1.1))


def test_many_prompts_span_launches():
    """More prompts than one launch holds."""
    lens = [1 + i % 3 for i in range(2500)] + [0, 0, 5]
    q, k, v = make(lens, 2, 1, 64, seed=14)
    pool = pool_for(1, 64)
    n0 = pool.launch_count()
    out = pool.prompt_attention(q, k, v, lens)
    assert pool.launch_count() - n0 == -(-2501 // 128)
    assert torch.equal(pool.prompt_attention(q[:6], k[:6], v[:6], (1, 2, 3)), out[:6])
    check(out[-5:], *reference(q[-5:], k[-5:], v[-5:], (5,), 64 ** -0.5))


def test_nothing_to_do_and_repeat_is_bitwise_equal():
    pool = pool_for(2, 128)
    q, k, v = make((400, 77), 8, 2, 128, seed=15)
    out = torch.full_like(q, 3.0)
    pool.prompt_attention(q, k, v, (), out=out)
    pool.prompt_attention(q, k, v, (0, 0), out=out)
    assert (out == 3.0).all()
    a = pool.prompt_attention(q, k, v, (400, 77))
    for _ in range(5):
        assert torch.equal(a, pool.prompt_attention(q, k, v, (400, 77)))


@pytest.mark.parametrize("D", [128, 256])
def test_captured_and_overlapping_calls(D):
    """A captured call replayed on new inputs, and calls on two streams at once."""
    lens = (300, 50)
    a, b = make(lens, 4, 2, D, seed=16), make(lens, 4, 2, D, seed=17)
    pool = pool_for(2, D)
    wa, wb = (pool.prompt_attention(*x, lens) for x in (a, b))
    static = [x.clone() for x in a]
    out = torch.zeros_like(wa)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        pool.prompt_attention(*static, lens, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, wa)
    for x, y in zip(static, b):
        x.copy_(y)
    torch.cuda.synchronize()
    graph.replay()
    outs = []
    for i in range(20):
        outs.append(pool.prompt_attention(*(a if i % 2 else b), lens, stream=s1 if i % 3 else s2))
    torch.cuda.synchronize()
    assert torch.equal(out, wb)
    for i, o in enumerate(outs):
        assert torch.equal(o, wa if i % 2 else wb), i
    pool.device_status()


def test_more_than_2_to_the_31_elements():
    """q and out hold 2.3e9 elements: the last prompts come out as in a call of their own."""
    Hq, D, n = 128, 256, 700
    lens = [100] * n + [33]
    rows = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(21)
    q = torch.empty((rows, Hq, D), dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, 10000):
        q[a:a + 10000] = torch.randn(q[a:a + 10000].shape, generator=g, device="cuda")
    k, v = (torch.randn((rows, 1, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pool = pool_for(1, D)
    out = pool.prompt_attention(q, k, v, np.array(lens))
    assert out.numel() > 2 ** 31
    tail = 3 * 100 + 33
    assert torch.equal(out[-tail:], pool.prompt_attention(q[-tail:], k[-tail:], v[-tail:], (100, 100, 100, 33)))
    assert torch.equal(out[:100], pool.prompt_attention(q[:100], k[:100], v[:100], (100,)))
    check(out[-33:, :4], *reference(q[-33:, :4], k[-33:], v[-33:], (33,), D ** -0.5))
    pool.device_status()


def test_largest_and_smallest_scales():
    """The limits of the softmax: the largest scale leaves each row its last key alone (its
    probability and the result are rounded to bf16: 2 2^-8), a denormal one weighs all alike."""
    q, k, v = make((40,), 1, 1, 64, seed=22)
    q = q.abs() + 0.5
    k[:, 0] = torch.arange(1, 41, device="cuda")[:, None].to(torch.bfloat16)   # the last key wins
    pool = pool_for(1, 64)
    out = pool.prompt_attention(q, k, v, (40,), sm_scale=65536.0).double()
    assert bool(((out - v.double()).abs() <= 2.0 ** -7 * v.double().abs()).all())
    check(pool.prompt_attention(q, k, v, (40,), sm_scale=1e-44), *reference(q, k, v, (40,), 0.0))
    pool.device_status()


def test_large_scores_keep_the_weights_of_moved_references():
    """Scaled scores near 3000 whose maximum rises with every key tile: the rounding of a reference is
    2^-24 of it and must not come between tiles."""
    n, D = 512, 128
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(q), make((n,), 1, 1, D, seed=23)[2]
    q[:, 0, 0], q[:, 0, 1] = 1.0, 1.0
    k[:, 0, 0] = 3008.0                                              # the same for all keys
    k[:, 0, 1] = (torch.arange(n, device="cuda") // 64 * 8).to(torch.bfloat16)   # + 8 (11.5 in log2) a tile
    pool = pool_for(1, D)
    check(pool.prompt_attention(q, k, v, (n,), sm_scale=1.0), *reference(q, k, v, (n,), 1.0))
    k[:, 0, 1] = (torch.arange(n, device="cuda") // 64 * 6).to(torch.bfloat16)   # + 6 (8.7): weights 1/403
    check(pool.prompt_attention(q, k, v, (n,), sm_scale=1.0), *reference(q, k, v, (n,), 1.0))
    pool.device_status()
