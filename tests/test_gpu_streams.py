"""GPU checks that what Pool allocates for a call on a given stream comes from that stream's memory: the
outputs, and decode's workspace, which is given back when the call returns and the kernels still run;
and that an output's memory also waits for the current stream that reads it."""
import pytest
import torch

from mixed_format_paged_mkv_b200 import Pool, api

pytestmark = pytest.mark.gpu


def stream_of(address):
    """The stream whose memory pool the address belongs to."""
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= address < s["address"] + s["total_size"])


@pytest.mark.parametrize("given", [False, True])
def test_allocations_belong_to_the_calls_stream(given, monkeypatch):
    s = torch.cuda.Stream()
    want = s.cuda_stream if given else torch.cuda.current_stream().cuda_stream
    kw = dict(stream=s) if given else {}
    pool = Pool(2, 64, 2, 8, 16, 16)
    x = torch.randn((100, 2, 64), device="cuda").to(torch.bfloat16)
    q = torch.randn((100, 4, 64), device="cuda").to(torch.bfloat16)
    pool.append([0], [100], x, x)
    torch.cuda.synchronize()
    seen = []
    lib = api.lib()

    class Watch:
        def __getattr__(self, name):
            fn = getattr(lib, name)
            if name != "mkv_decode_attention":
                return fn
            return lambda *a: (seen.append((stream_of(a[8].value), a[10])), fn(*a))[1]

    monkeypatch.setattr(api, "_lib", Watch())
    outs = [pool.decode([0], q[:1, None], **kw), *pool.materialise(0, **kw),
            pool.prompt_attention(q, x, x, [100], **kw),
            *pool.rope(q, x, torch.arange(100, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda"), **kw)]
    torch.cuda.synchronize()
    assert seen == [(want, want)]
    assert [stream_of(o.data_ptr()) for o in outs] == [want] * len(outs)


@pytest.mark.parametrize("call", ["decode", "materialise", "prompt_attention", "rope"])
def test_an_output_given_up_waits_for_its_reader(call):
    s, pool = torch.cuda.Stream(), Pool(2, 64, 2, 8, 16, 16)
    x = torch.randn((100, 2, 64), device="cuda").to(torch.bfloat16)
    q = torch.randn((100, 4, 64), device="cuda").to(torch.bfloat16)
    pos, inv = torch.arange(100, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    pool.append([0], [100], x, x)
    torch.cuda.synchronize()

    def once():
        if call == "decode":
            return pool.decode([0], q[:1, None], stream=s)
        if call == "materialise":
            return pool.materialise(0, stream=s)[0]
        if call == "prompt_attention":
            return pool.prompt_attention(q, x, x, [100], stream=s)
        return pool.rope(q, x, pos, inv, stream=s)[0]

    out = once()
    s.synchronize()
    want, address = out.cpu(), out.data_ptr()
    torch.cuda._sleep(200_000_000)                  # the reader comes later than the next call
    read = out.clone()
    del out
    again = [once() for _ in range(3)]
    assert address not in [a.data_ptr() for a in again]
    torch.cuda.synchronize()
    assert torch.equal(read.cpu(), want)
