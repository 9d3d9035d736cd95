"""Calls with stream= on a stream that is not ordered after the current one:
what queued work of the current stream still reads is not overwritten, before
the call or after its results are freed."""
import pytest

import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"


def dev16(a):
    return torch.from_numpy(a.view("int16")).to(DEV)


W = dev16(synth.random_bits(1024 * 4096, 3).reshape(1024, 4096))
X = dev16(synth.vectors(3, 256, 4096))
Q = wc.fp4_encode(W)
STACK = [wc.fp4_encode(dev16(synth.random_bits(8 * r * c, 4 + r).reshape(8, r, c)))
         for r, c in ((512, 1024), (1024, 256))]
TOKENS, ROUTER = dev16(synth.vectors(5, 64, 1024)), dev16(synth.vectors(6, 8, 1024))
HEAD, CODED = wc.encode(W, wc.BYTESPLIT)
CALLS = {
    "fp4_encode": lambda s: list(wc.fp4_encode(W, stream=s)[:2]),
    "fp4_decode": lambda s: [wc.fp4_decode(Q, stream=s)],
    "fp4_gemv": lambda s: [wc.fp4_gemv(Q, X, stream=s)],
    "moe": lambda s: list(wc.moe(TOKENS, ROUTER, *STACK, 2, stream=s)),
    "encode": lambda s: [wc.encode(W, wc.BYTESPLIT, stream=s)[1]],
    "decode": lambda s: [wc.decode(HEAD, CODED, stream=s)],
    "decode_gemv": lambda s: [wc.decode_gemv(HEAD, CODED, 1024, 4096, X, stream=s)],
    "gemv_bf16": lambda s: [wc.gemv_bf16(W, X, stream=s)],
}


def busy():
    """Work that keeps the current stream busy for some 10 ms."""
    a = torch.ones(4096, 4096, device=DEV)
    for _ in range(8):
        a = a @ a * 2.0 ** -12
    return a


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_the_current_stream_reads_stays(name):
    call = CALLS[name]
    ref = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    busy()
    call(side)  # both streams' pools are warm
    torch.cuda.synchronize()
    # memory of the outputs' sizes is read late on the current stream, and freed now
    held = [torch.full_like(t, 3) for t in ref]
    at = [h.data_ptr() for h in held]
    busy()
    late = [h.clone() for h in held]
    del held
    got = call(side)
    assert not {t.data_ptr() for t in got} & set(at)
    # and the outputs themselves: read late, freed, and asked for again
    torch.cuda.current_stream().wait_stream(side)
    busy()
    read = [t.clone() for t in got]
    del got
    again = call(side)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in late)
    assert all(torch.equal(a, b) for a, b in zip(read, ref))
    assert all(torch.equal(a, b) for a, b in zip(again, ref))


@pytest.mark.parametrize("name", ["fp4_decode", "fp4_encode", "fp4_gemv", "moe", "decode", "decode_gemv", "gemv_bf16"])
def test_on_a_joined_stream_of_a_graph(name):
    """A captured call on another stream, joined to the captured one: replays
    give the eager bits, with eager calls on that stream in between."""
    call, side = CALLS[name], torch.cuda.Stream()
    ref = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        for t in got:
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        other = call(side)
        torch.cuda.current_stream().wait_stream(side)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(other, ref))


def test_a_stream_that_is_a_handle_alone():
    class Handle:
        cuda_stream = torch.cuda.Stream().cuda_stream

    torch.cuda.synchronize()
    for name, call in CALLS.items():
        got = call(Handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, call(None))), name
