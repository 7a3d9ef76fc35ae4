"""The conveniences that allocate, on a stream that is not the current one: the memory that they
drop on return is not given out on the current stream while their kernels still use it."""
import pytest
import torch

from parity_utils import DEV

pytestmark = pytest.mark.gpu

FILL = 7


def attention(lib):
    """A list that is cut between blocks: parts go through the workspace."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    k, v = torch.randn(2, 200, 64, 4, 128, device=DEV, generator=gen).to(torch.bfloat16)
    q = torch.randn(1, 32, 128, device=DEV, generator=gen).to(torch.bfloat16)
    table = torch.arange(200, dtype=torch.int32, device=DEV).view(1, 200)
    lens = torch.full((1,), 12777, dtype=torch.int32, device=DEV)
    cache = lib.PagedCache(k, v)
    torch.cuda.synchronize()
    size = lib.kda_paged_decode_workspace_size(1, 32, 4, 128)
    return size, lambda s: lib.paged_decode(q, cache, table, lens, 128 ** -0.5, want_lse=True, stream=s)


def plan(lib):
    lens = torch.full((1000,), 20, dtype=torch.int32, device=DEV)
    zero = torch.zeros_like(lens)
    free = torch.arange(2000, dtype=torch.int32, device=DEV)
    table = torch.full((1000, 2), -1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    return 80000, lambda s: lib.page_plan(zero, lens, free, table, 16, 2000, 20000, stream=s)


def prefill(lib):
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, g = torch.randn(4, 512, 4, 128, device=DEV, generator=gen)
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    beta = torch.rand(512, 4, device=DEV, generator=gen)
    args = [x.to(torch.bfloat16) for x in (q, k, v)] + [-0.1 * g.abs(), beta]
    torch.cuda.synchronize()
    size = lib.kda_chunk_prefill_workspace_size(512, 1, 4)
    return size, lambda s: lib.prefill(*args, stream=s)


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("case", [attention, plan, prefill])
def test_dropped_memory_stays_with_its_stream(lib, case, as_handle):
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    size, call = case(lib)
    want = [None if x is None else x.clone() for x in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)              # a tenth of a second: the call stays pending
    got = call(stream)
    place = side if not as_handle else torch.cuda.ExternalStream(stream)
    taken = [torch.full((n,), FILL, dtype=torch.uint8, device=DEV) for n in [max(size, 16)] * 3]
    torch.cuda.synchronize()
    for t in taken:
        assert bool((t == FILL).all())
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        assert a is None or torch.equal(a, b)
    # the other way: what the current stream frees is not taken for the call while still in use
    spare = [torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for t in spare:
        t.fill_(FILL)                               # pending on the current stream
    del spare, t
    got = call(stream)
    place.synchronize()                             # the fills may come after the call
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert a is None or torch.equal(a, b)


def test_handle_of_the_default_stream(lib):
    size, call = prefill(lib)
    want = [x.clone() for x in call(None)]
    got = call(torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
