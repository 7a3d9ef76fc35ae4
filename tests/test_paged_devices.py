"""Tensors that are not on the cache's GPU are refused before their addresses go to a kernel,
whether or not a stream is given (CPU: host tensors that say they are on a GPU, and a stand-in
for the library)."""
import pytest
import torch

import gated_delta_rule_33_gb300 as kda

I32 = dict(dtype=torch.int32)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU `index`; its memory is never reached."""
    index = 0

    def get_device(self):
        return self.index


def on_gpu(t, index=0):
    out = t.as_subclass(OnGpu)
    out.index = index
    return out


@pytest.fixture(autouse=True)
def reached(monkeypatch):
    """Stands for the library: notes the calls that pass the binding's checks."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0
    monkeypatch.setattr(kda.kda, "_lib", Lib())
    return calls


def cache():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    return kda.PagedCache(on_gpu(k), on_gpu(k.clone()))


def append_args():
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    return [x, x.clone(), torch.zeros(5, **I32)]


def decode_args():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    return [q, torch.zeros(3, 2, **I32), torch.zeros(3, **I32), q.clone(), torch.zeros(3, 4),
            torch.zeros(1 << 16, dtype=torch.uint8)]


def plan_args():
    return [torch.zeros(3, **I32), torch.zeros(3, **I32), torch.zeros(8, **I32),
            torch.zeros(3, 4, **I32), torch.zeros(3, **I32), torch.zeros(4, **I32),
            torch.zeros(9, **I32), torch.zeros(1, **I32)]


def append(c, a, stream):
    kda.kda_paged_append(*a, c, stream=stream)


def decode(c, a, stream):
    kda.kda_paged_decode(a[0], c, a[1], a[2], 0.1, a[3], a[4], a[5], stream=stream)


def plan(c, a, stream):
    kda.kda_page_plan(*a[:4], 16, 4, *a[4:], stream=stream)


@pytest.mark.parametrize("stream", [0, 77])
@pytest.mark.parametrize("call,args", [(append, append_args), (decode, decode_args), (plan, plan_args)])
def test_every_tensor_is_checked(call, args, stream, reached):
    call(cache(), [on_gpu(t) for t in args()], stream)
    assert len(reached) == 1
    for i in range(len(args())):
        for elsewhere in (lambda t: t, lambda t: on_gpu(t, 1)):      # on the host, on another GPU
            a = [elsewhere(t) if j == i else on_gpu(t) for j, t in enumerate(args())]
            with pytest.raises(ValueError):
                call(cache(), a, stream)
    assert len(reached) == 1


def test_a_cache_on_the_host(reached):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = kda.PagedCache(k, k.clone())
    for call, args in ((append, append_args), (decode, decode_args)):
        for t in (lambda t: t, on_gpu):
            with pytest.raises(ValueError):
                call(c, [t(x) for x in args()], 0)
    with pytest.raises(ValueError):
        plan(c, plan_args(), 0)
    assert not reached
