"""The conveniences that allocate do it on the stream that they are given (CPU: torch's stream
context, its allocations and the entry points are stood in for).  Memory that is allocated on
another stream than the one that uses it may be given out again too early."""
import inspect

import pytest
import torch

from gated_delta_rule_33_gb300 import kda

CONVENIENCES = ["gate", "prefill", "prefill_gated", "decode_indexed", "short_conv", "short_conv_step",
                "backward", "backward_chunked", "prefill_checkpointed", "backward_from_checkpoints",
                "decode_gated", "gate_backward", "decode", "page_plan", "paged_decode"]


def test_the_list_is_whole():
    """Every function after the entry points' own that takes a stream is in the list."""
    names = [n for n, f in vars(kda).items()
             if inspect.isfunction(f) and f.__module__ == kda.__name__ and not n.startswith(("_", "kda_"))
             and "stream" in inspect.signature(f).parameters]
    assert sorted(names) == sorted(CONVENIENCES)


def arguments():
    x = torch.zeros(4, 2, 128)
    w = torch.zeros(256, 4)
    ints = torch.zeros(4, dtype=torch.int32)
    cache = kda.PagedCache(*(torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16) for _ in range(2)))
    return dict(q=x, k=x, v=x, g=x, beta=x[..., 0], f=x, b=x[..., 0], dO=x, dg=x, dbeta=x[..., 0],
                A_log=torch.zeros(128), dt_bias=torch.zeros(2, 128), state=x, state_pool=x,
                conv_state_pool=x, state_indices=ints, x_q=x, x_k=x, x_v=x, w_q=w, w_k=w, w_v=w,
                checkpoints=x, cached_lens=ints, new_lens=ints, free_pages=ints,
                block_table=ints.view(4, 1), page_size=16, num_pages=4, num_tokens=4, cache=cache,
                seq_lens=ints)


@pytest.mark.parametrize("positional", [False, True])
@pytest.mark.parametrize("handle", [None, 77])
@pytest.mark.parametrize("name", CONVENIENCES)
def test_allocations_are_on_the_given_stream(monkeypatch, name, handle, positional):
    on, made, ran = [], [], []

    class Context:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            on.append(self.stream)

        def __exit__(self, *_):
            on.pop()
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device: ("stream", h))
    monkeypatch.setattr(torch.cuda, "stream", Context)
    for maker in ("empty", "empty_like", "zeros", "zeros_like", "full"):
        real = getattr(torch, maker)
        monkeypatch.setattr(torch, maker, lambda *a, _f=real, **kw: made.append(list(on)) or _f(*a, **kw))
    for entry in [n for n in vars(kda) if n.startswith("kda_")]:
        stand_in = (lambda *a: 4096) if entry.endswith("_size") else lambda *a, **kw: ran.append(a)
        monkeypatch.setattr(kda, entry, stand_in)
    f = getattr(kda, name)
    params = inspect.signature(f).parameters
    have = arguments()
    made.clear()
    args = {n: have[n] for n, p in params.items() if p.default is inspect.Parameter.empty}
    if positional:
        f(*[handle if n == "stream" else args.get(n, p.default) for n, p in params.items()])
    else:
        f(**args, stream=handle)
    want = [] if handle is None else [("stream", handle)]
    assert len(ran) == 1 and made and all(m == want for m in made)
    assert not on
