"""Calls over trees and shared pages with tensors on a GPU that is not the current one: refused, since
kernels are launched on the current one."""
import pytest
import torch

import gated_delta_rule_33_gb300 as kda
from test_tree_boundary import calls, on_gpu, reached  # noqa: F401


@pytest.mark.parametrize("name", sorted(calls()))
def test_another_device_is_refused(reached, monkeypatch, name):  # noqa: F811
    call, tensors = calls()[name]
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    for current, gpu in ((0, 0), (1, 0), (0, 1), (1, 1)):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
        cache = kda.PagedCache(on_gpu(k, gpu), on_gpu(k.clone(), gpu))
        reached.clear()
        a = [on_gpu(t.clone(), gpu) for t in tensors]
        if current == gpu:
            call(cache, a, 77)
            assert reached == [name]
        else:
            with pytest.raises(ValueError, match="current device"):
                call(cache, a, 77)
            assert reached == []
