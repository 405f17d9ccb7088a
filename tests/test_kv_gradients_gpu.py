"""kv_attention on queries that require a gradient: the result is the same, and
a backward pass through it is refused instead of leaving the gradient out."""
from __future__ import annotations

import pytest
import torch

from test_kv_gpu import DEV, Scene, nv, say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_is_refused(nv, dtype):  # noqa: F811
    say("gradients", dtype)
    s = Scene(71, [2, 20], [700, 150], 4, 2, 64, 32, dtype=dtype)
    plain = s.q.to(DEV)
    want = nv.kv_attention(plain, *s.dev(), max_q=20, max_kv=702, window=300, scale=0.2)
    assert not want.requires_grad
    q = plain.clone().requires_grad_()
    got = nv.kv_attention(q, *s.dev(), max_q=20, max_kv=702, window=300, scale=0.2)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and got.requires_grad
    with pytest.raises(RuntimeError, match="no backward pass"):
        (got.float() * 2).sum().backward()
    assert q.grad is None
    # the middle of a graph
    x = torch.ones_like(plain).requires_grad_()
    with pytest.raises(RuntimeError, match="no backward pass"):
        nv.kv_attention(x * plain, *s.dev()).float().sum().backward()
    # none asked for
    with torch.no_grad():
        assert not nv.kv_attention(q, *s.dev()).requires_grad
    assert not nv.kv_attention(q.detach(), *s.dev()).requires_grad
    out = torch.empty_like(plain)
    assert not nv.kv_attention(q, *s.dev(), max_q=20, max_kv=702, window=300, scale=0.2, out=out).requires_grad
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_query_that_requires_a_gradient_on_a_stream(nv):  # noqa: F811
    s = Scene(72, [1, 1], [40, 3], 2, 1, 64, 16)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = nv.kv_attention(s.q.to(DEV), *s.dev())
    q = s.q.to(DEV).requires_grad_()
    work = torch.empty(64, dtype=torch.uint8, device=DEV)
    args = s.dev()
    torch.cuda.synchronize()
    got = nv.kv_attention(q, *args, workspace=work, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and got.requires_grad
