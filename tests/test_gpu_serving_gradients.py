"""Serving calls have no derivative: tensors that carry one are refused, in reverse and in forward mode."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from gpu_support import lib
from test_gpu_serving import BF16

pytestmark = pytest.mark.gpu


def _calls():
    z = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    i = torch.int32
    hg = lib()
    return {
        "qk_norm_rope": (lambda **a: hg.qk_norm_rope(**a), dict(
            q=z(2, 8, 64), k=z(2, 2, 64), positions=z(2, t=i), inv_freq=z(32, t=torch.float64), q_weight=z(64), k_weight=z(64))),
        "kv_append": (lambda **a: hg.kv_append(**a), dict(
            k=z(2, 2, 64), v=z(2, 2, 64), k_cache=z(4, 2, 16, 64), v_cache=z(4, 2, 16, 64),
            slots=torch.arange(2, device="cuda"), k_weight=z(64))),
        "paged_attention": (lambda **a: hg.paged_attention(**a), dict(
            q=z(2, 8, 64), k_cache=z(4, 2, 16, 64), v_cache=z(4, 2, 16, 64), block_table=z(2, 2, t=i), kv_len=z(2, t=i) + 3)),
    }


@pytest.mark.parametrize("name", ["qk_norm_rope", "kv_append", "paged_attention"])
def test_tensors_with_a_derivative(name):
    call, args = _calls()[name]
    call(**args)
    of = [k for k, x in args.items() if x.is_floating_point()]
    assert len(of) >= 3
    for k in of:
        with pytest.raises(ValueError, match="gradient"):
            call(**dict(args, **{k: args[k].clone().requires_grad_()}))
        with torch.no_grad():
            call(**dict(args, **{k: args[k].clone().requires_grad_()}))
        with fwd.dual_level():
            dual = fwd.make_dual(args[k], torch.ones_like(args[k]))
            with pytest.raises(ValueError, match="gradient"):
                call(**dict(args, **{k: dual}))
            with pytest.raises(ValueError, match="gradient"):  # a view of it
                call(**dict(args, **{k: dual.view_as(dual)}))
            call(**dict(args, **{k: fwd.unpack_dual(dual).primal}))
            call(**args)
    call(**args)
