"""Tensors with tangents (forward-mode derivatives) are refused: no operator carries them
on, and a result without a tangent would stand for a derivative of zero."""
import pytest
import torch
import torch.autograd.forward_ad as fa

import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def _cases():
    """name -> (the call by its tensors, the tensors)."""
    def z(*shape):
        return torch.zeros(*shape, device="cuda")

    ids = torch.zeros(20, dtype=torch.int64, device="cuda")
    order = sc.expert_sort(ids.view(10, 2), 3)
    A, D = -torch.ones(8, 4, device="cuda"), z(8)
    x, g = z(2, 20, 8), z(2, 20, 8)
    ssm, gated = sc.selective_scan_saved(x, A), sc.gated_scan_saved(x)
    norm = sc.layer_norm_saved(x)
    return {
        "embed": (lambda w: sc.embed(ids, w), (z(5, 8),)),
        "embed_grad": (lambda d: sc.embed_grad(ids, d, 5), (z(20, 8),)),
        "causal_conv": (lambda x, w, b, s: sc.causal_conv(x, w, b, state=s), (x, z(8, 4), z(8), z(2, 3, 8))),
        "causal_conv_grad": (lambda d, x, w: sc.causal_conv_grad(d, x, w), (g, x, z(8, 4))),
        "causal_conv_step": (lambda x, s, w: sc.causal_conv_step(x, s, w), (z(2, 8), z(2, 3, 8), z(8, 4))),
        "selective_scan": (lambda x, dt, A, B, C, D: sc.selective_scan(x, dt, A, B, C, D),
                           (x, g, A, z(2, 20, 1, 4), z(2, 20, 1, 4), D)),
        "selective_scan_grad": (lambda d, x, dt, A, B, C: sc.selective_scan_grad(d, x, dt, A, B, C, saved=ssm),
                                (g, x, g, A, z(2, 20, 1, 4), z(2, 20, 1, 4))),
        "selective_scan_step": (lambda x, dt, A, B, C, h: sc.selective_scan_step(x, dt, A, B, C, h),
                                (z(2, 8), z(2, 8), A, z(2, 1, 4), z(2, 1, 4), z(2, 8, 4))),
        "gated_scan": (lambda x, g, s: sc.gated_scan(x, g, state=s), (x, g, z(2, 8))),
        "gated_scan_grad": (lambda d, x, g: sc.gated_scan_grad(d, x, g, saved=gated), (x.clone(), x, g)),
        "gated_scan_step": (lambda x, g, h: sc.gated_scan_step(x, g, h), (z(2, 8), z(2, 8), z(2, 8))),
        "layer_norm": (lambda x, w, b, r: sc.layer_norm(x, w, b, residual=r), (x, z(8), z(8), g)),
        "layer_norm_grad": (lambda d, x, w, s: sc.layer_norm_grad(d, x, w, saved=norm, dsum=s), (g, x, z(8), g)),
        "expert_gather": (lambda x: sc.expert_gather(x, order), (z(10, 8),)),
        "expert_gather_grad": (lambda d: sc.expert_gather_grad(d, order), (z(20, 8),)),
        "expert_combine": (lambda y, w: sc.expert_combine(y, order, w), (z(20, 8), z(10, 2))),
        "expert_combine_grad": (lambda d, y, w: sc.expert_combine_grad(d, y, order, w), (z(10, 8), z(20, 8), z(10, 2))),
    }


def test_every_call_refuses_them():
    for name, (call, tensors) in _cases().items():
        for i in range(len(tensors)):
            for grad in (False, True):
                if grad and name.endswith(("_grad", "_step")):
                    continue  # these record nothing, or refuse as such
                with fa.dual_level():
                    args = list(tensors)
                    dual = fa.make_dual(args[i].clone().requires_grad_(grad), torch.ones_like(args[i]))
                    args[i] = dual
                    with pytest.raises(NotImplementedError):
                        call(*args)
        with fa.dual_level():
            call(*tensors)  # without a tangent


def test_where_forward_mode_is_off():
    x = torch.ones(2, 20, 8, device="cuda")
    want = sc.layer_norm(x)
    with fa.dual_level():
        dual = fa.make_dual(x, x)
        with fa._set_fwd_grad_enabled(False):
            assert torch.equal(sc.layer_norm(dual), want)
