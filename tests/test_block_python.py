"""The layer operators' Python functions without a GPU: signatures and refusals."""
import inspect

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F


def test_clip_grad_norm_takes_torchs_positional_arguments():
    """A caller of torch's function who passes norm_type third must not set eps by it."""
    ours = list(inspect.signature(F.clip_grad_norm_).parameters.values())
    torchs = list(inspect.signature(torch.nn.utils.clip_grad_norm_).parameters)
    positional = [p.name for p in ours if p.kind is p.POSITIONAL_OR_KEYWORD]
    assert positional == torchs[:len(positional)] == ["parameters", "max_norm", "norm_type"]
    p = torch.nn.Parameter(torch.zeros(3))
    assert float(F.clip_grad_norm_([p], 1.0)) == 0.0
    assert float(F.clip_grad_norm_([p], 1.0, 2, eps=1e-3)) == 0.0
    for norm_type in (1.0, float("inf"), 1e-6):
        with pytest.raises(ValueError, match="norm_type"):
            F.clip_grad_norm_([p], 1.0, norm_type)


def test_clip_grad_norm_takes_a_tied_parameter_once(monkeypatch):
    """In place, a tensor that is given twice would be scaled by two blocks at once."""
    from linear_cross_entropy_gemm_gb300 import block
    seen = []
    monkeypatch.setattr(block, "flce_clip_grads", lambda grads, *a, **k: seen.append(list(grads)))
    p, q = torch.nn.Parameter(torch.ones(3)), torch.nn.Parameter(torch.ones(3))
    p.grad, q.grad = torch.ones(3), torch.ones(3)
    F.clip_grad_norm_(iter([p, q, p, q, torch.nn.Parameter(torch.ones(1))]), 1.0)
    F.clip_grad_norm_(p, 1.0)
    assert [[id(g) for g in grads] for grads in seen] == [[id(p.grad), id(q.grad)], [id(p.grad)]]
