"""Rules that the drafted tokens' kernels keep, seen without a GPU: those that a run
cannot show, and the binding's."""
import os
import re

import numpy as np
import pytest
import torch

from block_sparse_gqa_msa_gb300 import api, autograd
from oracle import drafts

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_gqa_msa_gb300", "csrc")


def _code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_warp_group_moves_its_registers_in_one_place():
    """All warps of a warp group have to execute the same setmaxnreg: one call for the
    first group in front of the branch into its roles, one for the softmax groups."""
    code = _code("paged_tree.cu")
    assert len(re.findall(r"\bfewer_registers<k\w+>\(\)", code)) == 1
    assert len(re.findall(r"\bmore_registers<k\w+>\(\)", code)) == 1
    assert re.search(r"if \(warp < kSoftWarp0\) \{\s*fewer_registers<kOtherRegs>\(\);", code)
    # and that group is whole warp groups
    roles = dict(re.findall(r"\b(kCopyWarps|kCopyWarp0) = (\d+)", code))
    assert (int(roles["kCopyWarp0"]) + int(roles["kCopyWarps"])) % 4 == 0


def tiny_rest():
    """Rows where the first draft is not kept and leaves 1e-40, whose reciprocal passes
    fp32's range, or 1e-37, whose reciprocal does not; the second draft is a token
    without probability, or the one that is left."""
    p, q = np.zeros((12, 16), np.float32), np.zeros((12, 16), np.float32)
    for row, left in enumerate((1e-40, 1e-37) * 2):
        p[3 * row, 7], p[3 * row, 5], p[3 * row + 2, 9] = 0.5, left, 1.0
        q[3 * row, 7] = 1.0
    return dict(target=p, draft=q, tokens=[0, 7, 3] * 2 + [0, 7, 5] * 2, offs=[0, 3, 6, 9, 12],
                parents=[-1, 0, 0] * 4, u=np.full(12, 0.75, np.float32),
                u_last=np.full(4, 0.5, np.float32), max_path=3)


def test_a_rest_too_small_for_fp32_is_nothing():
    """The target itself is drawn from then: half of its sum is reached at token 7."""
    path, count, last = drafts.verify(**tiny_rest())
    assert path.tolist() == [[0, -1, -1]] * 3 + [[0, 2, -1]]
    assert count.tolist() == [1, 1, 1, 2] and last.tolist() == [7, 5, 7, 9]


def _stand_in_norm(q, k, q_weight, k_weight, *_, **__):
    return q * q_weight, k * k_weight


def _stand_in_norm_backward(dq, dk, q, k, q_weight, k_weight, *_, **__):
    return dq * q_weight, dk * k_weight, (dq * q).sum((0, 1)), (dk * k).sum((0, 1))


@pytest.mark.parametrize("op", ["norm", "attention"])
def test_second_derivatives_raise(monkeypatch, op):
    """A gradient penalty must not lose its term in silence.  (Kernels replaced by
    arithmetic on the CPU; what is tested is what autograd does with their results.)"""
    x = torch.randn(3, 2, 4).requires_grad_()
    if op == "norm":
        monkeypatch.setattr(api, "msa_norm_rope", _stand_in_norm)
        monkeypatch.setattr(api, "msa_norm_rope_backward", _stand_in_norm_backward)
        w = torch.randn(4).requires_grad_()
        out = sum(y.sum() for y in autograd.msa_norm_rope(x, x, w, w))
        leaves = (x, w)
    else:
        monkeypatch.setattr(api, "msa_forward", lambda p, q, k, v, s: (q * k * v, q.sum(2)))
        monkeypatch.setattr(api, "msa_backward", lambda p, q, k, v, o, lse, do, s: (do * k * v,) * 3)
        out = autograd.MSAFunction.apply(x, x, x, None, 1.0)[0].sum()
        leaves = (x,)
    # first derivatives are the same
    plain = torch.autograd.grad(out, leaves, retain_graph=True)
    assert not any(g.requires_grad for g in plain)
    grads = torch.autograd.grad(out, leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(grads, plain))
    other = (x ** 2).sum()  # a loss that is differentiable beside it
    with pytest.raises(RuntimeError, match="no gradients of their own"):
        (other + sum((g ** 2).sum() for g in grads)).backward()
