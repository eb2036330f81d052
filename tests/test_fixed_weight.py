"""What the operators' modules hold of a fixed weight: whether it is still the one
that was fixed, through changes, replacement and copies.  No GPU."""
import copy
import pickle

import pytest
import torch


def _modules():
    from fp32_emulated_gemm_amd.adapters import AdapterLinear
    from fp32_emulated_gemm_amd.gated import GatedLinear
    return GatedLinear(8, 6), AdapterLinear(8, 6, adapters=2, rank=3)


def _copies(m):
    return copy.deepcopy(m), pickle.loads(pickle.dumps(m))


@pytest.mark.parametrize("which", [0, 1])
def test_changes_and_replacement_are_seen(which):
    m = _modules()[which]
    with torch.no_grad():
        m.weight.mul_(2)                       # before it is fixed: any number of changes
    m.fix_weights()
    m._fixed.check(m.weight)
    with torch.no_grad():
        m.weight.mul_(2)
    with pytest.raises(RuntimeError):
        m._fixed.check(m.weight)
    m.fix_weights()
    m._fixed.check(m.weight)
    other = torch.nn.Parameter(m.weight.detach().clone())
    for _ in range(m.weight._version - other._version):
        with torch.no_grad():
            other.add_(0)
    assert other._version == m.weight._version
    m.weight = other                           # another tensor of the same version
    with pytest.raises(RuntimeError):
        m._fixed.check(m.weight)


@pytest.mark.parametrize("which", [0, 1])
def test_copies_are_as_fixed_as_the_original(which):
    m = _modules()[which]
    for c in _copies(m):
        assert c._fixed is None
    with torch.no_grad():
        m.weight.mul_(2)
    m.fix_weights()
    for c in _copies(m):
        assert c.weight is not m.weight and torch.equal(c.weight, m.weight)
        c._fixed.check(c.weight)
        with torch.no_grad():
            c.weight.mul_(2)
        with pytest.raises(RuntimeError):
            c._fixed.check(c.weight)
        m._fixed.check(m.weight)
    with torch.no_grad():
        m.weight.mul_(2)                       # changed since: so are its copies
    for c in _copies(m):
        with pytest.raises(RuntimeError):
            c._fixed.check(c.weight)


def test_modules_made_for_inference():
    """An inference tensor's changes are not counted; only its replacement is seen."""
    with torch.inference_mode():
        for m in _modules():
            m.fix_weights()
            m._fixed.check(m.weight)
            m.weight.mul_(2)
            m._fixed.check(m.weight)
            c = copy.deepcopy(m)
            c._fixed.check(c.weight)
            m.weight = torch.nn.Parameter(m.weight.clone(), requires_grad=False)
            with pytest.raises(RuntimeError):
                m._fixed.check(m.weight)
        from fp32_emulated_gemm_amd.adapters import AdapterLinear
        m = AdapterLinear.from_linear(torch.nn.Linear(8, 6), 2, 3)
        m._fixed.check(m.weight)
