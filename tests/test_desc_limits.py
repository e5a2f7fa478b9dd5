"""Descriptors at the documented limits, and what the classes raise for those beyond: no GPU."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def mb():
    import mlp_block_backprop_gb300 as mb
    return mb


def test_batches_of_just_below_two_to_the_forty_elements(mb):
    """129648 x 130473 x 65 = 2^40 - 16 elements are taken; one matrix more is not."""
    d = mb.make_ortho_desc(129648, 130473, batch=65)
    assert 129648 * 130473 * 65 < 1 << 40
    assert mb.mlpblk_orthogonalize_workspace_size(d) > 6 * ((1 << 40) - 16)      # three X in fp16
    assert mb.mlpblk_orthogonalize_workspace_size(mb.make_ortho_desc(129648, 130473, batch=66)) == 0
    assert mb.mlpblk_orthogonalize_workspace_size(mb.make_ortho_desc(131072, 131072, batch=64)) == 0
    assert mb.mlpblk_orthogonalize_workspace_size(mb.make_ortho_desc(131072, 131071, batch=64)) > 0


@pytest.mark.parametrize("kw,code", [(dict(width=16385), "MLPBLK_ENOTSUP"), (dict(block=64), "MLPBLK_ENOTSUP"), (dict(width=0), "MLPBLK_EINVAL"),
                                     (dict(tokens=-1), "MLPBLK_EINVAL"), (dict(eps=-1.0), "MLPBLK_EINVAL")])
def test_classes_raise_the_code_of_the_abi(mb, kw, code):
    with pytest.raises(mb.MlpBlkError) as e:
        mb.AddRmsNorm(**{**dict(tokens=4, width=64), **kw}, device="cpu")
    assert e.value.code == getattr(mb, code)


def test_orthogonalizer_raises_the_code_of_the_abi(mb, monkeypatch):
    with pytest.raises(mb.MlpBlkError) as e:
        mb.Orthogonalizer(0, 50, device="cpu")
    assert e.value.code == mb.MLPBLK_EINVAL
    made = mb.make_ortho_desc

    def of_another_type(*a, **kw):
        d = made(*a, **kw)
        d.dtype = 9
        return d

    monkeypatch.setattr(mb, "make_ortho_desc", of_another_type)
    with pytest.raises(mb.MlpBlkError) as e:
        mb.Orthogonalizer(40, 50, device="cpu")
    assert e.value.code == mb.MLPBLK_ENOTSUP
