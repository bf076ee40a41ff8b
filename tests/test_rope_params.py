"""Rotary parameters as the binding makes them (CPU)."""
import pytest

from adaptive_block_sparse_fractal_b200 import nabla


def test_one_number_or_one_per_axis():
    p = nabla.rope_params_of((22, 21, 21), theta=500.0, scale=(1.0, 0.5, 2.0), offset=[3, 0, -1.5])
    assert tuple(p.pairs) == (22, 21, 21)
    assert tuple(p.theta) == (500.0,) * 3
    assert tuple(p.scale) == (1.0, 0.5, 2.0) and tuple(p.offset) == (3.0, 0.0, -1.5)
    p = nabla.rope_params_of((8, 4), theta=(10.0, 20.0), offset=7)
    assert tuple(p.pairs) == (8, 4, 0)
    assert tuple(p.theta)[:2] == (10.0, 20.0) and tuple(p.offset)[:2] == (7.0, 7.0)


@pytest.mark.parametrize("name", ["theta", "scale", "offset"])
@pytest.mark.parametrize("values", [(), (2.0,), [2.0, 3.0], (1.0, 2.0, 3.0, 4.0)])
def test_another_number_of_values_is_refused(name, values):
    with pytest.raises(ValueError, match=name):
        nabla.rope_params_of((22, 21, 21), **{name: values})


def test_more_values_than_axes_are_refused():
    for n in (2, 3):
        with pytest.raises(ValueError, match="offset"):
            nabla.rope_params_of((16,), offset=(1.0,) * n)
