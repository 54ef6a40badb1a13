"""Arguments of the distillation loss at an edge: refused before anything is enqueued."""
import pytest

VALUE = -4


@pytest.mark.parametrize("T,status", [(3.5e-39, VALUE), (4.2e-39, VALUE), (1e-42, VALUE), (5e-39, 0), (1e-38, 0),
                                      (1e-30, 0), (1.0, 0), (3e38, 0)])
def test_temperature_whose_logarithm_factor_is_infinite(T, status):
    """log2(e) / T is the factor of every exponent: where fp32 has 1 / T but not that, 0 times it would be NaN."""
    import rotated_w4_linear_amd as paro
    a = 0x10000
    fn = paro.load_library().paro_distill_loss
    # (no rows: nothing is enqueued either way)
    assert fn(a, 0, a, 0, a, None, None, 0, 100, 8, T, 1.0, a, a, None) == status
