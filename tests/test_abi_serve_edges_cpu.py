"""Ends of the routing's and the adapters' binding: sizes past C's ints, matrices of no
rows (host only: none of these calls reaches a HIP API)."""
import pytest

import gemm_exl3_linear_amd as X

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("field", ["experts", "topk", "groups", "topk_groups"])
@pytest.mark.parametrize("past", [1 << 32, 3 << 32, -(1 << 32), 1 << 31])
def test_a_rules_numbers_are_not_taken_modulo_32_bits(field, past):
    sound = dict(experts=64, topk=2, groups=4, topk_groups=2)
    X.Exl3RouteRule(**sound)
    with pytest.raises(ValueError):
        X.Exl3RouteRule(**sound | {field: sound[field] + past})


def test_shapes_are_not_taken_modulo_32_bits():
    meta = lambda *s: torch.empty(s, dtype=torch.float16, device="meta")
    assert X.Exl3Router(meta(64, 128))._record.hidden == 128
    for shape in ((64 + (1 << 32), 128), (64, 128 + (1 << 32)), (64, 1 << 31)):
        with pytest.raises(ValueError):
            X.Exl3Router(meta(*shape))
    big = 1 << 32
    for a, b in (((2 + big, 8, 64), (2 + big, 5, 8)), ((2, 8 + big, 64), (2, 5, 8 + big))):
        with pytest.raises(ValueError):
            X.Exl3Lora(meta(*a), meta(*b))


def test_any_number_that_is_not_zero_renormalizes():
    for value, want in ((True, 1), (False, 0), (1, 1), (0, 0), (1 << 32, 1)):
        assert X.Exl3RouteRule(64, 2, renormalize=value)._record.renormalize == want


def test_rows_of_no_matrix_may_lie_anyhow():
    """Strides say nothing about a matrix without rows; with rows they do."""
    none = torch.empty((8, 0), dtype=torch.float16).t()
    assert none.stride() != (8, 1) and X._matrix(none, "x", 0, 8) == (0, 8, 8)
    assert X._f16_rows(none, 8) == (0, 8)
    with pytest.raises(ValueError):
        X._matrix(none, "x", 0, 16)
    with pytest.raises(ValueError):
        X._matrix(torch.empty((8, 2), dtype=torch.float16).t(), "x", 2, 8)
