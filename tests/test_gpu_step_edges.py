"""The layer's steps on a GPU at values and sizes where they are easily wrong (tests/step_edges.py)."""
import pytest

import step_edges
from test_gpu_steps import M, be  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", sorted(step_edges.CASES))
def test_edges(be, name):  # noqa: F811
    step_edges.CASES[name](be)


def test_router_scales_of_many_tokens(be):  # noqa: F811
    step_edges.route_scales(be, (30000,))  # the kernel of four threads per token


def test_router_low_scores_of_many_tokens(be):  # noqa: F811
    step_edges.route_low(be, (30000,))
