"""CPU tests of what the operators on a paged cache refuse, beside test_paged_oracle_abi.py."""
import pytest
import torch

from ag_gemm_gb300 import binding as B
from test_paged_oracle_abi import append, attention, batch, desc


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_a_scale_that_is_no_number_in_base_2_is_refused():
    assert append(desc(scale=2.0 ** 127), q=[257]) == attention(desc(scale=2.0 ** 127), q=[257]) == B.FO_ERR_ALIGN   # (what is checked next)
    for scale in (2.4e38, 3.4e38):
        assert append(desc(scale=scale)) == attention(desc(scale=scale)) == B.FO_ERR_INVALID_ARG


def test_a_workspace_without_room_for_a_status_is_refused():
    with pytest.raises(ValueError, match="smaller"):
        B.fo_kv_append(desc(), None, batch(), 3, [256], [256], [256], [256], [256], [256], ws=torch.zeros(48, dtype=torch.uint8), stream=0)
