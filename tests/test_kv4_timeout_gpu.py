"""Equal pieces of which some are never done: after a timeout the merge meets table entries that no CTA wrote."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv4_util as U  # noqa: E402
from mla_speculative_decode_tree_gb300 import binding as B  # noqa: E402


@pytest.mark.parametrize("fill", [0x00, 0x7F, 0x80, 0xFF, 0x01])
def test_a_timeout_with_a_workspace_of_other_contents(fill):
    """Five requests to a CTA, and the first one's expansion stalls: the entries of the others stay as they were.  They
    are kept inside the workspace, whatever they are; the call ends and reports, and the next one is right."""
    b = 760
    wl = U.workload(b, 4, [1] * b, [20] * b, b * 21 + 10, seed=1)
    d, v = U.device(wl), U.verifier(wl, 0, B.MLA_VERIFY_TEST_STALL_GATHER)
    table = v.workspace[256:256 + 8 * b]  # an int32 pair for each request's row group
    table.fill_(fill)
    v.run(d, b, wl["sm_scale"])
    assert v.status() & B.MLA_VERIFY_DEV_TIMEOUT
    assert bool((table.view(b, 8) == fill).all(dim=1).any())  # some were not written
    U.run_and_check(wl, 0, 0, "after the stall")
