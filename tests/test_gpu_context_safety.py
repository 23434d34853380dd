"""What the rotation, norm and draft-tree calls report, and what they hold up while they run."""
import numpy as np
import pytest

from test_gpu_tree import _case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa(cuda_device):
    import long_context_memory_b200 as m

    return m


@pytest.mark.parametrize("B", [1, 32, 33, 70])
@pytest.mark.parametrize("bad", ["only", "beside an empty one", "nothing drafted"])
def test_bad_documents_are_reported_in_every_batch(msa, cuda_device, B, bad):
    """A document id out of range raises the device error whatever the batch, also where its query has
    no pooled row left or no draft in use."""
    k = 2 if bad == "beside an empty one" else 1
    c = _case(B, B, 3, 4, 2, 64, 20, np.full(B, 20), k, False, cuda_device)
    ids = len(c["off"]) - 1
    _run(msa, c, cuda_device)
    assert msa.check_device_errors() == 0
    if bad == "beside an empty one":  # the last document has no rows
        c["off"] = np.append(c["off"], c["off"][-1])
        c["top"][-1] = ids
        ids += 1
        _run(msa, c, cuda_device)
        assert msa.check_device_errors() == 0
    if bad == "nothing drafted":
        c["n_draft"] = np.zeros(B, dtype=np.int32)
    for value in (ids, -1):
        c["top"][-1, -1] = value
        _run(msa, c, cuda_device)
        with pytest.raises(msa.MSAError):
            msa.check_device_errors()


@pytest.mark.parametrize("B,k", [(1, 2), (32, 1), (33, 1), (40, 0)])
def test_kernels_are_traced_under_their_own_names(msa, cuda_device, B, k):
    """The attention alone: no time of the plan's, and the counting of large batches' rows by its name."""
    c = _case(B, B, 3, 4, 2, 64, 20, np.full(B, 20), k, False, cuda_device)
    _run(msa, c, cuda_device)
    msa.trace_enable(True)
    try:
        msa.trace_reset()
        _run(msa, c, cuda_device)
        launches = {name: n for name, (_, n) in msa.trace_read().items() if n}
    finally:
        msa.trace_enable(False)
    want = {"tree_attend": 1, "tree_combine": 1}
    if B > 32 and k:
        want["tree_select"] = 1
    assert launches == want
