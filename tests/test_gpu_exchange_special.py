"""The token exchange at the ends of its ranges."""
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")

pytestmark = pytest.mark.gpu


def test_sort_of_the_most_slots():
    """2^31 - 1 slots, all of the first expert: the experts behind it start at
    row 2^31 - 1, where a row number plus a thread's passes 32 bits."""
    t, e = 2 ** 31 - 1, 3
    print(f"[gpu-case] sort {t}x1 experts={e}", flush=True)
    ids = torch.zeros(t, 1, dtype=torch.int32, device="cuda")
    plan = mg.sort_tokens(ids, e, m_aligned=1)
    assert plan.rows == t and plan.padded_offsets.tolist() == [t] * e
    step = 2 ** 27
    count = torch.arange(step, dtype=torch.int32, device="cuda")
    for at in range(0, t, step):
        n = min(step, t - at)
        assert torch.equal(plan.row_of[at:at + n, 0], count[:n] + at), at
        assert torch.equal(plan.slot_of[at:at + n], count[:n] + at), at
