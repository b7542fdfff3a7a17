"""The token exchange at the ends of its ranges."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
mg = pytest.importorskip("moe_grouped_block_amd")
import layer_ref as ref  # noqa: E402
from test_gpu_exchange import same_codes  # noqa: E402

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


@pytest.mark.parametrize("fmt,most", [("e4m3", 448.0), ("e5m2", 57344.0), ("e2m1x2", 6.0)])
def test_products_that_decide_by_their_last_bits(fmt, most):
    """combine_backward's MX rows from w dy with weights of 24 bits: the product
    is rounded once, to fp32, and its last bits decide the scale (amax one unit
    on each side of the border) and the codes (ties, and a unit beside them);
    products that overflow make the block NaN, subnormal ones are kept."""
    gen = torch.Generator().manual_seed(17)
    h, k = 512, 4
    one = torch.tensor(1.0)
    up, down = torch.nextafter(one, torch.tensor(2.0)), torch.nextafter(one, torch.tensor(0.0))
    weights = []
    for e in (-130, -126, -60, -3, 0, 5, 60, 110):
        for f in (one, up, down):
            weights.append(float(f) * 2.0 ** e)
    for e in (-20, 0, 30):                                # with dy = 1 in every block: amax on the border of two scales
        for f in (one, up, down):
            weights.append(most * float(f) * 2.0 ** e)
    w = torch.tensor(weights, dtype=torch.float64).float()
    w = torch.cat([w, -w, torch.rand(190, generator=gen), torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 3e38])])
    w = torch.cat([w, torch.rand(-w.numel() % k, generator=gen)])
    t = w.numel() // k
    w = w[torch.randperm(w.numel(), generator=gen)].reshape(t, k)
    # dy: 1 is each block's largest; the others run over 7-bit mantissas (ties of all three formats), some far smaller
    mant = 1.0 + torch.randint(0, 128, (t, h), generator=gen) / 128.0
    dy = (mant * torch.exp2(torch.randint(-12, 0, (t, h), generator=gen).float())).clamp(max=0.9921875)
    dy = torch.where(torch.rand(t, h, generator=gen) < 0.5, -dy, dy)
    dy[:, ::32] = 1.0
    dy[0, 1::2], dy[1, 5], dy[2, 40] = 3e38, -3e38, 1e-38
    dy = dy.to(torch.bfloat16)
    ids = torch.randint(0, 5, (t, k), generator=gen, dtype=torch.int32)
    plan = mg.sort_tokens(ids.cuda(), 5, m_aligned=1)
    print(f"[gpu-case] combine_backward {fmt} last bits, {t} tokens", flush=True)
    (codes, sf), _ = mg.combine_backward(dy.cuda(), plan, weights=w.cuda(), dtype=fmt)
    slot = plan.slot_of.cpu().long()
    product = dy.float()[slot // k] * w.reshape(-1)[slot][:, None]           # fp32, rounded once
    want, byte = ref.mx_encode(product.double(), fmt)
    assert (byte == 255).any() and (byte == 0).any()
    assert np.array_equal(sf.cpu().numpy(), byte)
    assert same_codes(codes.cpu().numpy(), want, fmt)
    # (rounded to bf16 first, scales and codes would differ)
    other, obyte = ref.mx_encode(product.to(torch.bfloat16).double(), fmt)
    assert not np.array_equal(obyte, byte) and not same_codes(other, want, fmt)
