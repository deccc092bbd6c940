"""The 4-bit key/value cache on a GPU at the edges of what its calls accept."""
import numpy as np
import pytest
import torch

import _kv_reference as ref
from test_gpu_kvcache import Setup, WIDE, check_attention, fa, ok, rows_alone  # noqa: F401 (fa: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_that_alternate_give_the_same_bits(fa, D):
    """Operands, and whether a page counts, pass between warps and CTAs: what is left of the call before, which had
    other data and other bad pages in the same places, must not show."""
    s = Setup(fa, [700, 200, 1300, 64], [300, 140, 90, 64], H=4, D=D, seed=7)
    s.append_all()
    ok(fa)
    good = s.d_table
    tables = [good, good.clone(), good.clone()]
    tables[1][0, 3], tables[1][2, 8], tables[1][2, 20] = -1, s.P, -1
    tables[2][0, 4], tables[2][1, 0], tables[2][2, 9] = s.P + 1, -1, -1
    qs = [s.queries(3).cuda() for _ in tables]
    want = []
    for turn in range(40):
        i = turn % 3
        s.d_table = tables[i]
        o, lse = rows_alone(fa, s, qs[i])
        if turn < 3:
            want.append((o, lse))
        else:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]), turn
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FP4ATTN_ERR_BAD_INDEX
    s.store_all()
    cu, lens = s.cu, s.lens
    o, lse, to, tl = ref.attention(qs[0].double().cpu().numpy(), s.pool, s.table, lens, cu, D, s.k_exp, s.v_exp, D ** -0.5,
                                   prompt=True)
    assert np.all(np.abs(want[0][0].double().cpu().numpy() - o) <= to)
    assert np.all(np.abs(want[0][1].double().cpu().numpy() - lse) <= tl)
    assert all(torch.all(torch.isfinite(o)) for o, _ in want)
