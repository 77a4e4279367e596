"""The router where a softmax has no value: one logit that is NaN, or +Inf,
makes every softmax value of its token NaN (softmax divides by the sum of all),
and so the token's weights and its row of the result.  The experts are then
tied, and the lowest numbers are taken.  -Inf logits have softmax value 0."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_moe import call, check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,top_k,expert,bad", [
    (8, 2, 3, "nan"), (8, 3, 0, "nan"), (40, 4, 37, "inf"), (256, 8, 255, "nan"), (2, 1, 1, "inf")])
def test_a_logit_without_a_softmax_spoils_its_token_only(E, top_k, expert, bad, renorm):
    """Token 5 alone has a value in the column that only the one expert's router row looks at."""
    mmq = require_gpu()
    d = make(9, 512, 256, E, top_k, renorm, True, 31)
    d["x"][:, 100] = 0
    d["w_router"][:, 100] = 0
    clean = [v.clone() for v in call(mmq, d)]
    # 2 x 3e38 is +Inf in float32; Inf - Inf is NaN
    d["x"][5, 100] = 2.0
    d["w_router"][expert, 100] = 3e38
    if bad == "nan":
        d["x"][:, 300] = 0
        d["w_router"][:, 300] = 0
        clean = [v.clone() for v in call(mmq, dict(d, x=d["x"].index_fill(1, torch.tensor([100], device="cuda"), 0)))]
        d["x"][5, 300] = -2.0
        d["w_router"][expert, 300] = 3e38
    out, ids, weights = call(mmq, d)
    assert ids[5].tolist() == list(range(top_k))
    assert torch.isnan(weights[5]).all() and torch.isnan(out[5]).all()
    keep = [t for t in range(9) if t != 5]
    for got, want in zip((ids, weights), clean[1:]):
        assert torch.equal(got[keep], want[keep])
    assert torch.isfinite(out[keep]).all()


def test_minus_inf_logits_have_no_weight():
    mmq = require_gpu()
    d = make(6, 512, 256, 8, 3, True, False, 33)
    d["x"][:, 100] = 0
    d["w_router"][:, 100] = 0
    d["x"][2, 100] = -2.0
    d["w_router"][[0, 1, 2, 3, 5, 6], 100] = 3e38
    out, ids, weights = call(mmq, d)
    assert sorted(ids[2, :2].tolist()) == [4, 7] and int(ids[2, 2]) == 0 and float(weights[2, 2]) == 0
    assert abs(float(weights[2].sum()) - 1) < 1e-6 and torch.isfinite(out).all()
