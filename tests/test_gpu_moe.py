"""The mixture-of-experts FFN against the formulas in 64 bits.

Tolerance, from f32 arithmetic on the dequantized weights.  A product
y = sum w x over n values, w = d sc q - dmin m, is off by at most
  B(n, x) = (2^-21 + (n / 16 + 40) 2^-23) sum (|d sc q| + |dmin m|) |x|
(the split of x into two fp16 values, 2^-22 each for the products and the
sub-block sums; matrix instructions that add 16 products at a time and may
truncate, 2^-23 each; the f32 steps per super-block).  silu has a slope of at
most 1.1, so h is off by Eh = 1.1 |u| Eg + (|silu(g)| + 1.1 Eg) Eu + 2^-20 |h|,
and y by sum |w| Eh + B(ffn, h).  The weights of the sum: a logit is off by
El = (model 2^-24 + 2^-22) sum |x Wr|, a softmax value by 2 max El + 2^-20 of
itself (and again for the division by the chosen values' sum).
The i-th chosen expert's logit is the i-th largest within 2 El.
"""
import numpy as np
import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def q4k(g, n, k, level, scale_max=64):
    """Random q4_K bytes [n][k/256][144] (CUDA) and their fields' products (d sc q, dmin m) in 64 bits."""
    sb = k // 256
    raw = torch.randint(0, 256, (n, sb, 144), generator=g, dtype=torch.uint8)
    d = ((torch.rand((n, sb, 1), generator=g) + 0.5) * level).half()
    dmin = (d.float() * 7.5).half()
    raw[..., 0:2] = d.view(torch.uint8)
    raw[..., 2:4] = dmin.view(torch.uint8)
    return raw.cuda().contiguous()


def fields(w):
    """(d sc q, dmin m), each [n][k] in 64 bits."""
    n, sb = w.shape[:2]
    b = w.cpu().numpy()
    half = b[..., :4].copy().view(np.float16).astype(np.float64)
    s = b[..., 4:16].astype(np.int64)
    sc, mn = np.zeros((n, sb, 8)), np.zeros((n, sb, 8))
    for j in range(8):
        if j < 4:
            sc[..., j], mn[..., j] = s[..., j] & 63, s[..., j + 4] & 63
        else:
            sc[..., j] = (s[..., j + 4] & 15) | ((s[..., j - 4] >> 6) << 4)
            mn[..., j] = (s[..., j + 4] >> 4) | ((s[..., j] >> 6) << 4)
    q = b[..., 16:].reshape(n, sb, 4, 32)
    v = np.stack([q & 15, q >> 4], axis=3).reshape(n, sb, 8, 32).astype(np.float64)
    one = (half[..., 0:1] * sc)[..., None] * v
    two = np.broadcast_to((half[..., 1:2] * mn)[..., None], one.shape)
    return one.reshape(n, -1), two.reshape(n, -1)


def make(T, model, ffn, E, top_k, renorm, residual, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, model), generator=g) * torch.exp(spread * torch.randn((T, model), generator=g))
    return dict(x=x.cuda(), w_router=(torch.randn((E, model), generator=g) / model ** 0.5).cuda(),
                w_gu=q4k(g, E * 2 * ffn, model, 1 / (184 * model ** 0.5)).view(E, 2 * ffn, model // 256, 144),
                w_down=q4k(g, E * model, ffn, 1 / (184 * ffn ** 0.5)).view(E, model, ffn // 256, 144),
                residual=torch.randn((T, model), generator=g).cuda() if residual else None, top_k=top_k, renorm=renorm)


def call(mmq, d, **more):
    return mmq.q4K_moe(d["x"], d["w_router"], d["w_gu"], d["w_down"], d["top_k"], renormalize=d["renorm"],
                       residual=d["residual"], **more)


def product(x, w, ex=None):
    """(x w^T, bound of its error) for x off by ex."""
    one, two = fields(w)
    n = x.shape[-1]
    y = x @ (one - two).T
    err = (2.0 ** -21 + (n / 16 + 40) * 2.0 ** -23) * (np.abs(x) @ (one + np.abs(two)).T)
    if ex is not None:
        err = err + ex @ np.abs(one - two).T
    return y, err


def check(d, got):
    out, ids, weights = [v.cpu().numpy() for v in got]
    x = d["x"].cpu().double().numpy()
    wr = d["w_router"].cpu().double().numpy()
    T, model = x.shape
    E, k = wr.shape[0], d["top_k"]
    logit = x @ wr.T
    el = (model * 2.0 ** -24 + 2.0 ** -22) * (np.abs(x) @ np.abs(wr).T)
    assert (np.sort(ids, axis=1)[:, 1:] != np.sort(ids, axis=1)[:, :-1]).all() and ids.min() >= 0 and ids.max() < E
    p = np.exp(logit - logit.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    best = -np.sort(-logit, axis=1)[:, :k]
    assert (np.abs(np.take_along_axis(logit, ids.astype(np.int64), 1) - best) <= 2 * el.max(1, keepdims=True)).all()
    w = np.take_along_axis(p, ids.astype(np.int64), 1)
    ew = w * (2 * el.max(1, keepdims=True) + 2.0 ** -20)
    if d["renorm"]:
        w = w / w.sum(1, keepdims=True)
        ew = 2 * w * (2 * el.max(1, keepdims=True) + 2.0 ** -20)
    assert (np.abs(weights - w) <= ew).all()
    ref = np.zeros_like(x) if d["residual"] is None else d["residual"].cpu().double().numpy().copy()
    tol = np.abs(ref) * 2.0 ** -23
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        gu, egu = product(x[t], d["w_gu"][int(e)])
        gate, up, eg, eu = gu[:, 0::2], gu[:, 1::2], egu[:, 0::2], egu[:, 1::2]
        silu = gate / (1 + np.exp(-gate))
        h = silu * up
        eh = 1.1 * np.abs(up) * eg + (np.abs(silu) + 1.1 * eg) * eu + 2.0 ** -20 * np.abs(h)
        y, ey = product(h, d["w_down"][int(e)], eh)
        ref[t] += w[t, j][:, None] * y
        tol[t] += w[t, j][:, None] * ey + ew[t, j][:, None] * np.abs(y) + (k + 2) * 2.0 ** -23 * w[t, j][:, None] * np.abs(y)
    assert np.isfinite(out).all()
    off = np.abs(out - ref)
    assert (off <= tol).all(), float((off / tol).max())
    # and far inside the bound on the whole
    assert np.linalg.norm(off) <= 1e-5 * np.linalg.norm(ref)


@pytest.mark.parametrize("T,model,ffn,E,top_k,renorm,residual", [
    (1, 256, 256, 1, 1, True, False),
    (1, 2048, 768, 64, 8, True, True),
    (2, 512, 256, 2, 2, False, True),
    (3, 768, 1280, 5, 3, True, False),
    (5, 4352, 512, 8, 1, False, False),       # more super-blocks than are held at once
    (7, 1024, 4608, 4, 2, True, True),
    (16, 1024, 512, 64, 6, False, False),
    (32, 512, 768, 8, 2, True, True),
    (33, 256, 512, 3, 3, False, True),        # every token in every expert
    (64, 512, 256, 4, 1, True, False),
    (64, 256, 256, 256, 8, True, True),
])
def test_values(T, model, ffn, E, top_k, renorm, residual):
    mmq = require_gpu()
    d = make(T, model, ffn, E, top_k, renorm, residual, 500 + T)
    check(d, call(mmq, d))
    assert mmq.status() == 0


def test_all_tokens_to_one_expert_and_ties():
    mmq = require_gpu()
    d = make(21, 512, 512, 6, 2, True, False, 3)
    d["w_router"][:] = 0                      # every expert ties: the lowest two, half the weight each
    out, ids, weights = call(mmq, d)
    assert (ids.cpu() == torch.tensor([0, 1], dtype=torch.int32)).all() and (weights == 0.5).all()
    one = call(mmq, dict(d, w_router=d["w_router"].clone(), renorm=False))[2]
    assert torch.allclose(one, torch.full_like(one, 1 / 6), rtol=1e-6)


def test_activations_of_any_size():
    """Tokens from the smallest normal numbers to near the largest that the
    formula itself carries in f32; each is as exact as the others."""
    mmq = require_gpu()
    d = make(6, 512, 256, 4, 2, True, False, 5, spread=0.0)
    base = d["x"][0].clone()
    for i, s in enumerate((1.0, 2.0 ** -100, 2.0 ** -60, 2.0 ** 30, 2.0 ** 20, 2.0 ** -140)):
        d["x"][i] = base * s
    d["w_router"][:] = 0                      # equal weights for experts 0 and 1
    out = call(mmq, d)[0].double().cpu().numpy()
    x = d["x"].double().cpu().numpy()
    ref, scale = np.zeros_like(x), np.zeros_like(x)
    for e in (0, 1):
        gu, _ = product(x, d["w_gu"][e])
        gate, up = gu[:, 0::2], gu[:, 1::2]
        with np.errstate(over="ignore"):
            h = gate / (1 + np.exp(-gate)) * up
        one, two = fields(d["w_down"][e])
        ref += 0.5 * (h @ (one - two).T)
        scale += 0.5 * (np.abs(h) @ (one + two).T)
    # tokens whose values stay normal f32 numbers throughout
    for i in (0, 2, 3, 4):
        assert (np.abs(out[i] - ref[i]) <= 1e-5 * scale[i].max()).all(), i
    assert np.isfinite(out).all()
    zero = call(mmq, dict(d, x=torch.zeros_like(d["x"])))[0]
    assert (zero == 0).all()


def test_nan_and_inf_stay_in_their_token():
    mmq = require_gpu()
    d = make(9, 512, 512, 8, 2, True, True, 7)
    clean = [v.clone() for v in call(mmq, d)]
    d["x"][3, 100] = float("nan")
    d["x"][6, 5] = float("inf")
    out, ids, weights = call(mmq, d)
    assert torch.isnan(out[3]).all() and torch.isnan(out[6]).all()
    assert int(ids.min()) >= 0 and int(ids.max()) < 8
    keep = [0, 1, 2, 4, 5, 7, 8]
    assert torch.equal(ids[keep], clean[1][keep]) and torch.equal(weights[keep], clean[2][keep])
    ok = torch.isclose(out[keep], clean[0][keep], rtol=1e-4, atol=1e-4)
    assert ok.all()


def test_in_place_streams_workspace_and_repeatability():
    mmq = require_gpu()
    d = make(13, 768, 512, 16, 4, True, True, 9)
    first = [v.clone() for v in call(mmq, d)]
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(first, call(mmq, d)))
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res = d["residual"].clone()
    side.wait_stream(torch.cuda.current_stream())
    out, _, _ = call(mmq, dict(d, residual=res), out=res, workspace=ws, stream=side)
    side.synchronize()
    assert out is res and torch.equal(res, first[0])
    with pytest.raises(mmq.MMQError) as e:
        call(mmq, d, workspace=ws[:1024])
    assert e.value.code == mmq.MMQ_ERR_ARG


def test_weights_past_32_bit_offsets():
    """The last expert's bytes start past 2^31."""
    mmq = require_gpu()
    T, model, ffn, E = 2, 4096, 8192, 60
    d = make(T, 256, 256, 2, 1, True, False, 11)
    g = torch.Generator().manual_seed(12)
    per_gu, per_down = 2 * ffn * model // 256 * 144, model * ffn // 256 * 144
    assert per_gu * (E - 1) > 2 ** 31
    d.update(x=torch.randn((T, model), generator=g).cuda(),
             w_gu=torch.zeros((E, 2 * ffn, model // 256, 144), dtype=torch.uint8, device="cuda"),
             w_down=torch.zeros((E, model, ffn // 256, 144), dtype=torch.uint8, device="cuda"),
             w_router=torch.zeros((E, model), device="cuda"))
    d["w_gu"][E - 1] = q4k(g, 2 * ffn, model, 1 / (184 * model ** 0.5))
    d["w_down"][E - 1] = q4k(g, model, ffn, 1 / (184 * ffn ** 0.5))
    d["w_router"][E - 1] = d["x"].sum(0) * 4
    got = call(mmq, d)
    assert (got[1] == E - 1).all()
    check(d, got)


def test_no_tokens():
    mmq = require_gpu()
    d = make(1, 256, 256, 2, 1, True, False, 11)
    out, ids, weights = call(mmq, dict(d, x=d["x"][:0], residual=None))
    assert out.shape == (0, 256) and ids.shape == (0, 1) and weights.shape == (0, 1)
