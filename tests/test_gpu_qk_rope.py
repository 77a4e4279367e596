"""Head norms + rotary positions + cache write against the formulas in 64 bits.

Tolerance per output y = a c - b s (a, b the normed values): one rounding to
the 16-bit type (2^-11 |y| for float16, 2^-8 |y| for bfloat16, and half the
float16 subnormal step 2^-25 absolute), plus the f32 arithmetic: the sum of D
squares is 8 fused steps and at most 5 shuffled adds, then a divide, an
rsqrt (2 ulp), two products and the rotation's two, in all under 24 roundings of 2^-24
relative to |a c| + |b s|.
"""
import numpy as np
import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-6
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
KIND = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(T, hq, hk, D, R, axes, kind, seed, norm=True, ld=None, rows=300, n_slots=None):
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hk) * D
    ld = ld or width
    buf = torch.randn((T, ld), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    n_slots = n_slots or T + 5
    half = R // 2
    parts = [half] if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    angle = torch.rand((rows, max(half, 1)), generator=g)[:, :half] * 6.3
    return dict(T=T, hq=hq, hk=hk, D=D, R=R, axes=axes, kind=kind, parts=parts, buf=buf.cuda(), width=width,
                cos=angle.cos().contiguous().cuda(), sin=angle.sin().contiguous().cuda(),
                pos=torch.randint(0, rows, (axes, T), generator=g).to(torch.int32).cuda(),
                slots=torch.randperm(n_slots, generator=g)[:T].to(torch.int32).cuda(),
                kc=torch.full((n_slots, hk, D), 3.0, dtype=KIND[kind]).cuda(),
                vc=torch.full((n_slots, hk, D), 5.0, dtype=KIND[kind]).cuda(),
                qw=(torch.rand(D, generator=g) + 0.5).cuda() if norm else None,
                kw=(torch.rand(D, generator=g) - 0.5).cuda() if norm else None)


def call(mmq, d, inter=False, **more):
    return mmq.qk_norm_rope(d["buf"][:, :d["width"]], d["hq"], d["cos"], d["sin"],
                            d["pos"] if d["axes"] > 1 else d["pos"][0], d["slots"], d["kc"], d["vc"],
                            q_weight=d["qw"], k_weight=d["kw"], eps=EPS, interleaved=inter, sections=d["parts"], **more)


def reference(d, inter):
    """(values, sum of magnitudes) of every head in 64 bits, pair by pair."""
    x = d["buf"][:, :d["width"]].cpu().double().numpy().reshape(d["T"], -1, d["D"])
    hq, hk, R = d["hq"], d["hk"], d["R"]
    x = x.copy()
    for lo, n, w in ((0, hq, d["qw"]), (hq, hk, d["kw"])):
        if w is not None:
            part = x[:, lo:lo + n]
            part *= w.cpu().double().numpy() / np.sqrt((part ** 2).mean(-1, keepdims=True) + EPS)
    y, mag = x.copy(), np.abs(x)
    cos, sin, pos = d["cos"].cpu().double().numpy(), d["sin"].cpu().double().numpy(), d["pos"].cpu().numpy()
    axis = np.repeat(np.arange(d["axes"]), d["parts"])
    for j in range(R // 2):
        ia, ib = (2 * j, 2 * j + 1) if inter else (j, j + R // 2)
        c, s = cos[pos[axis[j]], j][:, None], sin[pos[axis[j]], j][:, None]
        a, b = x[:, :hq + hk, ia], x[:, :hq + hk, ib]
        y[:, :hq + hk, ia], y[:, :hq + hk, ib] = a * c - b * s, a * s + b * c
        mag[:, :hq + hk, ia], mag[:, :hq + hk, ib] = abs(a * c) + abs(b * s), abs(a * s) + abs(b * c)
    return y, mag


def near(got, y, mag, kind):
    got = got.cpu().double().numpy()
    assert np.isfinite(got).all()
    tol = ULP[kind] * np.abs(y) * (1 + 2.0 ** -8) + 24 * 2.0 ** -24 * mag + 2.0 ** -25
    assert (np.abs(got - y) <= tol).all(), float((np.abs(got - y) / tol).max())


def check(d, q, inter):
    y, mag = reference(d, inter)
    hq, hk = d["hq"], d["hk"]
    near(q, y[:, :hq], mag[:, :hq], d["kind"])
    at = d["slots"].long().cpu()
    kept = (at >= 0).numpy()
    sel = at[kept]
    near(d["kc"].cpu()[sel], y[kept, hq:hq + hk], mag[kept, hq:hq + hk], d["kind"])
    near(d["vc"].cpu()[sel], y[kept, hq + hk:], mag[kept, hq + hk:], d["kind"])
    other = np.setdiff1d(np.arange(d["kc"].shape[0]), sel.numpy())
    assert (d["kc"].cpu()[other] == 3).all() and (d["vc"].cpu()[other] == 5).all()


@pytest.mark.parametrize("T,hq,hk,D,R,axes,inter,kind,norm", [
    (1, 1, 1, 16, 16, 1, False, "f16", True),
    (1, 32, 8, 128, 128, 1, False, "f16", True),
    (3, 5, 1, 64, 64, 1, True, "bf16", True),
    (7, 8, 2, 128, 64, 1, False, "bf16", False),
    (5, 3, 3, 80, 80, 1, False, "f16", True),
    (5, 4, 2, 96, 48, 2, True, "f16", True),
    (6, 2, 2, 256, 256, 3, False, "bf16", True),
    (9, 28, 4, 128, 128, 3, False, "f16", True),
    (4, 6, 2, 72, 40, 4, False, "f16", False),
    (2, 70, 1, 256, 8, 1, True, "f16", True),
    (131, 32, 32, 128, 128, 1, True, "bf16", True),
])
def test_values(T, hq, hk, D, R, axes, inter, kind, norm):
    mmq = require_gpu()
    d = make(T, hq, hk, D, R, axes, kind, 100 + T, norm)
    q = call(mmq, d, inter)
    assert mmq.status() == 0
    check(d, q, inter)


@pytest.mark.parametrize("first,second", [(0, 64), (13, 51), (62, 2)])
def test_sections_that_split_a_lane(first, second):
    mmq = require_gpu()
    d = make(11, 4, 2, 128, 128, 2, "f16", 7)
    d["parts"] = [first, second]
    q = call(mmq, d)
    assert mmq.status() == 0
    check(d, q, False)


def test_strided_rows_uncached_tokens_and_another_stream():
    mmq = require_gpu()
    d = make(37, 6, 2, 64, 64, 1, "f16", 3, ld=(6 + 4) * 64 + 36)
    d["slots"][::3] = -1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = call(mmq, d, stream=side)
    side.synchronize()
    assert mmq.status() == 0
    check(d, q, False)


def test_no_rotation_and_zero_rows():
    mmq = require_gpu()
    d = make(4, 3, 1, 64, 0, 1, "f16", 5)
    d["buf"][2] = 0
    q = call(mmq, d)
    assert mmq.status() == 0
    check(d, q, False)
    assert (q[2] == 0).all()


def test_no_tokens():
    mmq = require_gpu()
    d = make(1, 3, 1, 64, 64, 1, "f16", 5)
    d.update(buf=d["buf"][:0], pos=d["pos"][:, :0].contiguous(), slots=d["slots"][:0])
    assert call(mmq, d).shape == (0, 3, 64)
    assert (d["kc"] == 3).all() and mmq.status() == 0


def test_nan_stays_in_its_head():
    mmq = require_gpu()
    d = make(3, 4, 2, 128, 128, 1, "f16", 9)
    clean = call(mmq, d).clone()
    d["buf"][1, 2 * 128 + 5] = float("nan")
    d["buf"][2, 3 * 128 + 7] = float("inf")
    q = call(mmq, d)
    bad = torch.isnan(q).any(-1)
    assert bad.nonzero().tolist() == [[1, 2], [2, 3]]
    assert torch.equal(q[~bad], clean[~bad])


def test_slot_past_32_bit_offsets():
    mmq = require_gpu()
    d = make(2, 4, 8, 128, 128, 1, "f16", 11)
    n = 2_300_000   # 2.3e6 slots of 1024 values: offsets pass 2^31
    d["kc"] = torch.empty((n, 8, 128), dtype=torch.float16, device="cuda")
    d["vc"] = torch.empty((n, 8, 128), dtype=torch.float16, device="cuda")
    d["slots"] = torch.tensor([n - 1, 2_100_000], dtype=torch.int32, device="cuda")
    call(mmq, d)
    assert mmq.status() == 0
    y, mag = reference(d, False)
    at = d["slots"].long()
    near(d["kc"][at], y[:, 4:12], mag[:, 4:12], "f16")
    near(d["vc"][at], y[:, 12:], mag[:, 12:], "f16")


def test_positions_and_slots_out_of_range_are_reported_and_write_nothing():
    mmq = require_gpu()
    for what in ("position", "negative", "slot"):
        d = make(5, 4, 2, 128, 128, 2, "bf16", 13)
        if what == "slot":
            d["slots"][3] = d["kc"].shape[0]
        else:
            d["pos"][1, 3] = -1 if what == "negative" else d["cos"].shape[0]
        good = [0, 1, 2, 4]
        q = call(mmq, d)
        assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
        assert bool(torch.isnan(q[3]).all()) == (what != "slot")
        assert not torch.isnan(q[good]).any()
        touched = (d["kc"] != 3).any(-1).any(-1).nonzero().flatten().tolist()
        assert sorted(touched) == sorted(d["slots"][good].tolist())


def test_runs_are_bit_identical():
    mmq = require_gpu()
    d = make(65, 8, 4, 128, 128, 3, "bf16", 17)
    a = call(mmq, d).clone()
    ka = d["kc"].clone()
    b = call(mmq, d)
    assert torch.equal(a, b) and torch.equal(ka, d["kc"])
