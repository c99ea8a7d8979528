"""4-bit experts on the GPU against plain 64-bit forms (tests/_w4_ref.py).

Weights: exactly (q - z) s, or that rounded to bf16 (moe_w4_t allows both; with few rows per expert the products
run on the codes, with many on bf16 weights): a result has to agree with one of the two throughout.  Token rows
enter the products of codes rounded to 2^-15 of the largest value of their group (2^-23 for fp32 outputs).

Tolerances, counted before the first run: an output rounded to bf16 is off by 2^-8 of its value (half a step), one
in fp32 by 2^-24; sums by acc_bound (an fp32 step per addition); SwiGLU carries its two sums' errors on.
"""
import pytest
import torch

import _w4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import moe_layer_forward_b200 as m

    return m


def weights(gen, E, n, k, group, zero, few_bits=False):
    """A random 4-bit matrix on the CPU; few_bits: scales of 4 significant bits, as the quantiser gives."""
    G = -(-k // group)
    q = ref.pack(torch.randint(0, 16, (E, n, k), generator=gen))
    s = (0.5 + torch.rand((E, G, n), generator=gen)) * 0.4 / k ** 0.5
    if few_bits:
        s = (s.view(torch.int32) & ~0xFFFFF).view(F32)
    z = torch.randint(0, 16, (E, G, n), generator=gen, dtype=torch.uint8) if zero else None
    return q, s.to(BF), z, group


def put(moe, w):
    q, s, z, group = w
    return moe.W4Weights(q.to(DEV), s.to(DEV), None if z is None else z.to(DEV), group)


def segments(counts, gap=0):
    off, at = [], 0
    for c in counts:
        off.append(at)
        at += c + gap
    return torch.tensor(counts, dtype=torch.int32), torch.tensor(off + [at], dtype=torch.int32), at


# ------------------------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("E,n,k", [(1, 1, 32), (2, 33, 96), (3, 40, 288), (1, 7, 544), (2, 64, 1024)])
def test_quantize_is_exact(moe, E, n, k, group, dt, zero):
    gen = torch.Generator().manual_seed(E * n + k)
    x = torch.randn((E, n, k), generator=gen)
    x[:, ::3] *= 2.0 ** -40
    x[:, 1::4] = (x[:, 1::4] * 4).round() / 4  # quotients on the borders between two codes
    x[0, 0, :32] = 0
    x[-1, -1, -32:] = x[-1, -1, -32:].abs() + 1  # one sign only
    x = x.to(dt)
    got = moe.quantize_w4_weights(x.to(DEV), group=group, zero=zero)
    codes, s, z = ref.quantize(x, group, zero)
    assert torch.equal(got.s.cpu().double(), s)
    if zero:
        assert torch.equal(got.z.cpu().long(), z)
    assert torch.equal(ref.unpack(got.q.cpu()), codes)
    assert torch.equal(moe.unpack_w4(got.q).cpu().long(), codes) and torch.equal(moe.pack_w4(moe.unpack_w4(got.q)), got.q)
    # the weights are bf16 exactly, and within half a step of x (7 s >= max, so nothing is cut off beyond rounding z)
    w = ref.dequant(got.q.cpu(), got.s.cpu(), got.z.cpu() if zero else None, group, rounded=False)
    assert torch.equal(w.float().to(BF).double(), w)
    step = got.s.cpu().double().transpose(1, 2)[..., torch.arange(k) // group]
    assert ((w - x.double()).abs() <= step * (1.0 if zero else 0.5)).all()
    for out_dt in (F32, BF):
        out = torch.empty((E, n, k), dtype=out_dt, device=DEV)
        moe.moe_dequantize_w4(got, out)
        assert torch.equal(out.cpu().double(), w)


def test_quantize_groups_that_are_not_finite(moe):
    x = torch.randn((1, 4, 256))
    x[0, 0, 3], x[0, 1, 130], x[0, 2, 0], x[0, 3, 255] = float("nan"), float("inf"), -float("inf"), 2.0 ** 120
    for zero in (False, True):
        w = moe.quantize_w4_weights(x.to(DEV), group=128, zero=zero)
        bad = torch.isnan(w.s.float().cpu())[0]  # [G][n]
        assert bad.tolist() == [[True, False, True, False], [False, True, False, True]]


def test_quantize_smallest_scales(moe):
    x = torch.full((1, 2, 32), 2.0 ** -130)
    x[0, 1] = 7 * 2.0 ** -100
    w = moe.quantize_w4_weights(x.to(DEV), group=32)
    assert w.s.float().cpu().flatten().tolist() == [2.0 ** -100, 2.0 ** -100]
    assert ref.unpack(w.q.cpu())[0, :, 0].tolist() == [8, 15]


def test_dequantize_rounds_scales_of_many_bits(moe):
    gen = torch.Generator().manual_seed(3)
    w = weights(gen, 2, 40, 160, 64, True)
    out = torch.empty((2, 40, 160), dtype=BF, device=DEV)
    moe.moe_dequantize_w4(put(moe, w), out)
    assert torch.equal(out.cpu().double(), ref.dequant(*w))


# ------------------------------------------------------------------------------------------------ grouped products
COUNTS = {
    "one_row": [0, 0, 1, 0],
    "few": [0, 1, 3, 8, 9, 0, 2, 5],
    "passes": [17, 0, 40, 1],
    "empty": [0, 0, 0],
    "many": [130, 0, 64, 257, 3, 16],
    "large": [500, 129, 300],
    "wide": [192, 120, 193, 130],
    "widest": [400, 385, 577],
}


@pytest.mark.parametrize("case", list(COUNTS))
@pytest.mark.parametrize("d,f,group,zero", [(32, 32, 32, False), (256, 128, 128, False), (352, 224, 64, True),
                                            (736, 416, 128, True), (1056, 96, 32, True), (160, 1120, 64, False)])
def test_grouped_swiglu(moe, case, d, f, group, zero):
    counts = COUNTS[case]
    gen = torch.Generator().manual_seed(d + f)
    E = len(counts)
    ct, off, S = segments(counts, gap=1)
    S = max(S, 1)
    Wg, Wu, Wd = (weights(gen, E, f, d, group, zero), weights(gen, E, f, d, group, zero),
                  weights(gen, E, d, f, group, zero))
    x = torch.randn((S, d), generator=gen).to(BF)
    h = torch.full((S, f), 77.0, dtype=BF, device=DEV)
    y = torch.full((S, d), 77.0, dtype=BF, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grouped_swiglu_w4(x.to(DEV), put(moe, Wg), put(moe, Wu), put(moe, Wd), ct.to(DEV), off.to(DEV), h, y,
                              dev_status=status)
    assert status.item() == 0
    h, y = h.cpu().double(), y.cpu().double()
    inside = torch.zeros(S, dtype=torch.bool)
    for e, n in enumerate(counts):
        inside[int(off[e]):int(off[e]) + n] = True
    assert (h[~inside] == 77).all() and (y[~inside] == 77).all()

    def right(wg, wu, wd):
        ok_h = ok_y = True
        for e, n in enumerate(counts):
            o = int(off[e])
            if n == 0:
                continue
            hr, dh = ref.gate_up(x[o:o + n].double(), wg[e], wu[e], group)
            ok_h &= ref.within(h[o:o + n], hr, dh, 2.0 ** -8)
            # from the kernel's own h: only this product's errors
            ok_y &= ref.within(y[o:o + n], h[o:o + n] @ wd[e].T, ref.product_bound(h[o:o + n], wd[e], group), 2.0 ** -8)
        return ok_h, ok_y

    assert (True, True) in [right(*w) for w in ref.readings(Wg, Wu, Wd)]


def test_grouped_wide_rows_take_several_passes(moe):
    # rows so long that shared memory holds a few of them at a time
    gen = torch.Generator().manual_seed(5)
    d, f, counts = 16384, 64, [3, 0, 5]
    ct, off, S = segments(counts)
    Wg, Wu = weights(gen, 3, f, d, 128, False), weights(gen, 3, f, d, 128, False)
    Wd = weights(gen, 3, f, d, 128, True)
    x = torch.randn((S, d), generator=gen).to(BF)
    h = torch.empty((S, f), dtype=BF, device=DEV)
    y = torch.empty((S, f), dtype=BF, device=DEV)
    moe.moe_expert_gate_up_w4(x.to(DEV), put(moe, Wg), put(moe, Wu), ct.to(DEV), off.to(DEV), h)
    moe.moe_expert_down_w4(x.to(DEV), put(moe, Wd), ct.to(DEV), off.to(DEV), y)
    h, y = h.cpu().double(), y.cpu().double()

    def right(wg, wu, wd):
        ok = True
        for e, n in enumerate(counts):
            o = int(off[e])
            if n:
                xr = x[o:o + n].double()
                hr, dh = ref.gate_up(xr, wg[e], wu[e], 128)
                ok &= ref.within(h[o:o + n], hr, dh, 2.0 ** -8)
                ok &= ref.within(y[o:o + n], xr @ wd[e].T, ref.product_bound(xr, wd[e], 128), 2.0 ** -8)
        return ok

    assert any(right(*w) for w in ref.readings(Wg, Wu, Wd))


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts", [[3, 2], [70, 200]])
def test_grouped_scales_of_every_size(moe, counts, group, zero):
    """Scales far from 1, of either sign, zero, and of many or few bits beside one another."""
    gen = torch.Generator().manual_seed(group)
    ct, off, S = segments(counts)
    f, d = 416, 96
    q, s, z, _ = weights(gen, 2, d, f, group, zero)
    s = s.float()
    s[0, 0, 0:8] = torch.tensor([2.0 ** 11, 2.0 ** 20, -3.0, 0.0, 2.0 ** -110, 2.0 ** -60, 1.9921875 * 2 ** 10, -0.0])
    s[1] = (s[1].view(torch.int32) & ~0xFFFFF).view(F32)  # an expert whose scales have 4 significant bits
    s[1, :, 5] = -s[1, :, 5]
    Wd = (q, s.to(BF), z, group)
    x = torch.randn((S, f), generator=gen).to(BF)
    y = torch.empty((S, d), dtype=BF, device=DEV)
    moe.moe_expert_down_w4(x.to(DEV), put(moe, Wd), ct.to(DEV), off.to(DEV), y)
    y = y.cpu().double()

    def right(w):
        ok = True
        for e, n in enumerate(counts):
            o = int(off[e])
            xr = x[o:o + n].double()
            ok &= ref.within(y[o:o + n], xr @ w[e].T, ref.product_bound(xr, w[e], group), 2.0 ** -8)
        return ok

    assert any(right(*m) for m in ref.readings(Wd))


def test_grouped_long_rows_many_of_them(moe):
    gen = torch.Generator().manual_seed(15)
    d, f, counts = 16384, 32, [40, 0, 90]
    ct, off, S = segments(counts)
    Wg, Wu = weights(gen, 3, f, d, 128, True), weights(gen, 3, f, d, 128, True)
    x = torch.randn((S, d), generator=gen).to(BF)
    h = torch.empty((S, f), dtype=BF, device=DEV)
    moe.moe_expert_gate_up_w4(x.to(DEV), put(moe, Wg), put(moe, Wu), ct.to(DEV), off.to(DEV), h)
    h = h.cpu().double()

    def right(wg, wu):
        ok = True
        for e, n in enumerate(counts):
            o = int(off[e])
            if n:
                hr, dh = ref.gate_up(x[o:o + n].double(), wg[e], wu[e], 128)
                ok &= ref.within(h[o:o + n], hr, dh, 2.0 ** -8)
        return ok

    assert any(right(*m) for m in ref.readings(Wg, Wu))


@pytest.mark.parametrize("counts,S", [([0, 0], 200), ([0] * 256, 256), ([1] * 256, 256), ([300], 300), ([1], 1),
                                      ([0, 0, 0, 1], 2000), ([40] * 5, 4000)])
def test_grouped_extremes_of_experts_and_rows(moe, counts, S):
    """One expert and 256, none of the buffers' rows used, or few of many."""
    gen = torch.Generator().manual_seed(S)
    ct, off, used = segments(counts)
    E, d, f = len(counts), 64, 96
    W = [weights(gen, E, n, k, 32, True) for n, k in ((f, d), (f, d), (d, f))]
    x = torch.randn((S, d), generator=gen).to(BF)
    h, y = torch.full((S, f), 9.0, dtype=BF, device=DEV), torch.full((S, d), 9.0, dtype=BF, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grouped_swiglu_w4(x.to(DEV), *[put(moe, m) for m in W], ct.to(DEV), off.to(DEV), h, y, dev_status=status)
    assert status.item() == 0
    h, y = h.cpu().double(), y.cpu().double()
    assert (h[used:] == 9).all() and (y[used:] == 9).all()

    def right(wg, wu, wd):
        ok = True
        for e, n in enumerate(counts):
            if n:
                r = slice(int(off[e]), int(off[e]) + n)
                hr, dh = ref.gate_up(x[r].double(), wg[e], wu[e], 32)
                ok &= ref.within(h[r], hr, dh, 2.0 ** -8)
                ok &= ref.within(y[r], h[r] @ wd[e].T, ref.product_bound(h[r], wd[e], 32), 2.0 ** -8)
        return ok

    assert any(right(*m) for m in ref.readings(*W))


def test_grouped_waits_that_run_out(moe):
    """As for the other tensor-core kernels: a stalled wait gives up, is reported, and the next call is right."""
    gen = torch.Generator().manual_seed(16)
    E, per, d, f = 4, 50, 256, 128
    ct, off, S = segments([per] * E)
    W = [put(moe, weights(gen, E, n, k, 64, True)) for n, k in ((f, d), (f, d), (d, f))]
    x, ct, off = torch.randn((S, d), generator=gen).to(BF).to(DEV), ct.to(DEV), off.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(st=None):
        h, y = torch.zeros((S, f), dtype=BF, device=DEV), torch.zeros((S, d), dtype=BF, device=DEV)
        moe.moe_grouped_swiglu_w4(x, *W, ct, off, h, y, dev_status=st)
        return h, y

    first = call()
    torch.cuda.synchronize()
    moe.set_wait_limit(2_000_000, inject_stall=True)
    try:
        call(status)
    finally:
        moe.set_wait_limit(0, inject_stall=False)
    torch.cuda.synchronize()
    assert status.item() & moe.MOE_DEV_TIMEOUT
    again = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("counts", [[3, 5, 2, 9], [40, 150, 2, 300]])
def test_grouped_rows_do_not_mix(moe, counts):
    """A row of NaN, infinities or huge values changes nothing but its own outputs; a NaN scale only its columns."""
    gen = torch.Generator().manual_seed(6)
    ct, off, S = segments(counts)
    d, f = 288, 160
    Wg, Wu, Wd = weights(gen, 4, f, d, 64, True), weights(gen, 4, f, d, 64, True), weights(gen, 4, d, f, 32, False)
    x = torch.randn((S, d), generator=gen).to(BF)

    def go(x, Wd):
        h = torch.empty((S, f), dtype=BF, device=DEV)
        y = torch.empty((S, d), dtype=BF, device=DEV)
        moe.moe_expert_gate_up_w4(x.to(DEV), put(moe, Wg), put(moe, Wu), ct.to(DEV), off.to(DEV), h)
        moe.moe_expert_down_w4(h, put(moe, Wd), ct.to(DEV), off.to(DEV), y)
        return h.cpu(), y.cpu()

    h0, y0 = go(x, Wd)
    bad = x.clone()
    rows = [0, 4, S - 1]
    bad[0, 7], bad[4, 0], bad[S - 1] = float("nan"), float("inf"), 1e38
    h1, y1 = go(bad, Wd)
    keep = torch.ones(S, dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(h0[keep], h1[keep]) and torch.equal(y0[keep], y1[keep])
    assert torch.isnan(h1[0].float()).all() and torch.isnan(y1[0].float()).all()
    s = Wd[1].clone()
    s[1, 2, 33] = float("nan")
    h2, y2 = go(x, (Wd[0], s, Wd[2], Wd[3]))
    want = torch.zeros((S, d), dtype=torch.bool)
    want[int(off[1]):int(off[1]) + counts[1], 33] = True
    assert torch.equal(torch.isnan(y2.float()), want) and torch.equal(y2[~want], y0[~want])


@pytest.mark.parametrize("counts,offsets,S", [([5, 90], [0, 5], 20), ([-3, 4], [0, 0], 20), ([4, 4], [-2, 10], 20),
                                              ([4, 4], [0, 2000000000], 20), ([300, 300], [0, 290], 310)])
def test_segments_outside_the_buffers_are_cut_and_flagged(moe, counts, offsets, S):
    gen = torch.Generator().manual_seed(7)
    d, f = 64, 96
    W = [weights(gen, 2, f, d, 32, False), weights(gen, 2, f, d, 32, False)]
    x = torch.randn((S, d), generator=gen).to(BF)
    guard = 64
    buf = torch.full((S + guard, f), 5.0, dtype=BF, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ct = torch.tensor(counts, dtype=torch.int32, device=DEV)
    off = torch.tensor(offsets + [0], dtype=torch.int32, device=DEV)
    moe.moe_expert_gate_up_w4(x.to(DEV), put(moe, W[0]), put(moe, W[1]), ct, off, buf[:S], dev_status=status)
    assert status.item() == moe.MOE_DEV_BAD_COUNT
    assert (buf[S:] == 5).all()
    rows = sorted((max(o, 0), min(o + max(c, 0), S), e) for e, (c, o) in enumerate(zip(counts, offsets)))
    covered = torch.zeros(S, dtype=torch.int64)
    for lo, hi, _ in rows:
        covered[min(lo, S):max(min(lo, S), hi)] += 1
    assert (buf[:S].cpu()[covered == 0] == 5).all()
    got = buf[:S].cpu().double()

    def right(wg, wu):
        ok = True
        for lo, hi, e in rows:
            for r in range(min(lo, S), hi):
                if covered[r] == 1:
                    hr, dh = ref.gate_up(x[r:r + 1].double(), wg[e], wu[e], 32)
                    ok &= ref.within(got[r:r + 1], hr, dh, 2.0 ** -8)
        return ok

    assert any(right(*w) for w in ref.readings(*W))


# ------------------------------------------------------------------------------------------------ picks
def picks_reference(x, Wg, Wu, Wd, idx, w, residual, bits):
    """The products run on the codes: weights are exact; rows enter rounded to 2^-bits of their group's largest value."""
    wg, wu, wd = next(ref.readings(Wg, Wu, Wd))
    group = Wg[3]
    E, f = wg.shape[0], wg.shape[1]
    out, tol = residual.double().clone(), residual.double().abs() * 2.0 ** -24
    for t in range(idx.shape[0]):
        for i in range(idx.shape[1]):
            e = int(idx[t, i])
            if not 0 <= e < E:
                continue
            h, dh = ref.gate_up(x[t:t + 1].double(), wg[e], wu[e], group, bits)
            y = (h @ wd[e].T)[0]
            dy = (dh @ wd[e].abs().T + ref.product_bound(h.abs() + dh, wd[e], group, bits))[0]
            out[t] += w[t, i].double() * y
            # the weighted terms are summed in fp32: a step of the magnitudes per addition
            tol[t] += w[t, i].double().abs() * (dy + 16 * 2.0 ** -24 * y.abs())
    return out, tol


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 8), (1, 8, 32), (3, 5, 7), (8, 8, 16), (9, 2, 3), (16, 8, 128),
                                   (32, 8, 9), (256, 1, 256), (100, 2, 2)])
@pytest.mark.parametrize("d,f,group,zero", [(32, 32, 128, False), (256, 128, 32, True), (416, 352, 64, False)])
def test_picks(moe, T, k, E, d, f, group, zero):
    gen = torch.Generator().manual_seed(T + k + E + d)
    Wg, Wu, Wd = (weights(gen, E, f, d, group, zero), weights(gen, E, f, d, group, zero),
                  weights(gen, E, d, f, group, zero))
    v = torch.randn((T, d), generator=gen).to(BF)
    idx = torch.stack([torch.randperm(E, generator=gen)[:k] if k <= E else torch.randint(0, E, (k,), generator=gen)
                       for _ in range(T)]).to(torch.int32)
    w = torch.rand((T, k), generator=gen)
    dev = [put(moe, m) for m in (Wg, Wu, Wd)]
    for dt in (F32, BF):
        residual = torch.randn((T, d), generator=gen).to(dt)
        out = torch.full((T, d), 99.0, dtype=dt, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_picks_swiglu_w4(v.to(DEV), *dev, idx.to(DEV), w.to(DEV), residual.to(DEV), out, dev_status=status)
        assert status.item() == 0
        want, tol = picks_reference(v, Wg, Wu, Wd, idx, w, residual, 23 if dt == F32 else 15)
        half = 2.0 ** -24 if dt == F32 else 2.0 ** -8
        assert ((out.cpu().double() - want).abs() <= tol + half * (want.abs() + tol)).all()
        # in place, and the same bits again
        same = residual.to(DEV).clone()
        moe.moe_picks_swiglu_w4(v.to(DEV), *dev, idx.to(DEV), w.to(DEV), same, same)
        assert torch.equal(same, out)


def test_picks_bad_ids_and_an_expert_named_twice(moe):
    gen = torch.Generator().manual_seed(9)
    T, k, E, d, f = 3, 4, 5, 96, 64
    Wg, Wu, Wd = weights(gen, E, f, d, 32, True), weights(gen, E, f, d, 32, True), weights(gen, E, d, f, 32, True)
    v = torch.randn((T, d), generator=gen).to(BF)
    residual = torch.randn((T, d), generator=gen)
    w = torch.rand((T, k), generator=gen)
    idx = torch.tensor([[0, 0, 0, 0], [1, -1, 5, 1], [-7, 2147483647, 5, 99]], dtype=torch.int32)
    out = torch.empty((T, d), device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_picks_swiglu_w4(v.to(DEV), put(moe, Wg), put(moe, Wu), put(moe, Wd), idx.to(DEV), w.to(DEV), residual.to(DEV),
                            out, dev_status=status)
    assert status.item() == moe.MOE_DEV_BAD_EXPERT_ID
    want, tol = picks_reference(v, Wg, Wu, Wd, idx, w, residual, 23)
    assert ((out.cpu().double() - want).abs() <= tol + 2.0 ** -24 * (want.abs() + tol)).all()
    assert torch.equal(out[2].cpu(), residual[2])  # no valid pick: the residual alone


def test_picks_workspace_is_not_read_before_written(moe):
    gen = torch.Generator().manual_seed(10)
    T, k, E, d, f = 5, 3, 11, 160, 224
    dev = [put(moe, weights(gen, E, n, m, 64, True)) for n, m in ((f, d), (f, d), (d, f))]
    v = torch.randn((T, d), generator=gen).to(BF).to(DEV)
    idx = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).to(torch.int32).to(DEV)
    w, res = torch.rand((T, k), generator=gen).to(DEV), torch.randn((T, d), generator=gen).to(DEV)
    n = moe.picks_w4_workspace_bytes(v, dev[0], dev[2], idx)
    outs = []
    for fill in (0, 255):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device=DEV)
        out = torch.empty((T, d), device=DEV)
        moe.moe_picks_swiglu_w4(v, *dev, idx, w, res, out, ws=ws[:n])
        assert (ws[n:] == fill).all()
        outs.append(out)
    assert torch.equal(*outs)


# ------------------------------------------------------------------------------------------------ the layer
LAYERS = [
    # T, d, E, f, k, group, zero, x, out
    (1, 256, 32, 128, 8, 32, True, F32, F32),
    (1, 512, 16, 96, 2, 128, False, BF, BF),
    (7, 160, 9, 352, 3, 64, False, BF, F32),
    (40, 256, 32, 160, 4, 128, True, F32, BF),
    (128, 384, 64, 128, 8, 128, False, BF, BF),
    (600, 256, 16, 192, 4, 64, True, BF, BF),
    (1500, 128, 8, 256, 8, 32, False, F32, F32),
]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: f"T{c[0]}_E{c[2]}")
def test_forward(moe, case):
    T, d, E, f, k, group, zero, xd, od = case
    gen = torch.Generator().manual_seed(T + d)
    Wg, Wu, Wd = (weights(gen, E, f, d, group, zero), weights(gen, E, f, d, group, zero),
                  weights(gen, E, d, f, group, zero))
    x = torch.randn((T, d), generator=gen).to(xd).to(DEV)
    gamma = (1 + 0.1 * torch.randn(d, generator=gen)).to(DEV)
    W_r = (torch.randn((E, d), generator=gen) / d ** 0.5).to(DEV)
    b = (0.1 * torch.randn(E, generator=gen)).to(DEV)
    out = torch.empty((T, d), dtype=od, device=DEV)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    logits = torch.empty((T, E), device=DEV)
    status = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    dev = [put(moe, m) for m in (Wg, Wu, Wd)]
    moe.moe_forward_w4(x, gamma, W_r, b, *dev, out, top_k=k, topk_idx=idx, topk_w=w, logits=logits, dev_status=status)
    assert status.item() == 0
    # the routing is the layer's own, bit for bit
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    moe.moe_route(x, gamma, W_r, b, i2, w2)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    v = torch.empty((T, d), dtype=BF, device=DEV)
    moe.moe_rmsnorm(x, gamma, 1e-5, v)
    half = 2.0 ** -24 if od == F32 else 2.0 ** -8
    ok = False
    for m in ref.readings(Wg, Wu, Wd):
        want, tol = layer_reference(v.cpu(), *m, idx.cpu(), w.cpu(), x.cpu(), group, not picks_form(T, k, E, group), od)
        ok |= ref.within(out.cpu().double(), want, tol, half)
    assert ok


def picks_form(T, k, E, group):
    """Whether the layer carries h and y in fp32 (the form for few tokens)."""
    return T * k <= 256 and T * k <= {128: 6, 64: 3, 32: 1}[group] * E


def layer_reference(v, wg, wu, wd, idx, w, residual, group, rounded, od):
    """As picks_reference, by expert; rounded: h and y are rounded to bf16 on the way."""
    bits = 23 if od == F32 and not rounded else 15
    out, tol = residual.double().clone(), residual.double().abs() * 2.0 ** -24
    for e in range(wg.shape[0]):
        t, i = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h, dh = ref.gate_up(v[t].double(), wg[e], wu[e], group, bits)
        if rounded:
            dh = dh + 2.0 ** -8 * (h.abs() + dh)
        y = h @ wd[e].T
        dy = dh @ wd[e].abs().T + ref.product_bound(h.abs() + dh, wd[e], group, bits)
        if rounded:
            dy = dy + 2.0 ** -8 * (y.abs() + dy)
        ww = w[t, i].double()[:, None]
        out.index_add_(0, t, ww * y)
        tol.index_add_(0, t, ww.abs() * (dy + 16 * 2.0 ** -24 * y.abs()))
    return out, tol


def test_forward_no_tokens(moe):
    gen = torch.Generator().manual_seed(1)
    dev = [put(moe, weights(gen, 4, n, m, 32, False)) for n, m in ((64, 96), (64, 96), (96, 64))]
    x = torch.empty((0, 96), device=DEV)
    status = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    moe.moe_forward_w4(x, torch.ones(96, device=DEV), torch.zeros((4, 96), device=DEV), torch.zeros(4, device=DEV), *dev,
                       torch.empty_like(x), top_k=2, dev_status=status)
    assert status.item() == 0


def _layer_call(moe, gen, T, d, E, f, k, group=64):
    dev = [put(moe, weights(gen, E, n, m, group, True)) for n, m in ((f, d), (f, d), (d, f))]
    x = torch.randn((T, d), generator=gen).to(BF).to(DEV)
    args = (torch.ones(d, device=DEV), (torch.randn((E, d), generator=gen) / d ** 0.5).to(DEV), torch.zeros(E, device=DEV))
    out = torch.zeros((T, d), dtype=BF, device=DEV)
    n = moe.forward_w4_workspace_bytes(x, dev[0], out, k)
    return x, out, n, lambda ws, st=None: moe.moe_forward_w4(x, *args, *dev, out, top_k=k, ws=ws, dev_status=st)


@pytest.mark.parametrize("T", [2, 60, 400])
def test_forward_on_another_stream_and_captured(moe, T):
    gen = torch.Generator().manual_seed(T)
    x, out, n, call = _layer_call(moe, gen, T, 256, 12, 128, 4)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    call(ws)
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(ws)
    side.synchronize()
    assert torch.equal(out, want)
    # a replay takes new inputs from the same buffers; two graphs in order share one workspace
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(ws)
        graphs.append(g)
    out.zero_()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.copy_(x.flip(0))
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    out.zero_()
    call(ws)
    torch.cuda.synchronize()
    assert torch.equal(out, replayed) and not torch.equal(out, want)


@pytest.mark.parametrize("tokens", [(3, 200), (2, 3), (1, 8, 60, 300)])
def test_calls_at_once_with_their_own_workspaces(moe, tokens):
    """Several streams; the form for few tokens, whose CTAs wait for one another, among them and beside itself."""
    gen = torch.Generator().manual_seed(21)
    calls = [_layer_call(moe, gen, T, 256, 12, 128, 4) for T in tokens]
    ws = [torch.empty(c[2], dtype=torch.uint8, device=DEV) for c in calls]
    want = []
    for c, w in zip(calls, ws):
        c[3](w)
        want.append(c[1].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in tokens]
    for _ in range(10):
        for c, w, s in zip(calls, ws, streams):
            with torch.cuda.stream(s):
                c[3](w)
    torch.cuda.synchronize()
    assert all(torch.equal(c[1], w) for c, w in zip(calls, want))


def test_quantised_experts_agree_with_bf16_experts(moe):
    """The 4-bit layer on quantised weights is the bf16 layer on the weights that the codes stand for."""
    gen = torch.Generator().manual_seed(30)
    T, d, E, f, k = 96, 256, 16, 128, 4
    W = [(torch.randn(s, generator=gen) / s[2] ** 0.5).to(BF).to(DEV) for s in ((E, f, d), (E, f, d), (E, d, f))]
    w4 = [moe.quantize_w4_weights(m, group=64, zero=True) for m in W]
    wb = [torch.empty_like(m) for m in W]
    for a, b in zip(w4, wb):
        moe.moe_dequantize_w4(a, b)
    x = torch.randn((T, d), generator=gen).to(BF).to(DEV)
    args = (torch.ones(d, device=DEV), (torch.randn((E, d), generator=gen) / d ** 0.5).to(DEV), torch.zeros(E, device=DEV))
    o4, ob = torch.empty_like(x), torch.empty_like(x)
    moe.moe_forward_w4(x, *args, *w4, o4, top_k=k)
    moe.moe_forward(x, *args, *wb, ob, top_k=k)
    # both round h, y and the output to bf16: two half steps of each, at most
    scale = (ob.float() - x.float()).abs().max().item() + x.float().abs().max().item()
    assert (o4.float() - ob.float()).abs().max().item() <= 3 * 2.0 ** -8 * 2 * scale
    assert ((o4 - ob).float().norm() / ob.float().norm()).item() < 2.0 ** -8


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals(moe):
    gen = torch.Generator().manual_seed(2)
    E, d, f, S = 3, 96, 64, 6
    Wg, Wu, Wd = (put(moe, weights(gen, E, n, m, 32, True)) for n, m in ((f, d), (f, d), (d, f)))
    x = torch.zeros((S, d), dtype=BF, device=DEV)
    h, y = torch.zeros((S, f), dtype=BF, device=DEV), torch.zeros((S, d), dtype=BF, device=DEV)
    ct = torch.zeros(E, dtype=torch.int32, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    before = moe.kernel_launches()
    bad = [
        (TypeError, lambda: moe.moe_expert_gate_up_w4(x.float(), Wg, Wu, ct, off, h)),
        (ValueError, lambda: moe.moe_expert_gate_up_w4(x, Wg, Wu, ct, off[:E], h)),
        (ValueError, lambda: moe.moe_expert_gate_up_w4(x, Wg, Wu, ct, off, y)),
        (ValueError, lambda: moe.moe_expert_gate_up_w4(x, Wg, Wu._replace(group=64), ct, off, h)),
        (moe.MoEError, lambda: moe.moe_expert_gate_up_w4(x, Wg, Wu._replace(z=None), ct, off, h)),
        (ValueError, lambda: moe.moe_expert_gate_up_w4(x, Wg, Wd, ct, off, h)),
        (ValueError, lambda: moe.moe_expert_down_w4(h, Wd._replace(group=0), ct, off, y)),
        (ValueError, lambda: moe.moe_expert_down_w4(h, Wd._replace(q=Wd.q.cpu()), ct, off, y)),
        (ValueError, lambda: moe.moe_expert_down_w4(h, Wd, ct.cpu(), off, y)),
        (TypeError, lambda: moe.moe_expert_down_w4(h, Wd._replace(s=Wd.s.half()), ct, off, y)),
        (ValueError, lambda: moe.moe_expert_down_w4(h, Wd._replace(z=Wd.z.transpose(1, 2)), ct, off, y)),
        (ValueError, lambda: moe.moe_expert_down_w4(h.t().contiguous().t(), Wd, ct, off, y)),
        (ValueError, lambda: moe.moe_expert_down_w4(h, Wd, ct, off, y, dev_status=torch.zeros(1, dtype=torch.int64, device=DEV))),
        (ValueError, lambda: moe.quantize_w4_weights(torch.zeros((1, 8, 48), device=DEV))),
        (ValueError, lambda: moe.quantize_w4_weights(torch.zeros((1, 8, 64), device=DEV), group=16)),
        (TypeError, lambda: moe.quantize_w4_weights(torch.zeros((1, 8, 64), device=DEV, dtype=torch.float16))),
        (ValueError, lambda: moe.moe_dequantize_w4(Wd, torch.zeros((E, d, f + 32), device=DEV))),
        (ValueError, lambda: moe.moe_picks_swiglu_w4(x, Wg, Wu, Wd, torch.zeros((S, 2), dtype=torch.int32, device=DEV),
                                                     torch.zeros((S, 3), device=DEV), y, y)),
        (moe.MoEError, lambda: moe.moe_picks_swiglu_w4(x, Wg, Wu, Wd, torch.zeros((S, 9), dtype=torch.int32, device=DEV),
                                                       torch.zeros((S, 9), device=DEV), y, y)),
        (moe.MoEError, lambda: moe.moe_picks_swiglu_w4(x, Wg, Wu, Wd, torch.zeros((S, 2), dtype=torch.int32, device=DEV),
                                                       torch.zeros((S, 2), device=DEV), y, y,
                                                       ws=torch.empty(256, dtype=torch.uint8, device=DEV))),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    assert moe.kernel_launches() == before
