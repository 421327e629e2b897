"""Norm and rotation of query and key heads on the GPU against the oracle in binary64.

Tolerance.  u = (x rstd) w has three roundings of binary32 (rstd itself and two products), 3 * 2^-24; a turned value
adds two products: one rounded by itself, the other inside the fused sum, whose rounding is 2^-24 of the result.  With
m = |u1 c| + |u2 s| the binary32 value is within 5 * 2^-24 m of the exact one, and its rounding to bf16 adds at most
2^-8 of the result (half a step; 2^-134 where bf16 is subnormal)."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, bits_to_f64, device, to_dev
from oracle import layer

pytestmark = pytest.mark.gpu

EPS = 1e-6
NAN = 0x7FC1   # bf16 pattern of bytes that have to stay


def rope_table(P, rot):
    angle = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def gain(rng, D):
    return wl.to_bf16_bits((1 + 0.1 * rng.standard_normal(D)).astype(np.float32))


def check(out, x, weight, table, positions, sections, rot, interleaved, eps=EPS):
    """out: bits [T, H, D] of the call on bits x; rows with a position outside the table are not looked at."""
    ref, mag = layer.head_norm_rope(layer.bf16(x), None if weight is None else layer.bf16(weight), eps, table,
                                    positions, sections, rot, interleaved)
    inside = np.all((positions >= 0) & (positions < table.shape[0]), axis=0)
    got = bits_to_f64(out)[inside]
    ref, mag = ref[inside], mag[inside]
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 5 * 2.0 ** -24 * 1.01 * mag + 2.0 ** -134)


def spread(axes, half):
    sections = [half // axes] * axes
    sections[0] += half - sum(sections)
    return sections


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,axes,norm", [
    (1, 1, 0, 2, 2, 1, True), (1, 1, 1, 8, 8, 1, False), (3, 2, 1, 16, 16, 1, True), (2, 3, 2, 64, 64, 3, True),
    (5, 4, 2, 128, 128, 1, True), (1, 32, 8, 128, 128, 1, True), (7, 7, 1, 128, 128, 3, False), (4, 5, 5, 80, 32, 1, True),
    (6, 3, 3, 80, 40, 2, True), (9, 2, 1, 96, 80, 4, True), (2, 2, 2, 256, 256, 1, True), (3, 1, 1, 512, 64, 2, True),
    (2, 2, 1, 1024, 1024, 1, True), (2, 1, 1, 516, 516, 1, True), (3, 2, 1, 70, 36, 3, True), (2, 2, 1, 130, 66, 1, True),
    (2, 1, 1, 258, 130, 2, True), (1, 1, 1, 1022, 1022, 1, True), (2, 2, 2, 514, 2, 1, False), (300, 3, 1, 64, 48, 1, True),
    (1100, 28, 4, 128, 128, 3, True), (2100, 30, 10, 64, 64, 1, True), (3, 2, 1, 72, 72, 4, False)])
def test_against_oracle(T, Hq, Hk, D, rot, axes, norm, interleaved):
    rng = wl.rng_for((101, T, D, rot))
    P, sections = 50, spread(axes, rot // 2)
    x = wl.activations(rng, T, (Hq + 2 * Hk) * D, 0.02).reshape(T, Hq + 2 * Hk, D)
    table, positions = rope_table(P, rot), rng.integers(0, P, (axes, T)).astype(np.int32)
    qw, kw = (gain(rng, D), gain(rng, D)) if norm else (None, None)
    xd = bf16_to_dev(x)
    on = lambda w: None if w is None else bf16_to_dev(w)
    pos = to_dev(positions if axes > 1 else positions[0])
    q, k = bi8.qk_norm_rope(xd[:, :Hq], xd[:, Hq: Hq + Hk] if Hk else None, pos, to_dev(table), on(qw),
                            on(kw) if Hk else None, EPS, sections if axes > 1 else None, interleaved)
    assert (k is None) == (Hk == 0)
    check(bf16_bits(q), x[:, :Hq], qw, table, positions, sections, rot, interleaved)
    if Hk:
        check(bf16_bits(k), x[:, Hq: Hq + Hk], kw, table, positions, sections, rot, interleaved)
    assert np.array_equal(bf16_bits(xd), x)
    # in place the same bits, and the value heads stay
    again = bi8.qk_norm_rope(xd[:, :Hq], xd[:, Hq: Hq + Hk] if Hk else None, pos, to_dev(table), on(qw),
                             on(kw) if Hk else None, EPS, sections, interleaved, q_out=xd[:, :Hq],
                             k_out=xd[:, Hq: Hq + Hk] if Hk else None)
    assert again[0].data_ptr() == xd.data_ptr()
    now = bf16_bits(xd)
    assert np.array_equal(now[:, :Hq], bf16_bits(q)) and np.array_equal(now[:, Hq + Hk:], x[:, Hq + Hk:])
    if Hk:
        assert np.array_equal(now[:, Hq: Hq + Hk], bf16_bits(k))


@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("layout", ["heads first", "padded", "tokens apart"])
def test_strides_and_alignment(layout, shift):
    """Views at any offset, outputs of other layouts than the inputs, bytes around the outputs untouched."""
    rng = wl.rng_for((102, shift))
    T, Hq, Hk, D, rot = 9, 4, 2, 64, 32
    table, positions = rope_table(20, rot), rng.integers(0, 20, (1, T)).astype(np.int32)
    qw, kw = gain(rng, D), gain(rng, D)
    src = wl.activations(rng, 1, 4 * T * Hq * D + shift)[0]
    dst = np.full(src.size, NAN, np.uint16)
    srcd, dstd, dstk = bf16_to_dev(src), bf16_to_dev(dst), bf16_to_dev(dst)

    def view(t, H, out):
        if layout == "heads first":
            token, head = (D, T * D + 8) if out else (H * D, D)
        elif layout == "padded":
            token, head = (H * (D + 4) + 12, D + 4) if out else (H * (D + 8), D + 8)
        else:
            token, head = (H * D + (1 if shift == 1 else 4), D) if out else (2 * H * D, D)
        return torch.as_strided(t, (T, H, D), (token, head, 1), shift)

    q, k = bi8.qk_norm_rope(view(srcd, Hq, False), view(srcd, Hk, False), to_dev(positions[0]), to_dev(table),
                            bf16_to_dev(qw), bf16_to_dev(kw), EPS, q_out=view(dstd, Hq, True), k_out=view(dstk, Hk, True))
    for got, t, H, w in ((q, dstd, Hq, qw), (k, dstk, Hk, kw)):
        x = bf16_bits(view(srcd, H, False).contiguous())
        check(bf16_bits(got.contiguous()), x, w, table, positions, [rot // 2], rot, False)
        view(t, H, True).fill_(float("nan"))
        t[torch.isnan(t)] = 0
        assert not bf16_bits(t).any()   # only NaN were left outside the heads


def test_every_path_gives_the_same_values():
    """The same heads at offsets that leave chunks of 8, 4 and 1 values: bit for bit the same."""
    rng = wl.rng_for(103)
    T, H, D = 40, 3, 128
    x, w = wl.activations(rng, T, H * D + 4, 0.02), gain(rng, D)
    table, pos = to_dev(rope_table(64, D)), to_dev(rng.integers(0, 64, T).astype(np.int32))
    want = None
    for shift in (0, 1, 4):
        buf = bf16_to_dev(np.zeros((T, H * D + 16), np.uint16))
        buf[:, shift: shift + H * D + 4] = bf16_to_dev(x)
        view = torch.as_strided(buf, (T, H, D), (H * D + 16, D, 1), shift)
        got = bf16_bits(bi8.qk_norm_rope(view, None, pos, table, bf16_to_dev(w))[0])
        want = got if want is None else want
        assert np.array_equal(got, want)


def test_padding_tokens_are_left_as_they_were():
    rng = wl.rng_for(104)
    T, Hq, Hk, D, P = 70, 3, 2, 64, 10
    x = wl.activations(rng, T, (Hq + Hk) * D).reshape(T, Hq + Hk, D)
    table = rope_table(P, D)
    positions = rng.integers(0, P, (2, T)).astype(np.int32)
    positions[0, [0, 11]] = -1
    positions[1, [3, 69]] = P
    positions[1, 40] = -2 ** 31
    positions[0, 41] = 2 ** 31 - 1
    left = [0, 3, 11, 40, 41, 69]
    out = torch.full((T, Hq + Hk, D), -7.0, dtype=torch.bfloat16, device=device())
    xd = bf16_to_dev(x)
    bi8.qk_norm_rope(xd[:, :Hq], xd[:, Hq:], to_dev(positions), to_dev(table), sections=(20, 12), q_out=out[:, :Hq],
                     k_out=out[:, Hq:])
    assert torch.all(out[left] == -7)
    check(bf16_bits(out), x, None, table, positions, (20, 12), D, False)


@pytest.mark.parametrize("D,interleaved", [(64, False), (64, True), (36, False), (70, True)])
def test_special_values(D, interleaved):
    """Zero heads, huge and tiny values, eps of zero, infinities and NaN: of their own head only."""
    rng = wl.rng_for((105, D))
    T, H, rot = 8, 2, D // 4 * 2
    x = wl.activations(rng, T, H * D).reshape(T, H, D)
    x[0, 0] = 0
    x[1, 1] = wl.to_bf16_bits(np.full(D, 1e30, np.float32))      # squares past binary32
    x[2, 0] = wl.to_bf16_bits(np.full(D, 1e-30, np.float32))     # eps decides
    w, table = gain(rng, D), rope_table(16, rot)
    positions = rng.integers(0, 16, (1, T)).astype(np.int32)
    out = bi8.qk_norm_rope(bf16_to_dev(x), None, to_dev(positions[0]), to_dev(table), bf16_to_dev(w), None, EPS,
                           interleaved=interleaved)[0]
    check(bf16_bits(out), x, w, table, positions, [rot // 2], rot, interleaved)
    x[3, 1, D - 1] = 0x7FC0
    x[4, 0, 0] = 0x7F80
    out = bi8.qk_norm_rope(bf16_to_dev(x), None, to_dev(positions[0]), to_dev(table), bf16_to_dev(w), None, 0.0,
                           interleaved=interleaved)[0]
    got = bits_to_f64(bf16_bits(out))
    assert np.isnan(got[3, 1]).all() and np.isnan(got[0, 0]).all()   # 0 / 0 with eps = 0
    assert np.isnan(got[4, 0, 0])                                    # infinity / infinity
    fine = np.ones((T, H), bool)
    fine[3, 1] = fine[0, 0] = fine[4, 0] = False
    assert np.isfinite(got[fine]).all()
    # without a norm an infinity past rot is copied, and touches nothing else
    y = x.copy()
    y[3, 1, D - 1], y[4, 0, 0] = 0xFF80, 0x3F80
    got = bits_to_f64(bf16_bits(bi8.qk_norm_rope(bf16_to_dev(y), None, to_dev(positions[0]), to_dev(table),
                                                 interleaved=interleaved)[0]))
    assert got[3, 1, D - 1] == -np.inf and np.isfinite(got).sum() == got.size - 1


def test_refusals_of_the_binding():
    dev = device()
    x = torch.zeros(4, 3, 16, dtype=torch.bfloat16, device=dev)
    pos, tab = torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(8, 16, device=dev)
    w = torch.ones(16, dtype=torch.bfloat16, device=dev)
    ok = bi8.qk_norm_rope(x, x, pos, tab, w, w)
    assert ok[0].shape == x.shape
    for bad in (lambda: bi8.qk_norm_rope(x.float(), x, pos, tab), lambda: bi8.qk_norm_rope(x[0], x, pos, tab),
                lambda: bi8.qk_norm_rope(x, x, pos.long(), tab), lambda: bi8.qk_norm_rope(x, x.half(), pos, tab),
                lambda: bi8.qk_norm_rope(x, x, pos, tab.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bi8.qk_norm_rope(x, x[:3], pos, tab), lambda: bi8.qk_norm_rope(x, x[..., :8], pos, tab),
                lambda: bi8.qk_norm_rope(x, x, pos[:3], tab), lambda: bi8.qk_norm_rope(x, x, pos[None].repeat(2, 1), tab),
                lambda: bi8.qk_norm_rope(x, x, pos, tab, sections=(4, 4)), lambda: bi8.qk_norm_rope(x, x, pos, tab, w[:8]),
                lambda: bi8.qk_norm_rope(x, None, pos, tab, w, w), lambda: bi8.qk_norm_rope(x, x.cpu(), pos, tab),
                lambda: bi8.qk_norm_rope(x, x, pos.cpu(), tab),
                lambda: bi8.qk_norm_rope(x.transpose(1, 2), None, pos, tab),
                lambda: bi8.qk_norm_rope(x, x, pos, tab, q_out=x[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bi8.BlockInt8Error, match="overlap"):
        bi8.qk_norm_rope(x, None, pos, tab, q_out=x[:1].expand(4, 3, 16))
    with pytest.raises(bi8.BlockInt8Error, match="pairs"):
        bi8.qk_norm_rope(x, None, pos, tab, sections=(7,))
    # positions shared by all axes, and the empty call
    one = bi8.qk_norm_rope(x, None, pos[None].expand(3, 4), tab, sections=(2, 2, 4))[0]
    assert torch.equal(one, bi8.qk_norm_rope(x, None, pos, tab)[0])
    assert bi8.qk_norm_rope(x[:0], x[:0], pos[:0], tab)[1].shape == (0, 3, 16)


def test_captured_and_replayed():
    rng = wl.rng_for(106)
    T, Hq, Hk, D = 33, 4, 2, 128
    xs = [bf16_to_dev(wl.activations(rng, T, (Hq + Hk) * D)).view(T, Hq + Hk, D) for _ in range(4)]
    ps = [to_dev(rng.integers(-1, 64, T).astype(np.int32)) for _ in range(4)]
    tab, w = to_dev(rope_table(64, D)), bf16_to_dev(gain(rng, D))

    def call(x, p):
        return bi8.qk_norm_rope(x[:, :Hq], x[:, Hq:], p, tab, w, w, q_out=x[:, :Hq], k_out=x[:, Hq:])

    x, p = xs[0].clone(), ps[0].clone()
    call(x, p)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, p)
    for r in (1, 2, 3):
        x.copy_(xs[r])
        p.copy_(ps[r])
        g.replay()
        torch.cuda.synchronize()
        want = xs[r].clone()
        call(want, ps[r])
        torch.cuda.synchronize()
        assert torch.equal(x, want)
