"""Low-rank adapters on the GPU against the oracle in binary64.

Tolerance.  Products of bf16 values are exact in binary32.  A rank's t is a binary32 sum of K products in some order,
then scaled: within (K + 24) 2^-24 of sum |x a| s.  t enters the second product as hi + lo, within 2^-16 of itself (hi is
cut below 8 bits, lo rounded to 8 of what is left), and 2 R products and y are added: (2 R + 3) 2^-24 of sum |t b| + |y|.
The result's rounding to bf16 is within 2^-8 of it (2^-134 where bf16 is subnormal).  Sums of small whole numbers are
exact everywhere, and are compared bit for bit."""
import numpy as np
import pytest
import torch

import block_wise_int8_amd as bi8
import workloads as wl
from gpu_util import bf16_bits, bf16_to_dev, bits_to_f64, device, to_dev
from oracle import layer

pytestmark = pytest.mark.gpu


def make(rng, M, N, K, L, R, P, whole=False, pad=0):
    if whole:   # |t| <= 4 K, exact in 16 bits up to K = 2^14; |y + t b| kept small by few ones in a
        x = wl.to_bf16_bits(rng.integers(-2, 3, (M, K + pad)).astype(np.float32))
        a = wl.to_bf16_bits((rng.integers(-1, 2, (L, P * R, K)) * (rng.random((L, P * R, K)) < 8 / K)).astype(np.float32))
        b = wl.to_bf16_bits((rng.integers(-1, 2, (L, N, R)) * (rng.random((L, N, R)) < 4 / R)).astype(np.float32))
        y = wl.to_bf16_bits(rng.integers(-8, 9, (M, N + pad)).astype(np.float32))
        return x, a, b, y, (2.0 ** rng.integers(-1, 2, L)).astype(np.float32)
    return (wl.activations(rng, M, K + pad, 0.01), wl.to_bf16_bits((rng.standard_normal((L, P * R, K)) / K ** 0.5).astype(np.float32)),
            wl.to_bf16_bits((rng.standard_normal((L, N, R)) / R ** 0.5).astype(np.float32)),
            wl.activations(rng, M, N + pad), rng.uniform(0.25, 2, L).astype(np.float32))


def check(got, x, a, b, y, scales, adapter, parts, exact=False):
    K, R = x.shape[1], b.shape[2]
    ref, of_t, of_x = layer.lora_add(layer.bf16(y), layer.bf16(x), layer.bf16(a), layer.bf16(b), scales, adapter, parts)
    g = bits_to_f64(got)
    if exact:
        assert np.array_equal(g, bits_to_f64(wl.to_bf16_bits(ref.astype(np.float32))))
        return
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + 1.01 * (
        (K + 24) * 2.0 ** -24 * of_x + (2.0 ** -16 + (2 * R + 3) * 2.0 ** -24) * of_t + 2.0 ** -24 * np.abs(layer.bf16(y)))
    bare = np.array([not 0 <= e < len(a) for e in adapter], bool)
    tol[bare] = 0
    assert np.all(np.abs(g - ref) <= tol)


def choose(rng, M, L, how):
    if how == "own":
        return (np.arange(M) % L).astype(np.int32)
    if how == "one":
        return np.full(M, L - 1, np.int32)
    if how == "random":
        return rng.integers(-1, L, M).astype(np.int32)
    cuts = np.sort(rng.integers(0, M + 1, 5))
    return (rng.permutation(np.arange(6)) % (L + 1) - 1)[np.searchsorted(cuts, np.arange(M), side="right")].astype(np.int32)


SHAPES = [  # M, N, K, L, R, parts, adapters
    (1, 1, 1, 1, 8, None, "one"), (1, 64, 512, 3, 16, None, "one"), (2, 40, 33, 2, 8, None, "own"), (5, 100, 8, 4, 24, None, "own"),
    (16, 128, 256, 2, 32, None, "random"), (17, 33, 200, 5, 64, (16, 17), "random"), (63, 256, 129, 9, 40, (64, 128, 64), "own"),
    (64, 320, 640, 64, 16, (128, 128, 64), "own"), (65, 520, 1024, 3, 128, None, "runs"), (64, 96, 96, 1, 256, None, "one"),
    (33, 200, 72, 2, 256, None, "random"), (40, 130, 264, 3, 200, None, "runs"), (64, 300, 72, 2, 56, (100, 100, 50, 50), "runs"),
    (130, 1000, 1000, 7, 8, (999, 1), "runs"), (333, 500, 400, 5, 16, None, "random"), (700, 136, 96, 4, 48, (72, 64), "runs"),
    (2100, 264, 64, 3, 32, None, "runs"), (2500, 72, 40, 200, 8, None, "random"), (4200, 40, 24, 6, 64, (8, 8, 24), "runs"),
    (300, 2048, 128, 2, 96, None, "one"), (90, 4100, 520, 3, 16, None, "runs"), (3, 9000, 9000, 2, 16, None, "own")]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("M,N,K,L,R,parts,how", SHAPES)
def test_against_oracle(M, N, K, L, R, parts, how, whole):
    rng = wl.rng_for((121, M, N, K))
    P = 1 if parts is None else len(parts)
    x, a, b, y, s = make(rng, M, N, K, L, R, P, whole)
    adapter = choose(rng, M, L, how)
    yd = bf16_to_dev(y)
    out = bi8.lora_add(yd, bf16_to_dev(x), bf16_to_dev(a), bf16_to_dev(b), to_dev(adapter), to_dev(s), parts)
    assert out is yd
    check(bf16_bits(yd), x, a, b, y, s, adapter, parts or (N,), whole)


@pytest.mark.parametrize("K,N,xpad,ypad,shift", [
    (256, 512, 8, 8, 0), (256, 512, 3, 0, 0), (256, 512, 0, 5, 0), (255, 511, 2, 3, 0), (256, 512, 8, 8, 1), (96, 130, 4, 6, 2)])
def test_rows_apart(K, N, xpad, ypad, shift):
    """Any stride and offset of x and y; the columns behind the rows stay as they were."""
    rng = wl.rng_for((122, K, xpad, ypad, shift))
    M, L, R = 70, 3, 16
    x, a, b, _, s = make(rng, M, N, K, L, R, 1)
    adapter = choose(rng, M, L, "random")
    wide = wl.activations(rng, M, N + ypad + shift)
    xd = torch.zeros(M, K + xpad + shift, dtype=torch.bfloat16, device=device())
    xd[:, shift: shift + K] = bf16_to_dev(x)
    yd = bf16_to_dev(wide)
    bi8.lora_add(yd[:, shift: shift + N], xd[:, shift: shift + K], bf16_to_dev(a), bf16_to_dev(b), to_dev(adapter), to_dev(s))
    got = bf16_bits(yd)
    cols = slice(shift, shift + N)
    check(np.ascontiguousarray(got[:, cols]), x, a, b, np.ascontiguousarray(wide[:, cols]), s, adapter, (N,))
    got[:, cols] = wide[:, cols]
    assert np.array_equal(got, wide)


def test_a_row_does_not_depend_on_the_others():
    """Rows moved to other places and beside other adapters, NaN in their neighbours: the same bits."""
    rng = wl.rng_for(123)
    M, N, K, L, R = 128, 200, 300, 6, 16
    x, a, b, y, s = make(rng, M, N, K, L, R, 1)
    adapter = rng.integers(0, L, M).astype(np.int32)
    dev = [bf16_to_dev(a), bf16_to_dev(b)]

    def call(x, y, adapter):
        return bf16_bits(bi8.lora_add(bf16_to_dev(y), bf16_to_dev(x), *dev, to_dev(adapter), to_dev(s)))

    base = call(x, y, adapter)
    move = rng.permutation(M)
    assert np.array_equal(call(x[move], y[move], adapter[move]), base[move])
    bad = rng.random(M) < 0.5
    x2, y2 = x.copy(), y.copy()
    x2[bad] = 0x7FC0
    got = call(x2, y2, adapter)
    assert np.array_equal(got[~bad], base[~bad]) and np.isnan(bits_to_f64(got[bad])).all()
    # one adapter of NaN touches its own rows alone
    a2 = a.copy()
    a2[2] = 0x7FC0
    dev[0] = bf16_to_dev(a2)
    got = call(x, y, adapter)
    mine = adapter == 2
    assert np.array_equal(got[~mine], base[~mine]) and np.isnan(bits_to_f64(got[mine])).all()


def test_rows_without_an_adapter():
    rng = wl.rng_for(124)
    M, N, K, L, R = 100, 96, 64, 2, 8
    x, a, b, y, _ = make(rng, M, N, K, L, R, 1)
    adapter = rng.choice(np.array([-1, 0, 1, L, -2 ** 31, 2 ** 31 - 1]), M).astype(np.int32)
    x[~((adapter >= 0) & (adapter < L))] = 0x7FC0
    yd = bf16_to_dev(y)
    bi8.lora_add(yd, bf16_to_dev(x), bf16_to_dev(a), bf16_to_dev(b), to_dev(adapter))
    x[~((adapter >= 0) & (adapter < L))] = 0
    check(bf16_bits(yd), x, a, b, y, None, adapter, (N,))
    before = bf16_bits(yd)
    bi8.lora_add(yd, bf16_to_dev(x), bf16_to_dev(a), bf16_to_dev(b), torch.full((M,), -1, dtype=torch.int32, device=device()))
    assert np.array_equal(bf16_bits(yd), before)


def test_infinite_sums():
    """A t past binary32 gives infinities of its sign, as the sum does, and NaN only where b is 0."""
    M, N, K, R = 3, 16, 8, 8
    x = wl.to_bf16_bits(np.full((M, K), 1e30, np.float32))
    a = np.zeros((1, R, K), np.uint16)
    a[0, 0] = wl.to_bf16_bits(np.full(K, 1e30, np.float32))
    b = np.zeros((1, N, R), np.uint16)
    b[0, :8, 0], b[0, 8:12, 0] = 0x3F80, 0xBF80
    y = torch.zeros(M, N, dtype=torch.bfloat16, device=device())
    got = bits_to_f64(bf16_bits(bi8.lora_add(y, bf16_to_dev(x), bf16_to_dev(a), bf16_to_dev(b),
                                             torch.zeros(M, dtype=torch.int32, device=device()))))
    assert np.all(got[:, :8] == np.inf) and np.all(got[:, 8:12] == -np.inf) and np.isnan(got[:, 12:]).all()


def test_workspace():
    rng = wl.rng_for(125)
    M, N, K, L, R = 200, 64, 1100, 3, 24
    x, a, b, y, s = make(rng, M, N, K, L, R, 2)
    adapter = choose(rng, M, L, "random")
    args = [bf16_to_dev(x), bf16_to_dev(a), bf16_to_dev(b), to_dev(adapter), to_dev(s), (32, 32)]
    n = bi8.lora_add_workspace_size(M, K, R, 2)
    scratch = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=device())   # NaN wherever it is read unwritten
    one = bi8.lora_add(bf16_to_dev(y), *args, workspace=scratch[:n])
    assert torch.all(scratch[n:] == 0xFF)
    assert torch.equal(one, bi8.lora_add(bf16_to_dev(y), *args))
    check(bf16_bits(one), x, a, b, y, s, adapter, (32, 32))
    with pytest.raises(bi8.BlockInt8Error, match="workspace_bytes"):
        bi8.lora_add(bf16_to_dev(y), *args, workspace=scratch[: n - 1])


def test_refusals_of_the_binding():
    dev = device()
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device=dev)
    y, x, a, b, ids = z(4, 32), z(4, 16), z(2, 8, 16), z(2, 32, 8), z(4, d=torch.int32)
    assert bi8.lora_add(y, x, a, b, ids) is y
    for bad in (lambda: bi8.lora_add(y.float(), x, a, b, ids), lambda: bi8.lora_add(y, x.half(), a, b, ids),
                lambda: bi8.lora_add(y, x, a.float(), b, ids), lambda: bi8.lora_add(y, x, a, b, ids.long()),
                lambda: bi8.lora_add(y, x, a, b, ids, z(2))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bi8.lora_add(y, x[:3], a, b, ids), lambda: bi8.lora_add(y, x, a, z(2, 31, 8), ids),
                lambda: bi8.lora_add(y, x, z(2, 16, 16), b, ids), lambda: bi8.lora_add(y, x, z(3, 8, 16), b, ids),
                lambda: bi8.lora_add(y, x, a, b, ids[:3]), lambda: bi8.lora_add(y, x, a, b, ids, z(3, d=torch.float32)),
                lambda: bi8.lora_add(y, x, a, b, ids.cpu()), lambda: bi8.lora_add(z(32, 4).t(), x, a, b, ids),
                lambda: bi8.lora_add(z(1, 32).expand(4, 32), x, a, b, ids),
                lambda: bi8.lora_add(y, x, a, b, ids, parts=(16, 16))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bi8.lora_add(y, x, a, b, ids, parts=(31,)), lambda: bi8.lora_add(y, x, z(2, 4, 16), z(2, 32, 4), ids),
                lambda: bi8.lora_add(y, x, z(2, 16, 16), b, ids, parts=(32, 0)),
                lambda: bi8.lora_add(y, x, z(2, 264, 16), z(2, 32, 264), ids), lambda: bi8.lora_add(y, x, z(2, 0, 16), b, ids, parts=()),
                lambda: bi8.lora_add(y, x, z(2, 40, 16), b, ids, parts=(8, 8, 8, 4, 4))):
        with pytest.raises(bi8.BlockInt8Error):
            bad()
    assert bi8.lora_add(y[:0], x[:0], a, b, ids[:0]).shape == (0, 32)


@pytest.mark.parametrize("M", [1, 64, 200])
def test_captured_and_replayed(M):
    rng = wl.rng_for((126, M))
    N, K, L, R = 256, 512, 5, 16
    _, a, b, _, s = make(rng, M, N, K, L, R, 1)
    xs = [bf16_to_dev(wl.activations(rng, M, K)) for _ in range(4)]
    ys = [bf16_to_dev(wl.activations(rng, M, N)) for _ in range(4)]
    ids = [to_dev(choose(rng, M, L, "random")) for _ in range(4)]
    a, b, s = bf16_to_dev(a), bf16_to_dev(b), to_dev(s)
    x, y, e = xs[0].clone(), ys[0].clone(), ids[0].clone()
    scratch = torch.empty(bi8.lora_add_workspace_size(M, K, R), dtype=torch.uint8, device=device())
    bi8.lora_add(y, x, a, b, e, s, workspace=scratch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bi8.lora_add(y, x, a, b, e, s, workspace=scratch)
    for r in (1, 2, 3):
        x.copy_(xs[r])
        y.copy_(ys[r])
        e.copy_(ids[r])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bi8.lora_add(ys[r].clone(), xs[r], a, b, ids[r], s))


@pytest.mark.parametrize("M,N,K,L,R,parts", [
    (64, 264, 96, 40, 16, None), (70, 200, 72, 70, 64, (100, 100)), (100, 130, 100, 60, 24, None), (150, 96, 64, 90, 136, None),
    (130, 72, 136, 80, 256, None), (1100, 72, 40, 600, 8, None), (33, 1030, 1000, 20, 128, None)])
def test_many_adapters_one_of_them_crowded(M, N, K, L, R, parts):
    """More adapters than half the rows, and half the rows on one: rows go 16 at a time, and some have to go again."""
    rng = wl.rng_for((127, M, N, K))
    x, a, b, y, s = make(rng, M, N, K, L, R, 1 if parts is None else len(parts))
    adapter = rng.integers(0, L, M).astype(np.int32)
    adapter[rng.permutation(M)[: M // 2]] = L - 1
    yd = bf16_to_dev(y)
    bi8.lora_add(yd, bf16_to_dev(x), bf16_to_dev(a), bf16_to_dev(b), to_dev(adapter), to_dev(s), parts)
    check(bf16_bits(yd), x, a, b, y, s, adapter, parts or (N,))
