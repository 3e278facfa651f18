"""GPU parity of gnf4_int4_pack and gnf4_int4_linear.

Bars:
  * pack: codes, scales and zero points bit for bit;
  * linear: |y - o| <= 2^-8 |o| (one rounding to bf16) + K 2^-23 mag, o the
    fp64 value and mag = sum_k |x| (|q - 8| + |z - 8|) s + |bias| (the kernel
    adds the two exact products (q - 8) x and -(z - 8) x; each of the at most
    2 K fp32 additions is off by at most 2^-24 of a partial sum's magnitude).
"""

import numpy as np
import pytest
import torch

import oracle
from grouped_nf4_expert_amd import gnf4

from gpu_util import DEV, bf16_dev, host_f64, note

pytestmark = pytest.mark.gpu

SCALES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _weights(rng, N, K, group, zero_points, scale_dtype):
    """Random codes (all sixteen), scales over several binades, zero points."""
    packed = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = (0.01 * 2.0 ** rng.uniform(-3, 3, (N, K // group))).astype(np.float32)
    zeros = rng.integers(0, 16, (N, K // group), dtype=np.uint8) if zero_points else None
    s_dev = torch.from_numpy(scales).to(DEV).to(SCALES[scale_dtype])
    return (torch.from_numpy(packed).to(DEV), s_dev,
            None if zeros is None else torch.from_numpy(zeros).to(DEV))


def _check(y, x, packed, scales, zeros, bias, what):
    p, s = packed.cpu().numpy(), host_f64(scales)
    z = None if zeros is None else zeros.cpu().numpy()
    b = None if bias is None else host_f64(bias)
    xh = host_f64(x)
    o = oracle.ref_int4_linear(xh, p, s, z, b)
    mag = np.abs(xh) @ np.abs(oracle.ref_int4_unpack(p, s)).T
    if z is not None:
        dz = np.abs(z.astype(np.float64) - 8.0) * s
        mag += np.abs(xh) @ np.repeat(dz, xh.shape[1] // s.shape[1], axis=1).T
    if b is not None:
        mag += np.abs(b)
    g = host_f64(y)
    assert np.all(np.isfinite(g)), what
    bad = np.abs(g - o) > 2.0 ** -8 * np.abs(o) + xh.shape[1] * 2.0 ** -23 * mag
    assert not bad.any(), f"{what}: {int(bad.sum())}/{bad.size} outside tolerance"


# -------------------------------------------------------------------- pack

def _pack_input(N, K, group, seed):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    rows = w.reshape(-1, group)
    special = [np.zeros(group), np.abs(rows[0]), -np.abs(rows[0]), np.full(group, 1e-42),
               np.full(group, -3e38), np.linspace(-3e38, 3e38, group), np.full(group, 0.125),
               (np.arange(group) % 29 - 14) * 0.5,      # every midpoint of s = 1
               (np.arange(group) % 31 - 15) * 0.5]
    for i, v in enumerate(special):
        if 2 * i + 1 < rows.shape[0]:
            rows[2 * i + 1] = v.astype(np.float32)
    return w


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("w_dtype,scale", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"),
                                           ("bf16", "f32")])
def test_pack_bits(group, zero_points, w_dtype, scale):
    for N, K in ((1, group), (5, 3 * group), (33, 640)):
        note(f"int4_pack {N}x{K} group {group} zp {zero_points} {w_dtype}/{scale}")
        w = torch.from_numpy(_pack_input(N, K, group, N * K + group)).to(DEV)
        if w_dtype == "bf16":
            w = w.to(torch.bfloat16)
        packed, scales, zeros = gnf4.int4_pack(w, group, zero_points, SCALES[scale])
        torch.cuda.synchronize()
        p, s, z = oracle.ref_int4_pack(w.float().cpu().numpy(), group, zero_points, scale)
        assert np.array_equal(scales.float().cpu().numpy().view(np.uint32), s.view(np.uint32))
        assert np.array_equal(packed.cpu().numpy(), p)
        assert (zeros is None) == (z is None)
        if z is not None:
            assert np.array_equal(zeros.cpu().numpy(), z)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("scale", ["f32", "bf16"])
def test_pack_bits_beside_the_midpoints(zero_points, scale):
    """Weights one fp32 step to either side of every midpoint, over scales from
    subnormal to the largest."""
    rng = np.random.default_rng(31)
    with np.errstate(over="ignore", under="ignore"):
        s = np.float32(2.0) ** rng.integers(-149, 124, (400, 1)).astype(np.float32)
        s = (s * rng.uniform(1, 2, (400, 1))).astype(np.float32)
        mid = (rng.integers(-7, 7, (400, 32)) + 0.5).astype(np.float32) * s
        w = np.stack([mid, np.nextafter(mid, np.float32(np.inf)),
                      np.nextafter(mid, np.float32(-np.inf)), -mid], 2).reshape(400, 128)
        w[:, 0] = 7.0 * s[:, 0]
    w = np.where(np.isfinite(w), w, np.float32(3e38)).astype(np.float32)
    for group in (32, 128):
        packed, scales, zeros = gnf4.int4_pack(torch.from_numpy(w).to(DEV), group, zero_points,
                                               SCALES[scale])
        torch.cuda.synchronize()
        p, sc, z = oracle.ref_int4_pack(w, group, zero_points, scale)
        assert np.array_equal(scales.float().cpu().numpy().view(np.uint32), sc.view(np.uint32))
        assert np.array_equal(packed.cpu().numpy(), p)
        if z is not None:
            assert np.array_equal(zeros.cpu().numpy(), z)


def test_pack_stack_is_rows_and_empty_like_shapes():
    w = bf16_dev(_pack_input(12, 256, 64, 3)).view(3, 4, 256)
    packed, scales, zeros = gnf4.int4_pack(w, 64, True)
    flat = gnf4.int4_pack(w.view(12, 256), 64, True)
    torch.cuda.synchronize()
    assert packed.shape == (3, 4, 128) and scales.shape == (3, 4, 4) == zeros.shape
    for a, b in zip((packed, scales, zeros), flat):
        assert torch.equal(a.view(b.shape), b)


# ------------------------------------------------------------------ linear

@pytest.mark.parametrize("M,N,K,group", [
    (1, 1, 32, 32), (1, 16, 64, 64), (1, 17, 128, 128), (2, 100, 96, 32), (3, 15, 192, 64),
    (15, 33, 160, 32), (16, 64, 384, 128), (17, 31, 320, 64), (1, 2048, 2048, 128),
    (1, 130, 2880, 32), (5, 50, 2880, 64), (33, 48, 1152, 128), (64, 16, 64, 32),
    (65, 80, 256, 64), (130, 100, 1024, 128), (200, 5, 7168, 32)])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("scale", ["f32", "bf16"])
def test_linear_parity(M, N, K, group, zero_points, scale):
    note(f"int4_linear {M}x{N}x{K} group {group} zp {zero_points} {scale}")
    rng = np.random.default_rng(M * 7 + N * 3 + K + group)
    packed, scales, zeros = _weights(rng, N, K, group, zero_points, scale)
    x = bf16_dev(rng.standard_normal((M, K)))
    bias = bf16_dev(rng.standard_normal(N)) if zero_points else None
    guard = torch.full((M + 2, N), -512.0, dtype=torch.bfloat16, device=DEV)
    gnf4.int4_linear(x, packed, scales, zeros, bias, out=guard[1:M + 1])
    torch.cuda.synchronize()
    _check(guard[1:M + 1], x, packed, scales, zeros, bias, f"{M}x{N}x{K}")
    assert torch.all(guard[0] == -512.0) and torch.all(guard[M + 1] == -512.0)
    again = gnf4.int4_linear(x, packed, scales, zeros, bias)
    torch.cuda.synchronize()
    assert torch.equal(again, guard[1:M + 1])


@pytest.mark.parametrize("M,N,K,group", [
    (130, 3400, 160, 32), (300, 1700, 320, 64), (1030, 600, 192, 32), (257, 2500, 384, 128),
    (97, 6000, 1152, 128), (520, 1100, 2880, 32), (33, 70, 32, 32), (70, 300, 96, 32),
    (50, 33, 64, 64), (2000, 515, 64, 32), (600, 1030, 128, 128)])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("scale", ["f32", "bf16"])
def test_linear_many_tiles(M, N, K, group, zero_points, scale):
    """More tiles than the chip has CUs, and rows shorter than a step."""
    test_linear_parity(M, N, K, group, zero_points, scale)


@pytest.mark.parametrize("steps", [1, 2, 3, 5, 8, 9, 12, 16, 17, 23, 24, 31, 32, 33, 40, 47, 48,
                                   56, 64, 65, 100])
@pytest.mark.parametrize("N", [13, 600, 4500])
def test_linear_row_lengths(steps, N):
    """Every split of a row over the wavefronts, with a row that ends inside
    its last step where the group allows."""
    for group in (32, 64, 128):
        zp = (steps + group // 32) % 2 == 0
        K = steps * 128 - (group if group < 128 else 0)
        test_linear_parity(1 + steps % 16, N, K, group, zp, "bf16" if steps % 2 else "f32")


@pytest.mark.parametrize("N", [33000, 49990, 66001, 68033, 70017, 90050, 131201])
@pytest.mark.parametrize("K", [64, 128, 256, 512])
def test_linear_teams_of_unequal_shares(N, K):
    """Items that do not divide among the teams of a workgroup (the bar above,
    worked out in 64 bits on the GPU)."""
    rng = np.random.default_rng(N + K)
    packed, scales, _ = _weights(rng, N, K, 64, False, "f32")
    q = torch.stack([packed >> 4, packed & 15], 2).view(N, K).double() - 8
    w = (q.view(N, K // 64, 64) * scales.double()[..., None]).view(N, K)
    for M in (1, 5):
        note(f"int4_linear {M}x{N}x{K}")
        x = bf16_dev(rng.standard_normal((M, K)))
        y = gnf4.int4_linear(x, packed, scales).double()
        o = x.double() @ w.t().contiguous()
        mag = x.double().abs() @ w.t().contiguous().abs()
        bad = (y - o).abs() > 2.0 ** -8 * o.abs() + K * 2.0 ** -23 * mag
        assert not bad.any(), f"{int(bad.sum())} outside, first {bad.nonzero()[0].tolist()}"


def test_linear_rows_do_not_depend_on_each_other():
    """A row keeps its bits whatever the other rows hold, infinities and NaN
    among them (rows of one matrix-core tile)."""
    rng = np.random.default_rng(11)
    packed, scales, zeros = _weights(rng, 40, 256, 64, True, "bf16")
    x = bf16_dev(rng.standard_normal((20, 256)))
    ref = gnf4.int4_linear(x, packed, scales, zeros)
    y = x.clone()
    y[3, 5], y[7] = float("inf"), float("nan")
    got = gnf4.int4_linear(y, packed, scales, zeros)
    torch.cuda.synchronize()
    keep = [i for i in range(20) if i not in (3, 7)]
    assert torch.equal(got[keep], ref[keep])
    assert torch.isnan(got[7]).all()


def test_linear_activation_range():
    """Activations over bf16's range of exponents in one row."""
    rng = np.random.default_rng(12)
    packed, scales, zeros = _weights(rng, 64, 512, 128, False, "f32")
    for scale in (1e-30, 1e-4, 1e30):
        x = bf16_dev(rng.standard_normal((4, 512)) * scale * 2.0 ** rng.integers(-8, 8, (4, 512)))
        y = gnf4.int4_linear(x, packed, scales, zeros)
        torch.cuda.synchronize()
        _check(y, x, packed, scales, zeros, None, f"scale {scale}")


def test_linear_no_rows_and_offsets_past_32_bits():
    x0 = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    p = torch.zeros((8, 32), dtype=torch.uint8, device=DEV)
    s = torch.ones((8, 1), device=DEV)
    assert gnf4.int4_linear(x0, p, s).shape == (0, 8)
    N, K = (1 << 20) + 37, 8192           # 4.3 GB of codes
    note(f"int4_linear large {N}x{K}")
    gen = torch.Generator(device=DEV).manual_seed(5)
    packed = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gen)
    scales = torch.rand((N, K // 128), device=DEV, generator=gen) * 0.01 + 0.005
    x = torch.randn((2, K), device=DEV, generator=gen).to(torch.bfloat16)
    y = gnf4.int4_linear(x, packed, scales)
    torch.cuda.synchronize()
    for a in (0, N // 2, N - 40):
        sl = slice(a, a + 40)
        _check(y[:, sl], x, packed[sl], scales[sl], None, None, f"rows from {a}")


# -------------------------------------------------------- streams and graphs

def test_linear_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(13)
    packed, scales, zeros = _weights(rng, 96, 256, 64, True, "bf16")
    xs = [bf16_dev(rng.standard_normal((6, 256))) for _ in range(3)]
    refs = [gnf4.int4_linear(x, packed, scales, zeros) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gnf4.int4_linear(xs[0], packed, scales, zeros)
    side.synchronize()
    assert torch.equal(got, refs[0])
    x, out = xs[0].clone(), torch.empty_like(refs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gnf4.int4_linear(x, packed, scales, zeros, out=out)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, refs[i])


def test_linear_on_two_streams_at_once():
    rng = np.random.default_rng(14)
    packed, scales, zeros = _weights(rng, 700, 1024, 32, True, "f32")
    xs = [bf16_dev(rng.standard_normal((m, 1024))) for m in (1, 40, 500)]
    refs = [gnf4.int4_linear(x, packed, scales, zeros) for x in xs]
    outs = [torch.empty_like(r) for r in refs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, s in zip(xs, outs, streams):
            with torch.cuda.stream(s):
                gnf4.int4_linear(x, packed, scales, zeros, out=o)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


# ---------------------------------------------------------------- refusals

def test_refusals_on_the_gpu():
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV)
    p = torch.zeros((4, 64), dtype=torch.uint8, device=DEV)
    s = torch.ones((4, 1), device=DEV)
    with pytest.raises(gnf4.Gnf4Error, match="device memory"):
        gnf4.int4_linear(x.cpu(), p.cpu(), s.cpu())
    with pytest.raises(ValueError, match="expected cuda"):
        gnf4.int4_linear(x, p.cpu(), s)
    with pytest.raises(ValueError, match="contiguous"):
        gnf4.int4_linear(x.t().contiguous().t(), p, s)
    with pytest.raises(gnf4.Gnf4Error, match="invalid argument"):   # group 16
        gnf4.int4_linear(x, p, torch.ones((4, 8), device=DEV))
    off = torch.zeros(2 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 128)
    with pytest.raises(gnf4.Gnf4Error, match="invalid argument"):   # misaligned rows
        gnf4.int4_linear(off, p, s)
    sq = torch.ones((128, 1), device=DEV)
    with pytest.raises(gnf4.Gnf4Error, match="invalid argument"):   # y over x
        gnf4.int4_linear(x, torch.zeros((128, 64), dtype=torch.uint8, device=DEV), sq, out=x)
