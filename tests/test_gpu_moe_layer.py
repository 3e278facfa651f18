"""GPU parity of gnf4_moe_layer: a whole expert layer for a few tokens.

Routing is checked bit for bit (weights to 1e-6, exp is not bit-portable) and
the output against the fp64 oracle with a bound carried through the layer:
  * a gate or up sum is off by at most (H 2^-23 + L) mag, mag = sum |x w| (fp32
    additions), L = 2^-11 for NF4 (half a step of a level's fp16) and 0 for
    MXFP4 (its levels are exact); x is exact in fp16 after its row's power of
    two (values 2^28 below the row's largest lose less than 2^-24 mag);
  * h = w silu(g) u: those errors through its slopes (|silu'| <= 1.1), their
    product, and (2^-11 + 1e-5) |h| for its fp16 operand, exp and w;
  * out: sum |dh wd|, plus (k I 2^-23 + L) sum |h wd| for the fp32 additions
    and the levels, plus 2^-8 |out|.
"""

import numpy as np
import pytest
import torch

import oracle
from grouped_nf4_expert_amd import gnf4

from gpu_util import DEV, bf16_dev, host_f64, note

pytestmark = pytest.mark.gpu


class Layer:
    """Random stacks; experts outside `used` hold NaN scales, so a kernel that
    reads one shows."""

    def __init__(self, E, H, I, fmt, seed, used=None):
        self.E, self.H, self.I, self.fmt = E, H, I, fmt
        rng = np.random.default_rng(seed)
        self.host = {}
        dev = []
        for name, N, K in (("gu", 2 * I, H), ("dn", H, I)):
            p = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
            if fmt == "mxfp4":
                s = rng.integers(117, 123, (E, N, K // 32), dtype=np.uint8)
                nan = np.uint8(255)
            else:
                s = (0.06 * 2.0 ** rng.uniform(-3, 1, (E, N, K // 64))).astype(np.float32)
                if fmt == "nf4_bf16":
                    s = np.asarray(oracle.ref_round_bf16(s), dtype=np.float32)
                nan = np.float32("nan")
            if used is not None:
                for e in range(E):
                    if e not in used:
                        s[e] = nan
            self.host[name] = (p, s)
            sd = torch.from_numpy(s).to(DEV)
            if fmt == "nf4_bf16":
                sd = sd.to(torch.bfloat16)
            dev.append((torch.from_numpy(p).to(DEV), sd))
        self.gate_up, self.down = dev

    def weights(self, name, e):
        p, s = self.host[name]
        if self.fmt == "mxfp4":
            return oracle.ref_mx_unpack(p[e], s[e]).astype(np.float64)
        return oracle.ref_unpack(p[e], s[e]).astype(np.float64)


def expected(layer, logits, x, top_k, residual):
    """fp64 output, its bound, and the oracle's route."""
    r = oracle.ref_route_sort(logits, top_k)
    T, H, I = x.shape[0], layer.H, layer.I
    L = 0.0 if layer.fmt == "mxfp4" else 2.0 ** -11
    out, err = np.zeros((T, H)), np.zeros((T, H))
    if residual is not None:
        out += residual
    for t in range(T):
        for j in range(top_k):
            e, w = int(r["topk_ids"][t, j]), float(r["topk_w"][t, j])
            wgu, wd = layer.weights("gu", e), layer.weights("dn", e)
            gu = wgu @ x[t]
            dgu = (H * 2.0 ** -23 + L) * (np.abs(wgu) @ np.abs(x[t]))
            g, u, dg, du = gu[:I], gu[I:], dgu[:I], dgu[I:]
            sg = g / (1.0 + np.exp(-g))
            h = w * sg * u
            dh = w * (1.1 * dg * np.abs(u) + np.abs(sg) * du + 1.1 * dg * du)
            dh += (2.0 ** -11 + 1e-5) * np.abs(h)
            out[t] += wd @ h
            err[t] += np.abs(wd) @ dh
            err[t] += (top_k * I * 2.0 ** -23 + L) * (np.abs(wd) @ np.abs(h))
    return out, err + 2.0 ** -8 * np.abs(out), r


def run_case(T, E, top_k, H, I, fmt, residual, seed=0, logits=None, buffers=None):
    note(f"moe_layer T={T} E={E} k={top_k} H={H} I={I} {fmt} residual={residual}")
    rng = np.random.default_rng(seed + T * 31 + E)
    if logits is None:
        logits = rng.standard_normal((T, E)).astype(np.float32)
    used = set(oracle.ref_route_sort(logits, top_k)["topk_ids"].reshape(-1).tolist())
    layer = Layer(E, H, I, fmt, seed, used)
    x = bf16_dev(rng.standard_normal((T, H)))
    res = bf16_dev(rng.standard_normal((T, H))) if residual else None
    lg = torch.from_numpy(logits).to(DEV)
    out, ids, w = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, top_k, residual=res,
                                 buffers=buffers)
    torch.cuda.synchronize()
    o, bound, r = expected(layer, logits, host_f64(x), top_k,
                           None if res is None else host_f64(res))
    assert np.array_equal(ids.cpu().numpy(), r["topk_ids"])
    assert np.max(np.abs(w.cpu().numpy() - r["topk_w"])) <= 1e-6
    got = host_f64(out)
    assert np.all(np.isfinite(got)), "an expert nobody picked was read"
    bad = np.abs(got - o) > bound
    assert not bad.any(), (f"{int(bad.sum())}/{bad.size} outside; worst "
                           f"{np.max(np.abs(got - o) / bound):.2f} of the bound")
    first = out.clone()
    out2, _, _ = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, top_k, residual=res,
                                buffers=buffers)
    torch.cuda.synchronize()
    assert torch.equal(out2, first), "not deterministic"
    return layer, x, lg, res, first


@pytest.mark.parametrize("fmt", ["nf4", "nf4_bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,top_k,H,I", [
    (1, 1, 1, 64, 64), (1, 8, 2, 256, 128), (1, 64, 8, 320, 192), (2, 5, 5, 128, 64),
    (3, 100, 7, 64, 320), (7, 16, 4, 448, 128), (15, 3, 1, 192, 192), (16, 130, 8, 128, 64),
    (17, 6, 2, 256, 64), (33, 40, 3, 64, 128), (64, 8, 2, 128, 192), (64, 300, 8, 64, 64)])
def test_shapes(fmt, T, E, top_k, H, I):
    run_case(T, E, top_k, H, I, fmt, residual=T % 2 == 1)


@pytest.mark.parametrize("fmt", ["nf4", "nf4_bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,top_k,H,I", [
    (2, 4, 2, 4160, 64), (9, 3, 2, 6208, 128), (1, 3, 2, 8192, 64), (20, 3, 2, 7168, 64),
    (3, 4, 2, 64, 4160), (1, 3, 2, 128, 8192), (18, 2, 1, 64, 6144), (1, 2, 1, 5120, 5120)])
def test_long_rows(fmt, T, E, top_k, H, I):
    """Rows past 4096: items of one column tile, six to eight steps of K per
    wavefront."""
    run_case(T, E, top_k, H, I, fmt, residual=T % 2 == 1)


@pytest.mark.parametrize("T,E,top_k", [(3, 1024, 32), (12, 1024, 20), (8, 500, 32), (64, 16, 16),
                                       (64, 1024, 16), (9, 257, 1)])
def test_many_experts_and_picks(T, E, top_k):
    run_case(T, E, top_k, 64, 64, "nf4_bf16", residual=False)


@pytest.mark.parametrize("fmt", ["nf4", "nf4_bf16", "mxfp4"])
@pytest.mark.parametrize("T,H,I", [(11, 2112, 64), (13, 1728, 128), (17, 1344, 64), (7, 3264, 192)])
def test_items_that_do_not_divide_among_teams(fmt, T, H, I):
    """Every token on three experts of its own; some teams of a workgroup have
    an item less than others."""
    rng = np.random.default_rng(T)
    logits = rng.standard_normal((T, 3 * T)).astype(np.float32)
    for t in range(T):
        logits[t, 3 * t:3 * t + 3] += 20.0
    run_case(T, 3 * T, 3, H, I, fmt, False, logits=logits)


@pytest.mark.parametrize("T", [16, 40, 64])
def test_every_token_on_one_expert(T):
    """Groups of T rows (several matrix-core tiles) beside groups of none."""
    logits = np.tile(np.linspace(0, 1, 12, dtype=np.float32), (T, 1))
    logits[:, 5] = 9.0
    run_case(T, 12, 1, 128, 128, "nf4", True, logits=logits)


def test_equal_logits_take_the_lower_ids():
    run_case(9, 33, 4, 64, 64, "mxfp4", False, logits=np.zeros((9, 33), np.float32))


@pytest.mark.parametrize("T", [1, 8])
def test_decode_layer_shapes(T):
    run_case(T, 64, 8, 2048, 1024, "nf4", False)


def test_odd_widths_mxfp4():
    run_case(2, 16, 4, 2880, 2880, "mxfp4", True)


def test_buffers_serve_fewer_tokens_and_the_residual_may_be_the_output():
    H, I, E, k = 128, 64, 8, 2
    buf = gnf4.MoeLayerBuffers(20, E, k, H, I, DEV)
    for T in (20, 3, 17, 1):
        layer, x, lg, _, first = run_case(T, E, k, H, I, "nf4", False, buffers=buf)
    res = bf16_dev(np.random.default_rng(1).standard_normal((1, H)))
    want, _, _ = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, k, residual=res)
    buf1 = gnf4.MoeLayerBuffers(1, E, k, H, I, DEV)
    buf1.out.copy_(res)
    got, _, _ = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, k, residual=buf1.out,
                               buffers=buf1)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_no_tokens():
    layer = Layer(4, 64, 64, "nf4", 0)
    out, ids, w = gnf4.moe_layer(torch.empty((0, 4), device=DEV),
                                 torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                                 layer.gate_up, layer.down, 2)
    assert out.shape == (0, 64) and ids.shape == (0, 2) == w.shape


def test_tokens_do_not_depend_on_each_other():
    """NaN in one token's activations reaches that token's output only."""
    layer = Layer(6, 128, 64, "nf4", 3)
    rng = np.random.default_rng(4)
    lg = torch.from_numpy(rng.standard_normal((18, 6)).astype(np.float32)).to(DEV)
    x = bf16_dev(rng.standard_normal((18, 128)))
    ref, _, _ = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 2)
    x[4] = float("nan")
    got, _, _ = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 2)
    torch.cuda.synchronize()
    keep = [t for t in range(18) if t != 4]
    assert torch.equal(got[keep], ref[keep]) and torch.isnan(got[4]).all()


def test_mxfp4_scale_extremes():
    """Block scales over 40 binades in one row, and a NaN scale."""
    layer = Layer(2, 128, 64, "mxfp4", 5)
    rng = np.random.default_rng(6)
    p, s = layer.host["gu"]
    s[:] = rng.integers(90, 131, s.shape)
    layer.gate_up = (layer.gate_up[0], torch.from_numpy(s).to(DEV))
    logits = np.array([[0.0, 1.0], [1.0, 0.0]], np.float32)
    x = bf16_dev(rng.standard_normal((2, 128)) * 0.01)
    out, _, _ = gnf4.moe_layer(torch.from_numpy(logits).to(DEV), x, layer.gate_up, layer.down, 1)
    torch.cuda.synchronize()
    o, bound, _ = expected(layer, logits, host_f64(x), 1, None)
    assert np.all(np.abs(host_f64(out) - o) <= bound)
    ds = layer.down[1].clone()
    ds[1, 7, 0] = 255                      # expert 1, output column 7
    out, _, _ = gnf4.moe_layer(torch.from_numpy(logits).to(DEV), x, layer.gate_up,
                               (layer.down[0], ds), 1)
    torch.cuda.synchronize()
    nan = torch.isnan(out.float()).cpu().numpy()
    assert nan[0, 7] and nan.sum() == 1


def test_offsets_past_32_bits():
    """Stacks of more than 4 GB; the last expert is the one picked."""
    E, H, I = 520, 2048, 4096
    note("moe_layer 6.8 GB of codes")
    gen = torch.Generator(device=DEV).manual_seed(2)
    gp = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device=DEV, generator=gen)
    dp = torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, device=DEV, generator=gen)
    gs = torch.rand((E, 2 * I, H // 64), device=DEV, generator=gen) * 0.03 + 0.03
    ds = torch.rand((E, H, I // 64), device=DEV, generator=gen) * 0.03 + 0.03
    x = torch.randn((1, H), device=DEV, generator=gen).to(torch.bfloat16)
    lg = torch.zeros((1, E), device=DEV)
    lg[0, E - 1] = 3.0
    big, ids, _ = gnf4.moe_layer(lg, x, (gp, gs), (dp, ds), 1)
    one, _, _ = gnf4.moe_layer(torch.zeros((1, 1), device=DEV), x,
                               (gp[E - 1:].clone(), gs[E - 1:].clone()),
                               (dp[E - 1:].clone(), ds[E - 1:].clone()), 1)
    torch.cuda.synchronize()
    assert ids.item() == E - 1 and torch.equal(big, one)


# ----------------------------------------------------- streams, graphs, chains

def test_another_stream_and_graph_replays():
    layer = Layer(16, 256, 128, "nf4", 7)
    rng = np.random.default_rng(8)
    lgs = [torch.from_numpy(rng.standard_normal((5, 16)).astype(np.float32)).to(DEV)
           for _ in range(3)]
    xs = [bf16_dev(rng.standard_normal((5, 256))) for _ in range(3)]
    refs = [gnf4.moe_layer(l, x, layer.gate_up, layer.down, 3)[0] for l, x in zip(lgs, xs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    buf = gnf4.MoeLayerBuffers(5, 16, 3, 256, 128, DEV)
    with torch.cuda.stream(side):
        got, _, _ = gnf4.moe_layer(lgs[0], xs[0], layer.gate_up, layer.down, 3, buffers=buf)
    side.synchronize()
    assert torch.equal(got, refs[0])
    lg, x = lgs[0].clone(), xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 3, buffers=buf)
    for i in (1, 2, 0, 2):
        lg.copy_(lgs[i])
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, refs[i])
        eager, _, _ = gnf4.moe_layer(lgs[i], xs[i], layer.gate_up, layer.down, 3)
        torch.cuda.synchronize()
        assert torch.equal(eager, refs[i])


def test_two_calls_at_once_and_two_graphs():
    """Calls on two streams, and two graphs replayed side by side, each with
    buffers of its own."""
    layer = Layer(24, 512, 256, "nf4_bf16", 21)
    rng = np.random.default_rng(22)
    case = []
    for T in (3, 40):
        lg = torch.from_numpy(rng.standard_normal((T, 24)).astype(np.float32)).to(DEV)
        x = bf16_dev(rng.standard_normal((T, 512)))
        ref = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 4)[0]
        case.append((lg, x, ref, gnf4.MoeLayerBuffers(T, 24, 4, 512, 256, DEV),
                     torch.cuda.Stream(), torch.cuda.CUDAGraph()))
    torch.cuda.synchronize()
    for _ in range(20):
        for lg, x, _, buf, s, _ in case:
            with torch.cuda.stream(s):
                gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 4, buffers=buf)
    torch.cuda.synchronize()
    for lg, x, ref, buf, s, graph in case:
        assert torch.equal(buf.out, ref)
        with torch.cuda.graph(graph):
            gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 4, buffers=buf)
        buf.out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for _, _, _, _, s, graph in case:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, ref, buf, _, _ in case:
        assert torch.equal(buf.out, ref)


def test_layer_with_a_shared_int4_expert():
    """A layer as it is served: an int4 projection, a shared expert in int4
    whose output is the routed layer's residual, packed by the library."""
    T, E, k, H, I = 6, 16, 4, 256, 128
    rng = np.random.default_rng(9)
    layer = Layer(E, H, I, "nf4", 10)
    mats = {n: bf16_dev(rng.standard_normal(s) * 0.05)
            for n, s in (("o", (H, H)), ("gu", (2 * I, H)), ("dn", (H, I)), ("r", (E, H)))}
    q = {n: gnf4.int4_pack(w, 64, zero_points=n == "gu") for n, w in mats.items() if n != "r"}
    a = bf16_dev(rng.standard_normal((T, H)))
    x = gnf4.int4_linear(a, *q["o"])
    logits = x.float() @ mats["r"].float().t()
    shared = gnf4.int4_linear(gnf4.swiglu(gnf4.int4_linear(x, *q["gu"])), *q["dn"])
    out, _, _ = gnf4.moe_layer(logits, x, layer.gate_up, layer.down, k, residual=shared)
    torch.cuda.synchronize()
    o, bound, _ = expected(layer, logits.cpu().numpy(), host_f64(x), k, host_f64(shared))
    assert np.all(np.abs(host_f64(out) - o) <= bound)
    for n, src, dst in (("o", a, x),):
        p, s, z = q[n]
        ref = oracle.ref_int4_linear(host_f64(src), p.cpu().numpy(), host_f64(s))
        mag = np.abs(host_f64(src)) @ np.abs(oracle.ref_int4_unpack(p.cpu().numpy(), host_f64(s))).T
        assert np.all(np.abs(host_f64(dst) - ref) <= 2.0 ** -8 * np.abs(ref) + H * 2.0 ** -23 * mag)


def test_same_experts_as_the_separate_steps():
    """moe_layer against route_sort, grouped_gemm, swiglu and combine, within
    the separate steps' own tolerances (each of them rounds to bf16)."""
    T, E, k, H, I = 4, 8, 2, 256, 128
    layer = Layer(E, H, I, "nf4", 11)
    rng = np.random.default_rng(12)
    lg = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    x = bf16_dev(rng.standard_normal((T, H)))
    out, ids, w = gnf4.moe_layer(lg, x, layer.gate_up, layer.down, k)
    r = gnf4.route_sort(lg, k)
    y1 = gnf4.grouped_gemm(x, *layer.gate_up, r.group_sizes, r.group_expert_ids,
                           sorted_slots=r.sorted_slots, top_k=k)
    y2 = gnf4.grouped_gemm(gnf4.swiglu(y1), *layer.down, r.group_sizes, r.group_expert_ids)
    steps = gnf4.combine(y2, r.slot_rows, r.topk_w)
    torch.cuda.synchronize()
    assert torch.equal(ids, r.topk_ids) and torch.equal(w, r.topk_w)
    a, b = host_f64(out), host_f64(steps)
    assert np.all(np.abs(a - b) <= 0.03 * np.abs(b) + 0.02 * np.sqrt(np.mean(b * b)))


def test_refusals_on_the_gpu():
    layer = Layer(4, 64, 64, "nf4", 0)
    lg = torch.zeros((2, 4), device=DEV)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="expected cuda"):
        gnf4.moe_layer(lg.cpu(), x, layer.gate_up, layer.down, 2)
    with pytest.raises(gnf4.Gnf4Error, match="invalid argument"):
        gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 5)
    with pytest.raises(ValueError, match="buffers"):
        gnf4.moe_layer(lg, x, layer.gate_up, layer.down, 2,
                       buffers=gnf4.MoeLayerBuffers(1, 4, 2, 64, 64, DEV))
    with pytest.raises(gnf4.Gnf4Error, match="supported limits"):
        gnf4.moe_layer(torch.zeros((65, 4), device=DEV),
                       torch.zeros((65, 64), dtype=torch.bfloat16, device=DEV),
                       layer.gate_up, layer.down, 2)
