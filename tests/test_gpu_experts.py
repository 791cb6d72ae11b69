"""The experts' products, their gradients and the moves between token order and
expert order, against binary64."""
import ctypes

import numpy as np
import pytest
import torch

import moe_ref as ref
import nvfp4_quantization_moe_b200 as qz

pytestmark = pytest.mark.gpu
MX, NV = qz.FMT_MXFP8, qz.FMT_NVFP4


def stacked(g, E, N, K, fmt, std=0.1):
    w = (ref.randn(g, E, N, K) * std).to(torch.bfloat16).cuda()
    part = qz.quantize_expert_weights(w, fmt)
    return part


def weight64(part, e, K, fmt):
    q, sf, amax = part
    return ref.decode(q[e], sf[e], K, fmt == NV, True, None if amax is None else ref.decode_scale(amax[e].cpu()))


def tokens64(part, K, fmt):
    q, sf, amax = part
    return ref.decode(q, sf, K, fmt == NV, False, None if amax is None else ref.decode_scale(amax.cpu()).reshape(-1, 1))


def offsets_of(counts, align=1, gap=0):
    padded = (counts + align - 1) // align * align + gap
    return torch.cat([torch.zeros(1, dtype=torch.long), padded.cumsum(0)]).to(torch.int32)


def run_product(fmt, counts, N, K, *, seed=0, gather=True, gated=False, act=qz.ACT_NONE, bias=False, residual=False,
                pre=False, q=False, R=None, gap=0, pad=0, std=0.1, extra=0, max_ctas=0):
    """One call against binary64; buffers carry a canary in every row that is not live and in the columns past N."""
    g = ref.gen(seed + N + K)
    E = len(counts)
    counts = torch.tensor(counts)
    offsets = offsets_of(counts, gap=gap)
    S = int(offsets[-1]) + extra
    R = (max(S // 2, 1) if gather else S) if R is None else R
    x = qz.quantize_tokens((ref.randn(g, R, K)).to(torch.bfloat16).cuda(), fmt)
    w = stacked(g, E, N, K, fmt, std)
    up = stacked(g, E, N, K, fmt, std) if gated else None
    rows = torch.randint(0, R, (S,), generator=g, dtype=torch.int32) if gather else None
    if gather and S > 3:
        rows[1] = -1
        rows[2] = R
    b = (ref.randn(g, E, N)).to(torch.bfloat16) if bias else None
    ub = (ref.randn(g, E, N)).to(torch.bfloat16) if bias and gated else None
    r = ref.randn(g, S, N + pad).to(torch.bfloat16) if residual else None
    width = 2 * N if gated else N
    out = torch.full((S, N + pad), 7.5, dtype=torch.bfloat16).cuda()
    z = torch.full((S, width + pad), 7.5, dtype=torch.bfloat16).cuda() if pre else None
    oq = torch.full((S, N), 0x5A, dtype=torch.uint8).cuda() if q else None
    osf = torch.full((S, N // 32), 0x5A, dtype=torch.uint8).cuda() if q else None
    err = torch.zeros(1, dtype=torch.int32).cuda()
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    qz.expert_product(fmt, x, w, offsets.cuda(), counts.to(torch.int32).cuda(), out[:, :N], rows=cuda(rows), up=up,
                      bias=cuda(b), up_bias=cuda(ub), activation=act,
                      residual=None if r is None else r.cuda()[:, :N], pre=None if z is None else z[:, :width], q=oq,
                      sf=osf, err=err, max_ctas=max_ctas)
    torch.cuda.synchronize()
    assert err.item() == 0
    A = tokens64(x, K, fmt)
    A = torch.cat([A, torch.zeros(1, K, dtype=torch.float64)])
    live = torch.zeros(S, dtype=torch.bool)
    step = (K // 32 + 8) * 2.0 ** -22  # fp32 accumulation of one block of 32 products at a time, and the scales
    for e in range(E):
        at = torch.arange(int(offsets[e]), int(offsets[e]) + int(counts[e]))
        if not len(at):
            continue
        live[at] = True
        idx = rows[at].long() if gather else at
        a = A[torch.where((idx < 0) | (idx >= R), R, idx)]
        W = weight64(w, e, K, fmt)
        zz, dz = a @ W.T, (a.abs() @ W.abs().T) * step
        if b is not None:
            zz = zz + b[e].double()
            dz = dz + HALF32(zz)
        h, dh = ref.act(act, zz), 1.2 * dz
        if act in (qz.ACT_SILU, qz.ACT_GELU):
            # expf within 2 + 1.17 |argument| ulp (|argument| < 90 matters), a quotient of 2 ulp
            dh = dh + 112 * 2 * ref.HALF_F32 * h.abs()
        parts = [(zz, dz)]
        if gated:
            U = weight64(up, e, K, fmt)
            u, du = a @ U.T, (a.abs() @ U.abs().T) * step
            if ub is not None:
                u = u + ub[e].double()
                du = du + HALF32(u)
            parts.append((u, du))
            dh = dh * (u.abs() + du) + h.abs() * du
            h = h * u
        if r is not None:
            h = h + r[at, :N].double()
        # two fp32 roundings, then one to bf16 (of a value that may be off by dh)
        dh = dh + 2 * HALF32(h)
        ref.close(out[at.cuda(), :N], h, ref.HALF_BF16 * (h.abs() + dh) + dh + 1e-38, f"out of expert {e}")
        if z is not None:
            for i, (v, dv) in enumerate(parts):
                dv = dv + HALF32(v)
                ref.close(z[at.cuda(), i * N:(i + 1) * N], v, ref.HALF_BF16 * (v.abs() + dv) + dv + 1e-38, "pre")
    dead = (~live).cuda()
    assert (out[dead] == 7.5).all() and (out[:, N:] == 7.5).all()
    if z is not None:
        assert (z[dead] == 7.5).all() and (z[:, width:] == 7.5).all()
    if q:
        assert (oq[dead] == 0x5A).all() and (osf[dead] == 0x5A).all()
        lv = live.cuda()
        if live.any():
            want = qz.quantize_experts([out[:, :N][lv].contiguous()], MX, qz.SF_LINEAR)[0]
            assert torch.equal(oq[lv], want.q) and torch.equal(osf[lv].reshape(-1), want.sf.reshape(-1))
    return out, z, oq, osf


def HALF32(v):
    return ref.HALF_F32 * v.abs()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [3, 0, 130, 1], [128, 129, 127], [300, 0, 0, 5]])
@pytest.mark.parametrize("N,K", [(8, 32), (136, 96), (264, 352), (128, 128), (512, 544)])
def test_product(fmt, counts, N, K):
    run_product(fmt, counts, N, K)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", [qz.ACT_NONE, qz.ACT_RELU, qz.ACT_SILU, qz.ACT_GELU])
def test_product_epilogues(fmt, gated, act):
    for gather in (True, False):
        run_product(fmt, [70, 0, 33, 131], 160, 288, gather=gather, gated=gated, act=act, bias=True, residual=True,
                    pre=True, q=True, gap=3, pad=8, extra=5)
    run_product(fmt, [2, 9], 96, 64, gated=gated, act=act, q=True)
    run_product(fmt, [40], 72, 64, gated=gated, act=act, pre=True, gather=False)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("gated", [False, True])
def test_product_single_tokens(fmt, gated):
    """Decode: a token or a few per expert, many experts."""
    run_product(fmt, [1] * 8 + [0] * 24, 384, 1024, gated=gated, act=qz.ACT_SILU, q=True)
    run_product(fmt, [0] * 5 + [2, 0, 1, 4, 0, 16, 7], 256, 2048, gated=gated)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_many_tiles(fmt):
    """More tiles than CTAs, and any number of CTAs gives the same bits."""
    first = run_product(fmt, [700, 3, 0, 1025, 256], 776, 256, gated=True, act=qz.ACT_SILU, max_ctas=0)
    for ctas in (1, 7):
        again = run_product(fmt, [700, 3, 0, 1025, 256], 776, 256, gated=True, act=qz.ACT_SILU, max_ctas=ctas)
        assert torch.equal(first[0], again[0])


@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_long_contraction(fmt):
    run_product(fmt, [5, 150], 136, 4128, std=0.02)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_of_fused_weights(fmt):
    """Gate and up as views of one fused weight [E, 2N, K]."""
    g = ref.gen(4)
    E, N, K, S = 3, 256, 160, 90
    q, sf, amax = stacked(g, E, 2 * N, K, fmt)
    x = qz.quantize_tokens(ref.randn(g, S, K).to(torch.bfloat16).cuda(), fmt)
    half = qz.sf_bytes(N, K, fmt, qz.SF_SWIZZLED)
    offsets, counts = torch.tensor([0, 30, 60, 90], dtype=torch.int32).cuda(), torch.full((3,), 30, dtype=torch.int32).cuda()
    out = torch.zeros(S, N, dtype=torch.bfloat16).cuda()
    qz.expert_product(fmt, x, (q[:, :N], sf[:, :half], amax), offsets, counts, out, up=(q[:, N:], sf[:, half:], amax),
                      activation=qz.ACT_SILU)
    parts = []
    for lo in (0, N):
        p = (q[:, lo:lo + N].contiguous(), sf[:, lo // N * half:lo // N * half + half].contiguous(), amax)
        parts.append(p)
    want = torch.zeros_like(out)
    qz.expert_product(fmt, x, parts[0], offsets, counts, want, up=parts[1], activation=qz.ACT_SILU)
    assert torch.equal(out, want) and out.abs().sum() > 0


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("K", [96, 256])
def test_product_of_a_large_gather(fmt, K):
    """From 2048 slots on the rows are copied into slot order first: the same bits as gathering them in the product."""
    g = ref.gen(K)
    E, N, R, S = 3, 72, 300, 2500
    x = qz.quantize_tokens(ref.randn(g, R, K).to(torch.bfloat16).cuda(), fmt)
    w = stacked(g, E, N, K, fmt)
    rows = torch.randint(0, R, (S,), generator=g, dtype=torch.int32)
    rows[5], rows[2400] = -3, R + 7   # no row of x: zeros
    rows = rows.cuda()
    offsets = torch.tensor([0, 1000, 1010, S], dtype=torch.int32).cuda()
    counts = torch.tensor([990, 10, 1450], dtype=torch.int32).cuda()
    copied, gathered = (torch.full((S, N), 3.0, dtype=torch.bfloat16).cuda() for _ in range(2))
    qz.expert_product(fmt, x, w, offsets, counts, copied, rows=rows)
    half = 1200  # fewer slots at a time: no copy
    for lo, hi in ((0, half), (half, S)):
        o = (offsets[:E].long().clamp(lo, hi) - lo).to(torch.int32)
        end = (offsets[:E].long() + counts.long()).clamp(lo, hi) - lo
        qz.expert_product(fmt, x, w, o, (end - o.long()).to(torch.int32), gathered[lo:hi], rows=rows[lo:hi].contiguous())
    assert torch.equal(copied, gathered)
    assert (copied[5] == 0).all() and (copied[2400] == 0).all() and (copied[990:1000] == 3.0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("S", [300, 2500])  # gathered in the product, copied first
def test_slots_without_a_row_are_zeros_for_any_weight(fmt, gated, S):
    """A row of zeros times a weight of NaN or of an infinite amax: the slot has no row, so its products are 0."""
    g = ref.gen(S)
    E, N, K, R = 2, 64, 128, 50
    x = qz.quantize_tokens(ref.randn(g, R, K).to(torch.bfloat16).cuda(), fmt)
    w, up = stacked(g, E, N, K, fmt), stacked(g, E, N, K, fmt)
    for q, sf, amax in (w, up):
        if fmt == MX:
            q[0, 3, 5] = 0x7F  # NaN
        else:
            amax[0] = torch.inf
    rows = torch.randint(0, R, (S,), generator=g, dtype=torch.int32)
    none = [5, 7, 130, S - 1]
    rows[none] = torch.tensor([-1, R, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    out, pre = torch.full((S, N), 3.0, dtype=torch.bfloat16).cuda(), torch.full((S, 2 * N if gated else N), 3.0,
                                                                                dtype=torch.bfloat16).cuda()
    offsets = torch.tensor([0, S // 2], dtype=torch.int32).cuda()
    counts = torch.full((2,), S // 2, dtype=torch.int32).cuda()
    bias = ref.randn(g, E, N).to(torch.bfloat16).cuda()
    qz.expert_product(fmt, x, w, offsets, counts, out, rows=rows.cuda(), up=up if gated else None, bias=bias, pre=pre)
    for s in none:
        assert torch.equal(pre[s, :N], bias[2 * s // S]) and (not gated or (pre[s, N:] == 0).all())
        assert torch.equal(out[s], torch.zeros_like(bias[0]) if gated else bias[2 * s // S])
    assert torch.isnan(out[4, 3]) if fmt == MX else not torch.isfinite(out[4]).any()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_of_few_tokens_in_many_padded_slots(fmt):
    """A plan's unused slots are not copied: what their part of the workspace holds reaches no output."""
    g = ref.gen(17)
    E, N, K, T, k = 24, 264, 256, 60, 4
    x = qz.quantize_tokens(ref.randn(g, T, K).to(torch.bfloat16).cuda(), fmt)
    w = stacked(g, E, N, K, fmt)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    wide, tight = qz.plan_experts(ids, E, align=128), qz.plan_experts(ids, E)
    S = wide.rows.numel()
    p = qz.binding._Product(fmt=fmt, n=N, k=K, slots=S, x_rows=T, d_rows=0x1000, x_amax_per_row=1)
    need = qz.load().qz_product_bytes(ctypes.byref(p))
    assert need > 0 and S > 12 * T * k
    workspace = torch.full((need,), 0xFF, dtype=torch.uint8).cuda()  # NaN as codes, as scales and as an amax
    out = torch.full((S, N), 3.0, dtype=torch.bfloat16).cuda()
    qz.expert_product(fmt, x, w, wide.offsets, wide.counts, out, rows=wide.rows, workspace=workspace)
    want = torch.zeros(T * k, N, dtype=torch.bfloat16).cuda()
    qz.expert_product(fmt, x, w, tight.offsets, tight.counts, want, rows=tight.rows)
    assert torch.equal(out[wide.slots.long()], want[tight.slots.long()])
    assert (out[wide.rows < 0] == 3.0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_product_of_the_most_experts(fmt):
    counts = [0] * qz.MAX_ROUTE_EXPERTS
    for e, c in ((0, 1), (500, 3), (1000, 130), (1023, 2)):
        counts[e] = c
    run_product(fmt, counts, 16, 64, q=False)


def test_product_past_32_bits():
    """Rows whose element offsets pass 2^31 in out, pre, q and residual."""
    g = ref.gen(1)
    N, K, S, ld = 64, 64, 140000, 16384
    x = qz.quantize_tokens(ref.randn(g, 8, K).to(torch.bfloat16).cuda(), MX)
    w = stacked(g, 2, N, K, MX)
    big = torch.empty(S, ld, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(S, dtype=torch.int32).cuda()
    rows[-8:] = torch.arange(8, dtype=torch.int32).cuda()
    residual = ref.randn(g, 8, N).to(torch.bfloat16).cuda()
    big[-8:, N:2 * N] = residual
    offsets = torch.tensor([S - 8, S - 3, S], dtype=torch.int32).cuda()
    counts = torch.tensor([5, 3], dtype=torch.int32).cuda()
    qz.expert_product(MX, x, w, offsets, counts, big[:, :N], rows=rows, residual=big[:, N:2 * N], pre=big[:, 2 * N:3 * N])
    small = [torch.zeros(8, N, dtype=torch.bfloat16).cuda() for _ in range(2)]
    qz.expert_product(MX, x, w, offsets - (S - 8), counts, small[0], residual=residual, pre=small[1])
    assert torch.equal(big[-8:, :N], small[0]) and torch.equal(big[-8:, 2 * N:3 * N], small[1])
    assert small[0].abs().sum() > 0


def test_product_skips_bad_experts():
    g = ref.gen(6)
    x = qz.quantize_tokens(ref.randn(g, 40, 64).to(torch.bfloat16).cuda(), MX)
    w = stacked(g, 4, 64, 64, MX)
    out = torch.full((40, 64), 3.0, dtype=torch.bfloat16).cuda()
    err = torch.zeros(1, dtype=torch.int32).cuda()
    offsets = torch.tensor([0, 10, -5, 35], dtype=torch.int32).cuda()
    counts = torch.tensor([10, -1, 3, 6], dtype=torch.int32).cuda()  # negative count, negative offset, past the end
    qz.expert_product(MX, x, w, offsets, counts, out, err=err)
    assert err.item() == qz.DERR_SHAPE
    assert (out[10:] == 3.0).all() and not (out[:10] == 3.0).all()


def test_product_writes_nothing_without_rows():
    g = ref.gen(8)
    x = qz.quantize_tokens(ref.randn(g, 4, 64).to(torch.bfloat16).cuda(), MX)
    w = stacked(g, 2, 64, 64, MX)
    out = torch.full((4, 64), 3.0, dtype=torch.bfloat16).cuda()
    zero = torch.zeros(2, dtype=torch.int32).cuda()
    qz.expert_product(MX, x, w, zero, zero, out)
    assert (out == 3.0).all()
    qz.expert_product(MX, x, w, zero, zero, out[:0])


def test_product_on_a_stream_and_in_a_graph():
    g = ref.gen(10)
    x = qz.quantize_tokens(ref.randn(g, 64, 256).to(torch.bfloat16).cuda(), MX)
    w = stacked(g, 4, 256, 256, MX)
    offsets = torch.tensor([0, 16, 32, 48, 64], dtype=torch.int32).cuda()
    counts = torch.full((4,), 16, dtype=torch.int32).cuda()
    outs = [torch.zeros(64, 256, dtype=torch.bfloat16).cuda() for _ in range(4)]
    qz.expert_product(MX, x, w, offsets, counts, outs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, o in zip(streams, outs[1:3]):
        s.wait_stream(torch.cuda.current_stream())
        qz.expert_product(MX, x, w, offsets, counts, o, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qz.expert_product(MX, x, w, offsets, counts, outs[3])
    graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    counts.copy_(torch.tensor([1, 16, 0, 3], dtype=torch.int32))  # read on the device at each replay
    outs[3].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[3][16:32], outs[0][16:32]) and (outs[3][32:48] == 0).all() and (outs[3][1:16] == 0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("gated", [False, True])
def test_every_output_is_the_same_for_any_number_of_ctas(fmt, gated):
    outputs = [run_product(fmt, [300, 0, 7, 260], 288, 160, gated=gated, act=qz.ACT_GELU, bias=True, residual=True, pre=True,
                           q=True, max_ctas=ctas) for ctas in (0, 1, 5)]
    for other in outputs[1:]:
        for a, b in zip(outputs[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("gather", [False, True])
def test_product_of_no_rows(fmt, gather):
    """An x without rows: every slot has none, and its products are zeros."""
    g = ref.gen(12)
    N, K, S = 72, 96, 150
    w = stacked(g, 2, N, K, fmt)
    x = (torch.empty(0, K if fmt == MX else K // 2, dtype=torch.uint8).cuda(),
         torch.empty(0, K // (32 if fmt == MX else 16), dtype=torch.uint8).cuda(), torch.ones(1).cuda())
    b = ref.randn(g, 2, N).to(torch.bfloat16).cuda()
    rows = torch.arange(S, dtype=torch.int32).cuda() if gather else None
    out = torch.full((S, N), 3.0, dtype=torch.bfloat16).cuda()
    lists = torch.tensor([0, 131], dtype=torch.int32).cuda(), torch.tensor([130, 19], dtype=torch.int32).cuda()
    qz.expert_product(fmt, x, w, *lists, out, rows=rows, bias=b)
    assert torch.equal(out[:130], b[0].expand(130, N)) and torch.equal(out[131:], b[1].expand(19, N))
    assert (out[130] == 3.0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_data_gradient_of_columnwise_weights(fmt):
    """dA = dZ W as the product with the weights quantized down their columns, by the column-wise quantizer."""
    g = ref.gen(44)
    E, N, K, S = 3, 160, 288, 90
    W = (ref.randn(g, E, N, K) * 0.1).to(torch.bfloat16).cuda()
    parts = [qz.quantize_slots_colwise(W[e], fmt) for e in range(E)]
    region = qz.sf_bytes(K, N, fmt, qz.SF_SWIZZLED)
    w = (torch.stack([p[0] for p in parts]), torch.stack([p[1][:region] for p in parts]),
         torch.cat([p[2] for p in parts]) if fmt == NV else None)
    dz = qz.quantize_tokens(ref.randn(g, S, N).to(torch.bfloat16).cuda(), fmt)
    counts, offsets = torch.tensor([40, 0, 50], dtype=torch.int32), torch.tensor([0, 40, 40], dtype=torch.int32)
    out = torch.zeros(S, K, dtype=torch.bfloat16).cuda()
    qz.expert_product(fmt, dz, w, offsets.cuda(), counts.cuda(), out)
    A = tokens64(dz, N, fmt)
    for e in (0, 2):
        at = slice(int(offsets[e]), int(offsets[e] + counts[e]))
        T = weight64(w, e, N, fmt)  # [K, N]
        want, size = A[at] @ T.T, A[at].abs() @ T.abs().T
        tol = size * (N // 32 + 8) * 2.0 ** -22
        ref.close(out[at], want, tol + ref.HALF_BF16 * (want.abs() + tol) + 1e-38, "dA")
        # and close to the gradient of the unquantized weights: both operands are off by 2^-3 (e4m3: 2^-4) in norm at most
        exact = A[at] @ W[e].double().cpu()
        assert (want - exact).norm() < (2.0 ** -3 if fmt == NV else 2.0 ** -4) * exact.norm()


# --- weight gradient --------------------------------------------------------

@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [([1], 8, 8), ([0, 200, 3], 136, 264), ([128, 0, 129, 31], 264, 128),
                                        ([700, 64], 96, 520)])
def test_weight_grad(fmt, dtype, counts, N, K):
    g = ref.gen(N + K)
    E = len(counts)
    counts = torch.tensor(counts)
    offsets = offsets_of(counts, 128)
    S = int(offsets[-1]) + 128
    live = torch.zeros(S, 1)
    for e in range(E):
        live[int(offsets[e]):int(offsets[e]) + int(counts[e])] = 1
    dz = qz.quantize_slots_colwise((ref.randn(g, S, N) * live).to(torch.bfloat16).cuda(), fmt)
    x = qz.quantize_slots_colwise((ref.randn(g, S, K) * live).to(torch.bfloat16).cuda(), fmt)
    start = ref.randn(g, E, N, K).to(dtype)
    Z, X = (ref.decode(p[0], p[1], S, fmt == NV, True, None if p[2] is None else ref.decode_scale(p[2].cpu()))
            for p in (dz, x))
    for accumulate in (False, True):
        out = start.clone().cuda()
        qz.expert_weight_grad(fmt, dz, x, offsets.cuda(), counts.to(torch.int32).cuda(), out, accumulate=accumulate)
        for e in range(E):
            at = slice(int(offsets[e]), int(offsets[e]) + int(counts[e]))
            want, size = Z[:, at] @ X[:, at].T, Z[:, at].abs() @ X[:, at].abs().T
            tol = size * (int(counts[e]) // 32 + 8) * 2.0 ** -22
            if accumulate:
                want = want + start[e].double()
            tol = tol + (ref.HALF_F32 if dtype == torch.float32 else ref.HALF_BF16) * (want.abs() + tol) + 1e-38
            ref.close(out[e], want, tol, f"dW of expert {e}")


def test_weight_grad_refuses_unaligned_experts():
    g = ref.gen(2)
    S = 256
    dz = qz.quantize_slots_colwise(ref.randn(g, S, 32).to(torch.bfloat16).cuda(), MX)
    x = qz.quantize_slots_colwise(ref.randn(g, S, 32).to(torch.bfloat16).cuda(), MX)
    out = torch.full((3, 32, 32), 5.0).cuda()
    err = torch.zeros(1, dtype=torch.int32).cuda()
    offsets = torch.tensor([0, 64, 128], dtype=torch.int32).cuda()
    counts = torch.tensor([64, 64, 129], dtype=torch.int32).cuda()
    qz.expert_weight_grad(MX, dz, x, offsets, counts, out, err=err)
    assert err.item() == qz.DERR_ALIGN | qz.DERR_SHAPE
    assert (out[1:] == 5.0).all() and not (out[0] == 5.0).any()


# --- activation gradient ----------------------------------------------------

@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", [qz.ACT_NONE, qz.ACT_RELU, qz.ACT_SILU, qz.ACT_GELU])
@pytest.mark.parametrize("counts,N", [([1], 8), ([0, 200, 3], 136), ([64, 0, 0, 700], 520)])
def test_activation_grad(gated, act, counts, N):
    g = ref.gen(N + act)
    E = len(counts)
    counts = torch.tensor(counts)
    offsets = offsets_of(counts, 16)
    S, width = int(offsets[-1]) + 9, 2 * N if gated else N
    pre = (ref.randn(g, S, width) * 3).to(torch.bfloat16)
    dout = ref.randn(g, S, N).to(torch.bfloat16)
    wide = torch.full((S, width + 8), 7.5, dtype=torch.bfloat16).cuda()
    dbias = torch.full((E, width), 7.5).cuda()
    qz.expert_activation_grad(dout.cuda(), pre.cuda(), offsets.cuda(), counts.to(torch.int32).cuda(), wide[:, :width],
                              activation=act, gated=gated, dbias=dbias)
    z, d = pre[:, :N].double(), dout.double()
    want = d * ref.act_grad(act, z)
    if gated:
        want = torch.cat([want * pre[:, N:].double(), d * ref.act(act, z)], -1)
    live = torch.zeros(S, 1, dtype=torch.float64)
    for e in range(E):
        live[int(offsets[e]):int(offsets[e]) + int(counts[e])] = 1
    want = want * live
    # below 16 fp32 roundings of |d| (|u|) (1 + |z|) before the one to bf16; act' itself cancels
    size = d.abs() * 1.2 * (1 + z.abs())
    size = torch.cat([size * pre[:, N:].double().abs(), size], -1) if gated else size
    each = 16 * ref.HALF_F32 * size
    ref.close(wide[:, :width], want, each + ref.HALF_BF16 * (want.abs() + each) + 1e-38, "dpre")
    assert (wide[:, width:] == 7.5).all()
    for e in range(E):
        at = slice(int(offsets[e]), int(offsets[e]) + int(counts[e]))
        tol = each[at].sum(0) + (int(counts[e]) + 16) * ref.HALF_F32 * want[at].abs().sum(0) + 1e-38
        ref.close(dbias[e], want[at].sum(0), tol, "dbias")
    first = dbias.clone()
    qz.expert_activation_grad(dout.cuda(), pre.cuda(), offsets.cuda(), counts.to(torch.int32).cuda(), wide[:, :width],
                              activation=act, gated=gated, dbias=dbias)
    assert torch.equal(first, dbias)


def test_activation_grads_back_to_back_in_one_workspace():
    """The bias sums begin beside the gradient's end: each call adds its own pieces, not an earlier one's."""
    E, N, S = 12, 264, 3000
    counts = torch.tensor([250] * E, dtype=torch.int32)
    offsets = offsets_of(counts.long()).cuda()
    ws = torch.empty(qz.load().qz_activation_grad_bytes(S, N, 0, E), dtype=torch.uint8).cuda()
    pre = torch.ones(S, N, dtype=torch.bfloat16).cuda()
    # whole numbers: the sums are exact
    douts = [torch.randint(-8, 9, (S, N), generator=ref.gen(i)).to(torch.bfloat16).cuda() for i in range(4)]
    dpre, sums = torch.empty_like(pre), [torch.empty(E, N).cuda() for _ in range(40)]
    for i, s in enumerate(sums):
        qz.expert_activation_grad(douts[i % 4], pre, offsets, counts.cuda(), dpre, activation=qz.ACT_RELU, dbias=s,
                                  workspace=ws)
    want = [d.float().reshape(E, 250, N).sum(1) for d in douts]
    for i, s in enumerate(sums):
        assert torch.equal(s, want[i % 4]), i


@pytest.mark.parametrize("offsets,counts,bad", [([0, 100, 50], [100, 0, 60], 1), ([3, 10, 20], [7, 10, 5], 0),
                                                ([0, 40, 80], [30, -1, 5], 1), ([0, 60, 30], [40, 5, 110], 2),
                                                ([0, 0, 0], [0, 0, 129], 2)])
def test_activation_grad_skips_bad_experts(offsets, counts, bad):
    """Ranges that are not ascending, do not start at 0 or pass the end: reported, and nothing is written out of place."""
    S, N = 128, 16
    guard = torch.full((S + 64, N), 7.5, dtype=torch.bfloat16).cuda()
    sums = torch.full((4, N), 7.5).cuda()
    err = torch.zeros(1, dtype=torch.int32).cuda()
    one = torch.ones(S, N, dtype=torch.bfloat16).cuda()
    need = qz.load().qz_activation_grad_bytes(S, N, 0, 3)
    work = torch.full((need + 256,), 0x5A, dtype=torch.uint8).cuda()
    qz.expert_activation_grad(one, one, torch.tensor(offsets, dtype=torch.int32).cuda(),
                              torch.tensor(counts, dtype=torch.int32).cuda(), guard[:S], activation=qz.ACT_RELU,
                              dbias=sums[:3], workspace=work[:need], err=err)
    assert err.item() == qz.DERR_SHAPE
    assert (guard[S:] == 7.5).all() and (sums[3] == 7.5).all() and (work[need:] == 0x5A).all()
    assert (sums[bad] == 7.5).all()


@pytest.mark.parametrize("act", [qz.ACT_SILU, qz.ACT_GELU])
def test_activation_grad_against_differences(act):
    """dpre against central differences of the forward epilogue: x = 1 row of the identity, so pre = bias."""
    z = torch.linspace(-6, 6, 256).to(torch.bfloat16)
    n = z.numel()
    one = torch.zeros(1, n, dtype=torch.bfloat16)
    count, off = torch.ones(1, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    d = torch.zeros(1, n, dtype=torch.bfloat16).cuda()
    qz.expert_activation_grad(torch.ones_like(one).cuda(), z.reshape(1, n).cuda(), off, count, d, activation=act)
    h = 2.0 ** -4
    diff = (ref.act(act, z.double() + h) - ref.act(act, z.double() - h)) / (2 * h)
    ref.close(d[0], diff, ref.HALF_BF16 * diff.abs() + h * h / 6 * 1.5 + 1e-6, "dpre")


# --- activations of values that are not ordinary numbers ---------------------

def activated(act, z, gated):
    """expert_product's activation of the values z (as a bias on products of zeros), and expert_activation_grad's
    outputs for them: (act(z), act'(z)), gated also act(z) as du."""
    N, z = z.numel(), z.to(torch.bfloat16).reshape(1, -1).cuda()
    x = qz.quantize_tokens(torch.zeros(1, 32, dtype=torch.bfloat16).cuda(), MX)
    w = stacked(ref.gen(1), 1, N, 32, MX)
    off, cnt = torch.zeros(1, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda()
    out, one = torch.zeros(1, N, dtype=torch.bfloat16).cuda(), torch.ones(1, N, dtype=torch.bfloat16).cuda()
    kw = dict(up=w, up_bias=one) if gated else {}
    qz.expert_product(MX, x, w, off, cnt, out, bias=z, activation=act, **kw)
    d = torch.zeros(1, 2 * N if gated else N, dtype=torch.bfloat16).cuda()
    qz.expert_activation_grad(one, torch.cat([z, one], 1) if gated else z, off, cnt, d, activation=act, gated=gated)
    d = d[0].double().cpu()
    return (out[0].double().cpu(), d[:N]) + ((d[N:],) if gated else ())


def same_values(got, want):
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))


SPECIAL = torch.tensor([torch.nan, torch.inf, -torch.inf, 3e38, -3e38, 1e-38, -1e-38, 0.0, -0.0, 2.5, -2.5, 1.0, -1.0, 0.5,
                        -0.5, 64.0])


@pytest.mark.parametrize("gated", [False, True])
def test_relu_keeps_nan(gated):
    z = SPECIAL.to(torch.bfloat16).double()
    got = activated(qz.ACT_RELU, SPECIAL, gated)
    same_values(got[0], z.clamp(min=0))
    same_values(got[1], (z > 0).double())
    if gated:
        same_values(got[2], z.clamp(min=0))


def same_function(got, want, z, what):
    """NaN and infinities where the definition has them; elsewhere the rounding to bf16 and below 16 fp32 roundings of
    1.2 (1 + |z|), and of an exponential's argument (|z| from 64 on makes no difference any more)."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(torch.isinf(got), torch.isinf(want)) and torch.equal(got[torch.isinf(got)], want[torch.isinf(want)]), what
    on = torch.isfinite(want)
    size = 1.2 * (1 + z[on].abs().clamp(max=64))
    each = 16 * ref.HALF_F32 * size + 2 * 80 * ref.HALF_F32 * want[on].abs()
    ref.close(got[on], want[on], each + ref.HALF_BF16 * (want[on].abs() + each) + 1e-38, what)


@pytest.mark.parametrize("act", [qz.ACT_SILU, qz.ACT_GELU])
@pytest.mark.parametrize("gated", [False, True])
def test_activations_of_infinities(act, gated):
    """Both are inf at inf; at -inf the definitions' quotient and product are NaN."""
    z = SPECIAL.to(torch.bfloat16).double()
    want = z / (1 + torch.exp(-z)) if act == qz.ACT_SILU else ref.act(act, z)
    assert want[1] == torch.inf and torch.isnan(want[2]) and want[4] == 0
    got = activated(act, SPECIAL, gated)
    same_function(got[0], want, z, "act")
    if gated:
        same_function(got[2], want, z, "du")


@pytest.mark.parametrize("act", [qz.ACT_SILU, qz.ACT_GELU])
@pytest.mark.parametrize("gated", [False, True])
def test_derivatives_of_large_values(act, gated):
    """0 or 1 where the activation is flat or straight, up to the largest bf16."""
    z = torch.tensor([3e38, -3e38, 2e19, -2e19, 1e13, -1e13, 2e4, -2e4, 9e3, -9e3, 300.0, -300.0, 64.0, -64.0, 5.0, -5.0])
    got = activated(act, z, gated)
    z = z.to(torch.bfloat16).double()
    same_function(got[1], ref.act_grad(act, z), z, "act'")
    assert got[1][:12].tolist() == [1.0, 0.0] * 6


# --- dispatch and combine ---------------------------------------------------

@pytest.mark.parametrize("T,E,k,H,align", [(1, 4, 2, 8, 1), (1, 1, 1, 8, 128), (5, 7, 3, 72, 16), (64, 16, 8, 1032, 1),
                                           (37, 128, 8, 2048, 128), (300, 3, 1, 264, 32), (9, 60, 32, 520, 4)])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_and_combine(T, E, k, H, align, weighted):
    g = ref.gen(T + H)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if T > 4:
        ids[1] = -1
        ids[2, 0] = -1
    plan = qz.plan_experts(ids.cuda(), E, align=align)
    slots, rows = plan.slots.cpu().long(), plan.rows.cpu()
    S, pad = plan.rows.numel(), 16
    x, y = ref.randn(g, T, H + pad).to(torch.bfloat16), ref.randn(g, S, H).to(torch.bfloat16)
    w = ref.randn(g, T, k) if weighted else None
    r = ref.randn(g, T, H).to(torch.bfloat16) if weighted else None
    live = slots >= 0
    at = slots.clamp(min=0)
    ww = (w.double() if weighted else torch.ones(T, k, dtype=torch.float64)) * live
    cw = w.cuda() if weighted else None
    out = torch.full((T, H + pad), 7.5, dtype=torch.bfloat16).cuda()
    qz.combine_experts(y.cuda(), plan.slots, out[:, :H], weights=cw, residual=None if r is None else r.cuda())
    terms = ww.unsqueeze(-1) * y[at].double()
    want, size = terms.sum(1), terms.abs().sum(1)
    if r is not None:
        want, size = want + r.double(), size + r.double().abs()
    tol = (k + 1) * ref.HALF_F32 * size
    ref.close(out[:, :H], want, tol + ref.HALF_BF16 * (want.abs() + tol) + 1e-38, "combine")
    assert (out[:, H:] == 7.5).all()

    back = torch.full((S, H + pad), 7.5, dtype=torch.bfloat16).cuda()
    dots = torch.full((T, k), 7.5).cuda()
    qz.dispatch_experts(x.cuda()[:, :H], plan.slots, plan.rows, back[:, :H], weights=cw,
                        other=y.cuda() if weighted else None, dots=dots if weighted else None)
    want = torch.zeros(S, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if live[t, j]:
                want[slots[t, j]] = ww[t, j] * x[t, :H].double()
    ref.close(back[:, :H], want, ref.HALF_BF16 * want.abs() * (1 + 2.0 ** -15) + 1e-38, "dispatch")
    assert (back[rows < 0][:, :H] == 0).all() and (back[:, H:] == 7.5).all()
    if weighted:
        prod = x[:, :H].double().unsqueeze(1) * y[at].double() * live.unsqueeze(-1)
        # 8 products in a chain, 5 + 3 levels of a tree and ceil(H / 2048) passes
        ref.close(dots, prod.sum(-1), (20 + H // 2048) * ref.HALF_F32 * prod.abs().sum(-1) + 1e-38, "dots")


@pytest.mark.parametrize("H", [8, 264, 2056])
def test_dots_of_pairs_without_a_slot(H):
    """They are 0, also where the token's row holds NaN or infinities."""
    g = ref.gen(H)
    T, k, S = 6, 6, 40
    x = ref.randn(g, T, H).to(torch.bfloat16)
    x[0], x[1, H - 1], x[2, 0], x[3, H // 2] = torch.nan, torch.inf, -torch.inf, torch.nan
    slots = torch.arange(T * k, dtype=torch.int32).reshape(T, k)
    slots[0], slots[1], slots[2, ::2], slots[3, 1], slots[4] = -1, S, -7, -1, -1
    rows = torch.full((S,), -1, dtype=torch.int32)
    live = (slots >= 0) & (slots < S)
    for t in range(T):
        rows[slots[t][live[t]].long()] = t
    y, w = ref.randn(g, S, H).to(torch.bfloat16).cuda(), ref.randn(g, T, k).cuda()
    out, dots = torch.empty(S, H, dtype=torch.bfloat16).cuda(), torch.full((T, k), 7.5).cuda()
    qz.dispatch_experts(x.cuda(), slots.cuda(), rows.cuda(), out, weights=w, other=y, dots=dots)
    assert (dots.cpu()[~live] == 0).all()
    for t in (1, 2, 3):
        assert not torch.isfinite(dots.cpu()[t][live[t]]).any()


def test_dispatch_of_few_tokens_zeroes_many_slots():
    g = ref.gen(2)
    ids = torch.randint(0, 128, (3, 8), generator=g, dtype=torch.int32).cuda()
    plan = qz.plan_experts(ids, 128, align=128)
    x = ref.randn(g, 3, 264).to(torch.bfloat16).cuda()
    y = torch.full((plan.rows.numel(), 264), 7.5, dtype=torch.bfloat16).cuda()
    qz.dispatch_experts(x, plan.slots, plan.rows, y)
    live = plan.rows >= 0
    assert int(live.sum()) == 24 and (y[~live] == 0).all() and torch.equal(y[live], x[plan.rows[live].long()])


def test_combine_in_place_of_the_residual_and_empty_calls():
    g = ref.gen(1)
    r = ref.randn(g, 6, 64).to(torch.bfloat16).cuda()
    y = ref.randn(g, 12, 64).to(torch.bfloat16).cuda()
    slots = torch.arange(12, dtype=torch.int32).reshape(6, 2).cuda()
    want = torch.empty_like(r)
    qz.combine_experts(y, slots, want, residual=r)
    qz.combine_experts(y, slots, r, residual=r)
    assert torch.equal(r, want)
    qz.combine_experts(y, slots[:0], r[:0])
    empty = torch.full((12, 64), 3.0, dtype=torch.bfloat16).cuda()
    qz.dispatch_experts(r[:0], slots[:0], torch.full((12,), -1, dtype=torch.int32).cuda(), empty)
    assert (empty == 0).all()
    none = torch.full((6, 2), -1, dtype=torch.int32).cuda()
    qz.combine_experts(y, none, want)
    assert (want == 0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("raw", [False, True])
def test_quantizers_of_the_operands_on_another_stream(fmt, raw):
    """Their table of pointers belongs to the launch: nothing allocated meanwhile may take its place."""
    g = ref.gen(31)
    w = ref.randn(g, 5, 64, 96).to(torch.bfloat16).cuda()
    x = ref.randn(g, 128, 96).to(torch.bfloat16).cuda()
    want = (qz.quantize_expert_weights(w, fmt), qz.quantize_tokens(x, fmt), qz.quantize_slots_colwise(x, fmt))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for call, t in ((qz.quantize_expert_weights, w), (qz.quantize_tokens, x), (qz.quantize_slots_colwise, x)):
        got.append(call(t, fmt, stream=side.cuda_stream if raw else side))
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (16, 64, 512, 512, 512, 4096)]
    torch.cuda.synchronize()
    del junk
    regions = [(64, 96), None, (96, 128)]
    for a, b, region in zip(got, want, regions):
        assert torch.equal(a[0], b[0])
        n = qz.sf_bytes(*region, fmt, qz.SF_SWIZZLED) if region else None
        assert torch.equal(a[1][..., :n], b[1][..., :n])
        assert (a[2] is None) == (fmt == MX) and (a[2] is None or torch.equal(a[2], b[2]))


@pytest.mark.parametrize("raw", [False, True])
def test_calls_that_allocate_on_another_stream(raw):
    """Outputs and scratch of a call on a side stream: neither blocks that the current stream's work still uses, nor
    blocks that the current stream may take while the call runs."""
    g = ref.gen(41)
    T, E, k, H, N = 5000, 32, 4, 256, 96   # more than 16384 pairs: a plan with scratch; and a product with one
    logits = ref.randn(g, T, E).cuda()
    x = qz.quantize_tokens(ref.randn(g, T, H).to(torch.bfloat16).cuda(), MX)
    w = stacked(g, E, N, H, MX)
    dw = ref.randn(g, T, k).cuda()
    ids, weights = qz.route_experts(logits, k)
    plan = qz.plan_experts(ids, E, align=16)
    S = plan.rows.numel()
    pre, dout = ref.randn(g, S, N).to(torch.bfloat16).cuda(), ref.randn(g, S, N).to(torch.bfloat16).cuda()
    assert qz.load().qz_plan_bytes(T, k, E) > 0 and S >= 4096

    def calls(stream):
        """(outputs that are kept, outputs that are dropped at once) of each call."""
        out, dpre = (torch.zeros(S, N, dtype=torch.bfloat16).cuda() for _ in range(2))
        dbias = torch.zeros(E, N).cuda()
        if stream is not None:
            torch.cuda.current_stream().synchronize()
        kw = dict(stream=stream)
        yield lambda: qz.route_experts(logits, k, **kw)[1]  # the ids are freed while the router runs
        yield lambda: qz.route_experts_grad(logits, ids, dw, **kw)
        yield lambda: qz.plan_experts(ids, E, align=16, **kw).slots
        yield lambda: qz.expert_product(MX, x, w, plan.offsets, plan.counts, out, rows=plan.rows, **kw)
        yield lambda: (qz.expert_activation_grad(dout, pre, plan.offsets, plan.counts, dpre, activation=qz.ACT_SILU,
                                                 dbias=dbias, **kw), dbias)[1]

    want = [call().clone() for call in calls(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.zeros(1 << 26, device="cuda")
    sizes = [T * k * 4, T * E * 4, 4 * (2 * E + 1 + S + T * k), S * H, 1 << 20, 1 << 16]
    got, kept = [], []
    for call in calls(side.cuda_stream if raw else side):
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        for _ in range(20):
            busy.add_(1.0)
        for b in blocks:
            b.fill_(0xFF)   # still to come when the call is made
        kept.append([b.sum(dtype=torch.int64) for b in blocks])
        del b, blocks
        got.append(call())
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
        side.synchronize()
        del junk
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for sums in kept:   # nothing of a call's was written into what the current stream still read
        assert [int(v) for v in sums] == [255 * n for n in sizes]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_grad_is_the_same_for_any_number_of_ctas(fmt, dtype):
    g = ref.gen(51)
    counts, offsets = torch.tensor([200, 0, 384], dtype=torch.int32).cuda(), torch.tensor([0, 256, 256], dtype=torch.int32).cuda()
    live = torch.ones(640, 1)
    live[200:256] = 0
    dz, x = (qz.quantize_slots_colwise((ref.randn(g, 640, n) * live).to(torch.bfloat16).cuda(), fmt) for n in (264, 520))
    outs = [torch.ones(3, 264, 520, dtype=dtype).cuda() for _ in range(3)]
    for out, ctas in zip(outs, (0, 1, 5)):
        qz.expert_weight_grad(fmt, dz, x, offsets, counts, out, accumulate=True, max_ctas=ctas)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and outs[0].abs().sum() > 0


@pytest.mark.parametrize("fmt", [MX, NV])
def test_weight_grad_without_slots(fmt):
    empty = torch.empty(0, 64, dtype=torch.bfloat16).cuda()
    part = qz.quantize_slots_colwise(empty, fmt)
    lists = torch.zeros(3, dtype=torch.int32).cuda()
    out = torch.full((2, 64, 64), 3.0).cuda()
    qz.expert_weight_grad(fmt, part, part, lists, lists[:2], out, accumulate=True)
    assert torch.all(out == 3.0)
    qz.expert_weight_grad(fmt, part, part, lists, lists[:2], out)
    assert torch.all(out == 0.0)


# --- the layer --------------------------------------------------------------

def test_serving_layer():
    """Norm + quantize, route, plan, gated product, down product, combine: as a decode or prefill step runs."""
    T, E, k, H, I = 45, 8, 3, 256, 160
    g = ref.gen(21)
    x = ref.randn(g, T, H).to(torch.bfloat16).cuda()
    gate, up, down = (stacked(g, E, *s, MX) for s in ((I, H), (I, H), (H, I)))
    logits = ref.randn(g, T, E).to(torch.bfloat16).cuda()
    logits[7] = -torch.inf  # a padded token
    y, h = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(T, H, dtype=torch.uint8).cuda()
    sf = torch.empty(T, H // 32, dtype=torch.uint8).cuda()
    qz.rmsnorm_quantize(x, torch.zeros_like(x), torch.ones(H, dtype=torch.bfloat16).cuda(), 1e-6, y, h, MX, q, sf,
                        qz.SF_LINEAR)
    ids, w = qz.route_experts(logits, k)
    plan = qz.plan_experts(ids, E)
    S = plan.rows.numel()
    mid = torch.zeros(S, I, dtype=torch.bfloat16).cuda()
    mq = torch.zeros(S, I, dtype=torch.uint8).cuda()
    msf = torch.zeros(S, I // 32, dtype=torch.uint8).cuda()
    qz.expert_product(MX, (q, sf), gate[:2], plan.offsets, plan.counts, mid, rows=plan.rows, up=up[:2],
                      activation=qz.ACT_SILU, q=mq, sf=msf)
    o = torch.zeros(S, H, dtype=torch.bfloat16).cuda()
    qz.expert_product(MX, (mq, msf), down[:2], plan.offsets, plan.counts, o)
    out = torch.empty_like(x)
    qz.combine_experts(o, plan.slots, out, weights=w, residual=h)
    A = ref.decode(q, sf, H, False, False)
    M = ref.decode(mq, msf, I, False, False)
    want, size = h.double().cpu(), h.double().cpu().abs()
    ids, w, slots = ids.cpu(), w.double().cpu(), plan.slots.cpu()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                assert t == 7
                continue
            z = A[t] @ weight64(gate, e, H, MX).T
            m = ref.act(qz.ACT_SILU, z) * (A[t] @ weight64(up, e, H, MX).T)
            # the quantized hidden row: half a bf16 step, then half an e4m3 step (or of the block's smallest one)
            block = m.abs().reshape(-1, 32).amax(-1).repeat_interleave(32)
            ref.close(M[slots[t, j]], m, (ref.HALF_E4M3 + 2 * ref.HALF_BF16) * m.abs() + block * 2.0 ** -16 * 1.01
                      + 1e-4 * block, "hidden")
            term = w[t, j] * (M[slots[t, j]] @ weight64(down, e, I, MX).T)
            want[t] += term
            size[t] += term.abs()
    ref.close(out, want, 2 * ref.HALF_BF16 * size + 1e-4 * size, "layer")
    assert torch.equal(out[7], h[7])


def test_training_layer():
    """Forward with saved pre-activations, then every gradient, against autograd in binary64 on the quantized operands'
    values: the straight-through gradients of the quantizers."""
    T, E, k, H, I = 60, 4, 2, 128, 96
    g = ref.gen(33)
    x = ref.randn(g, T, H).to(torch.bfloat16).cuda()
    gate, up, down = ((ref.randn(g, E, *s) * 0.1).to(torch.bfloat16).cuda() for s in ((I, H), (I, H), (H, I)))
    logits = ref.randn(g, T, E).cuda()
    dy = ref.randn(g, T, H).to(torch.bfloat16).cuda()
    ids, w = qz.route_experts(logits, k)
    plan = qz.plan_experts(ids, E, align=128)
    S = plan.rows.numel()
    off, cnt, rows, slots = plan
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16).cuda()  # noqa: E731
    xs = qz.dispatch_experts(x, slots, rows, bf(S, H))
    pre, mid, o = bf(S, 2 * I), bf(S, I), bf(S, H)
    qg, qu, qd = (qz.quantize_expert_weights(v, MX) for v in (gate, up, down))
    qx = qz.quantize_tokens(x, MX)
    qz.expert_product(MX, qx, qg, off, cnt, mid, rows=rows, up=qu, activation=qz.ACT_SILU, pre=pre)
    qz.expert_product(MX, qz.quantize_tokens(mid, MX), qd, off, cnt, o)
    # backward
    do, dots = bf(S, H), torch.empty(T, k).cuda()
    qz.dispatch_experts(dy, slots, rows, do, weights=w, other=o, dots=dots)
    dlogits = qz.route_experts_grad(logits, ids, dots)
    dmid = bf(S, I)
    qdo = qz.quantize_tokens(do, MX)
    qz.expert_product(MX, qdo, qz.quantize_expert_weights(down.transpose(1, 2).contiguous(), MX), off, cnt, dmid)
    ddown = torch.zeros(E, H, I).cuda()
    cdo, cmid = qz.quantize_slots_colwise(do, MX), qz.quantize_slots_colwise(mid, MX)
    qz.expert_weight_grad(MX, cdo, cmid, off, cnt, ddown)
    dpre, dbias = bf(S, 2 * I), torch.zeros(E, 2 * I).cuda()
    qz.expert_activation_grad(dmid, pre, off, cnt, dpre, activation=qz.ACT_SILU, gated=True, dbias=dbias)
    dgate = torch.zeros(E, 2 * I, H).cuda()
    qz.expert_weight_grad(MX, qz.quantize_slots_colwise(dpre, MX), qz.quantize_slots_colwise(xs, MX), off, cnt, dgate)
    fused = torch.cat([gate, up], 1).transpose(1, 2).contiguous()
    dxs, dx = bf(S, H), bf(T, H)
    qz.expert_product(MX, qz.quantize_tokens(dpre, MX), qz.quantize_expert_weights(fused, MX), off, cnt, dxs)
    qz.combine_experts(dxs, slots, dx)

    X, G, U, D, L = (v.double().cpu().requires_grad_() for v in (x, gate, up, down, logits))
    p = torch.softmax(torch.gather(torch.softmax(L, -1).log(), 1, ids.cpu().long()), -1)
    ic = ids.cpu()
    bg = torch.zeros(E, 2 * I, dtype=torch.float64, requires_grad=True)
    out = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ic[t, j])
            z = torch.cat([G[e], U[e]]) @ X[t] + bg[e]
            out[t] = out[t] + p[t, j] * (D[e] @ (ref.act(2, z[:I]) * z[I:]))
    grads = torch.autograd.grad((out * dy.double().cpu()).sum(), [X, G, U, D, L, bg])
    # each operand of a product is off by at most half an e4m3 step (2^-4 of a value); the products behind one another
    # leave less than 3 of these, and their errors are independent: compared by norms
    got = [dx, dgate[:, :I], dgate[:, I:], ddown, dlogits, dbias]
    for name, a, b in zip(("dx", "dgate", "dup", "ddown", "dlogits", "dbias"), got, grads):
        rel = (a.double().cpu() - b).norm() / b.norm()
        assert rel < 3 * ref.HALF_E4M3, (name, float(rel))


def test_training_layer_in_nvfp4():
    """The same layer with NVFP4 operands: hidden rows in bf16, quantized between the products; every gradient."""
    T, E, k, H, I = 60, 4, 2, 128, 96
    g = ref.gen(35)
    x = ref.randn(g, T, H).to(torch.bfloat16).cuda()
    gate, up, down = ((ref.randn(g, E, *s) * 0.1).to(torch.bfloat16).cuda() for s in ((I, H), (I, H), (H, I)))
    logits = ref.randn(g, T, E).cuda()
    dy = ref.randn(g, T, H).to(torch.bfloat16).cuda()
    ids, w = qz.route_experts(logits, k)
    off, cnt, rows, slots = plan = qz.plan_experts(ids, E, align=128)
    S = plan.rows.numel()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16).cuda()  # noqa: E731
    qg, qu, qd = (qz.quantize_expert_weights(v, NV) for v in (gate, up, down))
    pre, mid, o, out = bf(S, 2 * I), bf(S, I), bf(S, H), bf(T, H)
    qz.expert_product(NV, qz.quantize_tokens(x, NV), qg, off, cnt, mid, rows=rows, up=qu, activation=qz.ACT_SILU, pre=pre)
    qz.expert_product(NV, qz.quantize_tokens(mid, NV), qd, off, cnt, o)
    qz.combine_experts(o, slots, out, weights=w, residual=x)
    # backward: the weights quantized down their columns
    def columns(v):
        parts = [qz.quantize_slots_colwise(v[e], NV) for e in range(E)]
        return tuple(torch.stack([p[i] for p in parts]) for i in (0, 1)) + (torch.cat([p[2] for p in parts]),)

    do, dots, dmid = bf(S, H), torch.empty(T, k).cuda(), bf(S, I)
    qz.dispatch_experts(dy, slots, rows, do, weights=w, other=o, dots=dots)
    dlogits = qz.route_experts_grad(logits, ids, dots)
    qz.expert_product(NV, qz.quantize_tokens(do, NV), columns(down), off, cnt, dmid)
    ddown = torch.zeros(E, H, I).cuda()
    qz.expert_weight_grad(NV, qz.quantize_slots_colwise(do, NV), qz.quantize_slots_colwise(mid, NV), off, cnt, ddown)
    dpre, dbias = bf(S, 2 * I), torch.zeros(E, 2 * I).cuda()
    qz.expert_activation_grad(dmid, pre, off, cnt, dpre, activation=qz.ACT_SILU, gated=True, dbias=dbias)
    dgate = torch.zeros(E, 2 * I, H).cuda()
    xs = qz.dispatch_experts(x, slots, rows, bf(S, H))
    qz.expert_weight_grad(NV, qz.quantize_slots_colwise(dpre, NV), qz.quantize_slots_colwise(xs, NV), off, cnt, dgate)
    dxs, dx = bf(S, H), bf(T, H)
    qz.expert_product(NV, qz.quantize_tokens(dpre, NV), columns(torch.cat([gate, up], 1)), off, cnt, dxs)
    qz.combine_experts(dxs, slots, dx)

    X, G, U, D, L = (v.double().cpu().requires_grad_() for v in (x, gate, up, down, logits))
    ic = ids.cpu()
    p = torch.softmax(torch.gather(L, 1, ic.long()), -1)
    bg = torch.zeros(E, 2 * I, dtype=torch.float64, requires_grad=True)
    want = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            z = torch.cat([G[ic[t, j]], U[ic[t, j]]]) @ X[t] + bg[ic[t, j]]
            want[t] = want[t] + p[t, j] * (D[ic[t, j]] @ (ref.act(2, z[:I]) * z[I:]))
    grads = torch.autograd.grad((want * dy.double().cpu()).sum(), [X, G, U, D, L, bg])
    # a quantized operand is off by 0.1 of its norm (steps of 0.5, 1 and 2 on values of which the largest of 16 is 6),
    # 2^-3 at most; fewer than eight of them, with independent errors, stand behind one another: sqrt(8) < 3
    got = [out.double() - x.double(), dx, dgate[:, :I], dgate[:, I:], ddown, dlogits, dbias]
    for name, a, b in zip(("out", "dx", "dgate", "dup", "ddown", "dlogits", "dbias"), got, (want.detach(), *grads)):
        rel = (a.double().cpu() - b).norm() / b.norm()
        assert rel < 3 * 2.0 ** -3, (name, float(rel))
