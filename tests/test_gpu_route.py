"""Router, its gradient and the expert order against binary64 definitions."""
import numpy as np
import pytest
import torch

import moe_ref as ref
import nvfp4_quantization_moe_b200 as qz

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = qz.SCORE_SOFTMAX, qz.SCORE_SIGMOID


def check_route(x, k, score, bias=None, groups=1, top=1, renorm=True, scale=1.0):
    ids, w = qz.route_experts(x, k, score=score, bias=bias, n_groups=groups, top_groups=top, renormalize=renorm,
                              scale=scale)
    rid, rw = ref.route(x, k, score == SIGMOID, bias, groups, top, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # expf within 2 ulp for x - max, a sum of up to 1024 terms in a tree (10 roundings), a quotient and a
    # factor: below 16 roundings; the logit difference is exact or rounded once, |x - max| 2^-24 relative
    rw = torch.from_numpy(rw)
    span = 16 + ref.clean(x.cpu()).clamp(min=-200).abs().amax(-1, keepdim=True)
    ref.close(w, rw, span * ref.HALF_F32 * 2 * rw.abs() + 1e-37, "weights")
    return ids, w


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 31, 5), (65, 33, 8), (7, 128, 8), (9, 256, 8), (5, 300, 32),
                                   (2, 1024, 32), (130, 60, 4)])
@pytest.mark.parametrize("score,biased,renorm", [(SOFTMAX, False, True), (SOFTMAX, True, False), (SIGMOID, True, True),
                                                 (SIGMOID, False, False), (SOFTMAX, False, False)])
def test_route(T, E, k, score, biased, renorm, dtype):
    g = ref.gen(T * 7 + E)
    x = (ref.randn(g, T, E) * 2).to(dtype).cuda()
    bias = (ref.randn(g, E) * 0.3).cuda() if biased else None
    check_route(x, k, score, bias, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (64, 4, 1, 6), (32, 32, 7, 7), (62, 2, 1, 3), (96, 3, 3, 4),
                                            (160, 8, 3, 6)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(E, groups, top, k, score, biased):
    g = ref.gen(E + groups)
    x = ref.randn(g, 67, E).to(torch.bfloat16).cuda()
    bias = (ref.randn(g, E) * 0.2).cuda() if biased else None
    check_route(x, k, score, bias, groups, top)


@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_index(biased):
    g = ref.gen(3)
    x = torch.randint(-2, 3, (40, 96), generator=g).float().cuda()
    x[0] = 0.0
    x[1, ::2] = -0.0
    bias = torch.zeros(96).cuda() if biased else None
    for score in (SOFTMAX, SIGMOID):
        check_route(x, 8, score, bias)
        check_route(x, 8, score, bias, groups=8, top=3)


def test_scores_closer_than_fp32_are_told_apart():
    """Biased scores that differ by less than an fp32 step: the order is binary64's."""
    x = torch.zeros(4, 64)
    x[:, 40] = 2.0 ** -26           # sigmoid 0.5 + 2^-28, which is 0.5 in fp32
    x[1, 7] = 2.0 ** -25
    x[2] = 30.0 + torch.arange(64) * 0.0625  # all round to 1 in fp32
    bias = torch.zeros(64)
    bias[5] = 2.0 ** -29
    ids, _ = check_route(x.cuda(), 4, SIGMOID, bias.cuda())
    assert ids[0, 0].item() == 40 and ids[1, 0].item() == 7


@pytest.mark.parametrize("at", [-85.0, -70.0, -59.0, -46.0, -30.0, -12.0, -1.0])
def test_close_groups_and_biased_scores_of_small_sigmoids(at):
    """Their fp32 values are off by more, relative to themselves, the further the logits are below 0."""
    if at == -46.0:
        check_route(torch.tensor([[-46.489601, -46.718143, -46.608604, -46.586235]]).cuda(), 1, SIGMOID, groups=2)
    g = ref.gen(int(-at))
    T = 1500
    logit = lambda p: torch.log(p) - torch.log1p(-p)  # noqa: E731
    # two groups of two: the last logit makes their sums equal but for its own rounding
    x = (at + 2 * torch.rand(T, 1, generator=g) - 0.4 * torch.rand(T, 4, generator=g)).double()
    s = torch.sigmoid(x.float().double())
    x[:, 3] = logit((s[:, 0] + s[:, 1] - s[:, 2]).clamp(min=float(s.min()) / 4))
    check_route(x.float().cuda(), 1, SIGMOID, groups=2)
    # biases of the scores' size: expert j's logit makes its biased score expert 0's but for its own rounding
    size = float(torch.sigmoid(torch.tensor(at, dtype=torch.float64)))
    bias = (torch.rand(40, generator=g) * size).float()
    x = (at + 2 * torch.rand(T, 40, generator=g)).double()
    s0 = torch.sigmoid(x[:, :1].float().double())
    x[:, 1:4] = logit((s0 + bias[0].double() - bias[1:4].double()).clamp(min=size / 8))
    check_route(x.float().cuda(), 6, SIGMOID, bias.cuda())


@pytest.mark.parametrize("E", [256, 1000, 1024])
def test_close_biased_scores_of_long_softmax_rows(E):
    """A sum whose small terms are lost in a row of additions to a large one: the choice is binary64's all the same."""
    g = ref.gen(E)
    T = 300
    x = (-16.65 + 0.02 * torch.rand(T, E, generator=g)).float()
    x[:, 0] = 0.0
    x[T // 2:, 0] = x[T // 2:, 32] = -4.0 * torch.rand(T - T // 2, generator=g)
    p = ref.scores(x.double(), False)
    # biases that make eight experts' biased scores those of expert 0 in one row, and close in the others
    bias = torch.zeros(E)
    bias[100:108] = (p[3, 0] - p[3, 100:108]).float()
    check_route(x.cuda(), 6, SOFTMAX, bias.cuda(), renorm=False)
    check_route(x.cuda(), 6, SOFTMAX, bias.cuda(), groups=4, top=2)


@pytest.mark.parametrize("mask", [-1e9, -3.4028234663852886e38, -50.0])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (128, 1, 1, 8), (60, 4, 2, 6), (40, 1, 1, 32)])
def test_experts_masked_by_a_finite_bias(mask, E, groups, top, k):
    """Disabled experts, whole groups of them, and rows where too few others are left, so that masked ones are chosen."""
    g = ref.gen(E)
    x = ref.randn(g, 60, E).float()
    x[7] = 0.25
    x[8:30] = (x[8:30] * 4).round() / 4  # many ties
    for off in ([3], list(range(E // 2)), list(range(E - 4))):
        bias = (ref.randn(g, E) * 0.1).float()
        bias[5] = bias[6]
        bias[off] = mask
        for score in (SOFTMAX, SIGMOID):
            check_route(x.cuda(), k, score, bias.cuda(), groups, top)
        bias -= 3.0  # every biased score below 0
        check_route(x.cuda(), k, SIGMOID, bias.cuda(), groups, top)
        bias[[9, 11]] = torch.inf  # always chosen first, the lower one before the other
        check_route(x.cuda(), k, SIGMOID, bias.cuda(), groups, top)


def test_masked_experts():
    g = ref.gen(5)
    x = ref.randn(g, 12, 40)
    x[0] = -torch.inf                     # nothing left
    x[1, 3:] = -torch.inf                 # fewer than top_k
    x[2, ::2] = torch.nan
    x[3] = torch.nan
    x[4, 9] = torch.inf
    x[5, 10:12] = torch.inf
    x[6] = torch.finfo(torch.float32).min
    x[7, 1:] = -1e4
    x[8] = -500.0                         # every sigmoid underflows fp32
    bias = ref.randn(g, 40) * 0.1
    bias[17] = -torch.inf
    bias[18] = torch.nan
    for score in (SOFTMAX, SIGMOID):
        for b in (None, bias.cuda()):
            for renorm in (True, False):
                ids, w = check_route(x.cuda(), 6, score, b, renorm=renorm)
                assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[3] == -1).all()
                check_route(x.cuda(), 6, score, b, groups=4, top=2, renorm=renorm)
    xb = x.to(torch.bfloat16).cuda()
    check_route(xb, 6, SOFTMAX)


def test_strided_logits_stream_and_graph():
    g = ref.gen(9)
    wide = ref.randn(g, 33, 200).cuda()
    x = wide[:, 3:131]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = check_route(x, 8, SOFTMAX)
    with torch.cuda.stream(s):
        ids2, w2 = qz.route_experts(x, 8)
    s.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gi, gw = qz.route_experts(x, 8)
        plan = qz.plan_experts(gi, 128, align=16)
    for seed in (1, 2):
        wide.copy_(ref.randn(ref.gen(seed), 33, 200))
        graph.replay()
        torch.cuda.synchronize()
        ids, w = qz.route_experts(x, 8)
        assert torch.equal(gi, ids) and torch.equal(gw, w)
        for a, b in zip(plan, ref.plan(ids.cpu().numpy(), 128, 16)):
            assert np.array_equal(a.cpu().numpy(), b)


# --- gradient ---------------------------------------------------------------

def grad_reference(x, ids, g, sigmoid, renorm, scale):
    x = x.double().cpu().requires_grad_()
    p = torch.sigmoid(x) if sigmoid else torch.softmax(x, -1)
    live = ids.cpu() >= 0
    w = torch.where(live, torch.gather(p, 1, ids.cpu().long().clamp(min=0)), 0.0)
    if renorm:
        w = w / w.sum(-1, keepdim=True)
    return torch.autograd.grad((w * scale * g.double().cpu() * live).sum(), x)[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 33, 5), (66, 128, 8), (3, 256, 8), (2, 1024, 32)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad(T, E, k, score, renorm, dtype):
    g = ref.gen(E + k)
    x = (ref.randn(g, T, E) * 2).to(dtype).cuda()
    ids = torch.topk(x.float(), k, dim=-1).indices.to(torch.int32)
    dw = ref.randn(g, T, k).cuda()
    got = qz.route_experts_grad(x, ids, dw, score=score, renormalize=renorm, scale=2.5)
    want = grad_reference(x, ids, dw, score == SIGMOID, renorm, 2.5)
    # products of weights <= 1 and 2.5 |g|, sums of up to 32 of them: below 64 fp32 roundings of the largest term
    size = 2.5 * dw.double().cpu().abs().amax(-1, keepdim=True)
    tol = 64 * ref.HALF_F32 * size + (ref.HALF_BF16 * want.abs() if dtype == torch.bfloat16 else 0)
    ref.close(got, want, tol, "dlogits")


def test_route_grad_repeated_and_missing_choices():
    g = ref.gen(1)
    x = ref.randn(g, 4, 20).cuda()
    ids = torch.tensor([[3, 3, 3], [5, -1, 7], [-1, -1, -1], [0, 19, 0]], dtype=torch.int32).cuda()
    dw = ref.randn(g, 4, 3).cuda()
    for score in (SOFTMAX, SIGMOID):
        got = qz.route_experts_grad(x, ids, dw, score=score, renormalize=False)
        want = grad_reference(x, ids, dw, score == SIGMOID, False, 1.0)
        ref.close(got, want, 64 * ref.HALF_F32 * 3, "dlogits")
        assert (got[2] == 0).all()
        again = qz.route_experts_grad(x, ids, dw, score=score, renormalize=False)
        assert torch.equal(got, again)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_against_differences(score, renorm):
    g = ref.gen(11)
    x = ref.randn(g, 1, 16).cuda()
    x[0, [2, 5, 9]] += 4  # the choice stays the same under the steps below
    dw = ref.randn(g, 1, 3).cuda()
    ids, _ = qz.route_experts(x, 3, score=score, renormalize=renorm)
    got = qz.route_experts_grad(x, ids, dw, score=score, renormalize=renorm)
    h = 2.0 ** -5
    step = torch.cat([x + h * torch.eye(16).cuda(), x - h * torch.eye(16).cuda()])
    i, w = qz.route_experts(step, 3, score=score, renormalize=renorm)
    back = torch.zeros(32, 16, dtype=torch.float64).cuda().scatter_(1, i.long(), w.double())
    loss = (back[:, ids[0].long()] * dw.double()).sum(-1)
    diff = (loss[:16] - loss[16:]) / (2 * h)
    # third derivatives of a (renormalized) weight stay below 1: h^2 / 6 per unit of |g|; fp32 weights over 2h
    tol = float(dw.abs().sum()) * (h * h / 6 + 4 * ref.HALF_F32 / h)
    ref.close(got[0], diff, tol, "dlogits")


def test_route_grad_of_tiny_scores():
    """Sigmoids far below fp32's range keep their ratios, and their gradients."""
    x = torch.tensor([[-200.0, -201.0, -199.5, -400.0], [-30.0, -31.0, -29.0, -90.0]]).cuda()
    ids, w = check_route(x, 3, SIGMOID)
    dw = torch.tensor([[1.0, -2.0, 0.5], [3.0, 1.0, -1.0]]).cuda()
    got = qz.route_experts_grad(x, ids, dw, score=SIGMOID)
    ref.close(got, grad_reference(x, ids, dw, True, True, 1.0), 64 * ref.HALF_F32 * 3, "dlogits")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_route_grad_of_one_renormalized_choice_is_zero(score, dtype):
    """Its weight is the constant ``scale``: w = s / s, and g - g w = 0 exactly."""
    g = ref.gen(13)
    x = (ref.randn(g, 300, 64) * 2).to(dtype).cuda()
    x[0] = -200.0
    ids, w = qz.route_experts(x, 1, score=score, scale=2.5)
    assert (w == 2.5).all()
    got = qz.route_experts_grad(x, ids, ref.randn(g, 300, 1).cuda(), score=score, scale=2.5)
    assert (got == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E,groups", [(128, 1), (128, 4), (256, 8), (256, 32), (512, 2), (1024, 16)])
def test_router_of_rows_that_wide_loads_cannot_read(dtype, score, E, groups):
    """Rows from an odd element on (or with an odd stride, or an odd bias) are read otherwise: the same choice."""
    T, k = 70, 8
    g = ref.gen(E + groups)
    x = ref.randn(g, T, E).to(dtype).cuda()
    x[3] = -torch.inf
    x[4, : E - 2] = torch.nan
    bias = (ref.randn(g, E) * 0.1).cuda() if groups > 1 else None
    kw = dict(score=score, n_groups=groups, top_groups=(groups + 1) // 2, renormalize=groups != 4)
    ids, w = qz.route_experts(x, k, bias=bias, **kw)
    wide = torch.zeros(T, E + 1, dtype=dtype).cuda()
    wide[:, 1:] = x
    flat = torch.zeros(T * E + 1, dtype=dtype).cuda()
    flat[1:] = x.reshape(-1)
    others = [(wide[:, 1:], bias), (flat[1:].view(T, E), bias)]
    if bias is not None:
        odd = torch.zeros(E + 1).cuda()
        odd[1:] = bias
        others.append((x, odd[1:]))
    for y, b in others:
        ids2, w2 = qz.route_experts(y, k, bias=b, **kw)
        assert torch.equal(ids, ids2)
        # a softmax's sum in another order: at most 32 + 5 additions on either side
        ref.close(w2, w.double().cpu(), 2 * 37 * 2 * ref.HALF_F32 * w.double().cpu().abs(), "weights")


# --- expert order -----------------------------------------------------------

@pytest.mark.parametrize("T,E,k,align", [(0, 4, 2, 8), (1, 1, 1, 1), (1, 128, 8, 128), (5, 7, 3, 16), (333, 60, 4, 1),
                                         (1024, 128, 8, 128), (1025, 256, 8, 32), (3000, 1024, 8, 4), (70000, 16, 2, 128),
                                         (8192, 1, 1, 1024), (32, 1024, 8, 64), (33, 8, 8, 1), (257, 1, 1, 1),
                                         (100, 1024, 8, 8), (2048, 300, 8, 16), (2049, 1000, 8, 1)])
def test_plan(T, E, k, align):
    g = ref.gen(T + E)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if T > 4:
        ids[2] = -1
        ids[3, 0] = E           # outside: no slot
        ids[4] = ids[4, 0]      # one expert several times
    plan = qz.plan_experts(ids.cuda(), E, align=align)
    assert plan.rows.numel() == qz.plan_slots(T, k, E, align)
    for name, a, b in zip(plan._fields, plan, ref.plan(ids.numpy(), E, align)):
        assert np.array_equal(a.cpu().numpy(), b), name


def test_plan_of_one_expert_and_of_none():
    ids = torch.full((9000, 2), 3, dtype=torch.int32).cuda()
    plan = qz.plan_experts(ids, 8, align=128)
    assert plan.counts.tolist() == [0, 0, 0, 18000, 0, 0, 0, 0]
    assert torch.equal(plan.slots.reshape(-1).cpu(), torch.arange(18000, dtype=torch.int32))
    plan = qz.plan_experts(torch.full_like(ids, -1), 8, align=128)
    assert plan.counts.sum() == 0 and plan.offsets.sum() == 0 and (plan.rows == -1).all() and (plan.slots == -1).all()


@pytest.mark.parametrize("T", [20, 300, 4000])  # one CTA, one cluster, two launches
def test_plan_in_a_graph(T):
    E, k = 40, 8
    g = ref.gen(T)
    ids = torch.zeros(T, k, dtype=torch.int32).cuda()
    plan = qz.plan_experts(ids, E, align=16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = qz.plan_experts(ids, E, align=16)
    for _ in range(3):
        new = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
        ids.copy_(new)
        graph.replay()
        for name, a, b in zip(plan._fields, plan, ref.plan(new.numpy(), E, 16)):
            assert np.array_equal(a.cpu().numpy(), b), name


def test_plans_back_to_back_in_one_workspace():
    """The second launch begins beside the first one's end: every plan counts its own choices, not an earlier one's."""
    E, k, T = 200, 4, 20000
    g = ref.gen(77)
    lists = [torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32) for _ in range(4)]
    lists[1].clamp_(max=3)
    sorted_ = [ref.plan(i.numpy(), E, 8) for i in lists]
    ids = [i.cuda() for i in lists]
    ws = torch.empty(qz.load().qz_plan_bytes(T, k, E), dtype=torch.uint8).cuda()
    plans = [qz.plan_experts(ids[i % 4], E, align=8, workspace=ws) for i in range(40)]
    for i, plan in enumerate(plans):
        for name, a, b in zip(plan._fields, plan, sorted_[i % 4]):
            assert np.array_equal(a.cpu().numpy(), b), (i, name)
