"""Host side of the mixture-of-experts entry points, without a GPU: every
refusal is returned before any launch, sizes of the plan, ctypes mirrors of the
structs, and the binding's own checks."""
import contextlib
import ctypes
import os
import subprocess

import pytest
import torch

import nvfp4_quantization_moe_b200 as qz
from nvfp4_quantization_moe_b200 import build as qzbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A = 0x10000
BAD, ALIGN, OK = qz.QZ_ERR_INVALID_ARG, qz.QZ_ERR_ALIGNMENT, qz.QZ_OK


@pytest.fixture(scope="module")
def lib():
    qzbuild.build()
    return qz.load()


def test_structs_match_the_header(tmp_path):
    b = qz.binding
    mirrors = {"qz_router": b._Router, "qz_product": b._Product, "qz_weight_grad": b._WeightGrad}
    limits = {"QZ_MAX_ROUTE_EXPERTS": b.MAX_ROUTE_EXPERTS, "QZ_MAX_TOP_K": b.MAX_TOP_K, "QZ_MAX_GROUPS": b.MAX_GROUPS,
              "QZ_TYPE_BF16": b.TYPE_BF16, "QZ_TYPE_F32": b.TYPE_F32, "QZ_SCORE_SOFTMAX": b.SCORE_SOFTMAX,
              "QZ_SCORE_SIGMOID": b.SCORE_SIGMOID, "QZ_ACT_NONE": b.ACT_NONE, "QZ_ACT_RELU": b.ACT_RELU,
              "QZ_ACT_SILU": b.ACT_SILU, "QZ_ACT_GELU": b.ACT_GELU}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "qz.h"', "int main(void) {"]
    for cname, cls in mirrors.items():
        lines.append(f'  printf("{cname}.size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    lines += [f'  printf("{n} %d\\n", (int)({n}));' for n in limits] + ["  return 0;", "}"]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for name, value in limits.items():
        assert int(got[name]) == value, name
    for cname, cls in mirrors.items():
        assert int(got[cname + ".size"]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, (cname, f)


def test_router_refusals(lib):
    def route(T=4, E=16, ld=None, kind=0, x=A, bias=None, ids=A, w=A, k=2, score=0, groups=1, top=1, scale=1.0, r=True):
        router = qz.binding._Router(score, k, groups, top, 1, scale)
        return lib.qz_route_experts(P(x), kind, T, E, E if ld is None else ld, P(bias), ctypes.byref(router) if r else None,
                                    P(ids), P(w), None)

    for kw in (dict(T=-1), dict(T=2 ** 27), dict(E=0), dict(E=1025), dict(ld=15), dict(kind=2), dict(x=None), dict(ids=None),
               dict(w=None), dict(k=0), dict(k=17), dict(k=33, E=64), dict(score=2), dict(groups=0), dict(groups=3),
               dict(groups=64, E=64), dict(groups=4, top=0), dict(groups=4, top=5), dict(groups=4, top=1, k=5),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(r=False)):
        assert route(**kw) == BAD, kw
    for kw in (dict(x=A + 1), dict(x=A + 2, kind=1), dict(bias=A + 2), dict(ids=A + 1), dict(w=A + 2)):
        assert route(**kw) == ALIGN, kw
    assert route(T=0) == OK and route(T=0, x=None, ids=None, w=None) == OK

    def grad(T=4, E=16, ldd=16, ids=A, g=A, d=A, k=2, score=0, x=A):
        router = qz.binding._Router(score, k, 1, 1, 1, 1.0)
        return lib.qz_route_experts_grad(P(x), 0, T, E, E, ctypes.byref(router), P(ids), P(g), P(d), ldd, None)

    for kw in (dict(ldd=15), dict(ids=None), dict(g=None), dict(d=None), dict(k=17), dict(score=-1), dict(x=None)):
        assert grad(**kw) == BAD, kw
    assert grad(d=A + 1) == ALIGN and grad(ids=A + 2) == ALIGN and grad(T=0) == OK


def test_plan_sizes_and_refusals(lib):
    assert qz.plan_slots(1, 8, 128, 1) == 8 and qz.plan_slots(1, 8, 128, 128) == 8 * 128
    assert qz.plan_slots(100, 2, 3, 16) == 256 and qz.plan_slots(0, 2, 3, 16) == 0
    for bad in ((-1, 2, 3, 16), (4, 0, 3, 16), (4, 33, 64, 16), (4, 2, 0, 16), (4, 2, 1025, 16), (4, 2, 3, 0), (4, 2, 3, 3),
                (4, 2, 3, 2048)):
        assert qz.plan_slots(*bad) == 0
    assert lib.qz_plan_bytes(2048, 8, 128) == 0 and lib.qz_plan_bytes(2049, 8, 128) > 0
    assert lib.qz_plan_bytes(-1, 8, 128) == 0 and lib.qz_plan_bytes(1 << 20, 8, 0) == 0

    def plan(T=4, k=2, E=8, align=16, ids=A, off=A, cnt=A, rows=A, slots=A, ws=None, n=0):
        return lib.qz_plan_experts(P(ids), T, k, E, align, P(off), P(cnt), P(rows), P(slots), P(ws), n, None)

    for kw in (dict(T=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(align=0), dict(align=24), dict(ids=None),
               dict(off=None), dict(cnt=None), dict(rows=None), dict(slots=None), dict(T=9000), dict(T=9000, ws=A, n=8)):
        assert plan(**kw) == BAD, kw
    for kw in (dict(ids=A + 2), dict(off=A + 1), dict(rows=A + 2), dict(slots=A + 3), dict(cnt=A + 2)):
        assert plan(**kw) == ALIGN, kw


def product(lib, opts=None, **kw):
    base = dict(fmt=0, activation=0, n_experts=4, x_amax_per_row=0, n=64, k=128, x_rows=10, slots=20, x_q=A, x_sf=A,
                x_amax=None, d_rows=A, d_offsets=A, d_counts=A, w_q=A, w_sf=A, w_amax=None, up_q=None, up_sf=None,
                up_amax=None, w_stride=64 * 128, w_sf_stride=512, bias=None, up_bias=None, residual=None, ld_residual=0,
                out=A, ld_out=64, pre=None, ld_pre=0, q=None, sf=None)
    base.update(kw)
    return lib.qz_expert_product(ctypes.byref(qz.binding._Product(**base)), None, ctypes.byref(opts) if opts else None)


def test_product_refusals(lib):
    fp4 = dict(fmt=1, w_stride=64 * 64, w_sf_stride=1024, x_amax=A, w_amax=A)
    for kw in (dict(fmt=2), dict(activation=4), dict(activation=-1), dict(n_experts=0), dict(n_experts=1025), dict(n=0),
               dict(n=60), dict(k=0), dict(k=48), dict(x_rows=-1), dict(slots=-1), dict(slots=2 ** 31), dict(x_rows=2 ** 31),
               dict(w_stride=64 * 128 - 16), dict(w_stride=64 * 128 + 8), dict(w_sf_stride=496), dict(w_sf_stride=520),
               dict(ld_out=56), dict(ld_out=68), dict(residual=A, ld_residual=60), dict(pre=A, ld_pre=32),
               dict(up_sf=A), dict(up_bias=A), dict(up_amax=A), dict(q=A), dict(q=A, sf=A, n=40, ld_out=40),
               dict(up_q=A), dict(up_q=A, up_sf=A, pre=A, ld_pre=64), dict(d_offsets=None), dict(d_counts=None),
               dict(w_q=None), dict(w_sf=None), dict(out=None), dict(x_q=None), dict(x_sf=None), dict(fmt=1),
               dict(fp4, x_amax=None), dict(fp4, w_amax=None), dict(fp4, up_q=A, up_sf=A)):
        assert product(lib, **kw) == BAD, kw
    for kw in (dict(x_q=A + 8), dict(w_q=A + 8), dict(w_sf=A + 8), dict(out=A + 8), dict(residual=A + 2, ld_residual=64),
               dict(pre=A + 8, ld_pre=64), dict(q=A + 8, sf=A), dict(bias=A + 2), dict(x_sf=A + 2), dict(d_rows=A + 2),
               dict(d_offsets=A + 2), dict(d_counts=A + 1), dict(up_q=A + 8, up_sf=A), dict(up_q=A, up_sf=A + 8)):
        assert product(lib, **kw) == ALIGN, kw
    big = dict(slots=4096, x_rows=100)
    sized = qz.binding._Product(fmt=0, k=128, slots=4096, x_rows=100, d_rows=A)
    need = lib.qz_product_bytes(ctypes.byref(sized))
    assert need >= 4096 * (128 + 4)
    for field, value in (("slots", 100), ("d_rows", None), ("x_rows", 0), ("k", 48), ("fmt", 2), ("slots", -1)):
        other = qz.binding._Product.from_buffer_copy(sized)
        setattr(other, field, value)
        assert lib.qz_product_bytes(ctypes.byref(other)) == 0, field
    assert lib.qz_product_bytes(None) == 0
    assert product(lib, opts=qz.binding._Opts(None, 0, P(A), need - 1), **big) == BAD
    assert product(lib, opts=qz.binding._Opts(None, 0, P(A + 8), need), **big) == ALIGN
    assert product(lib, slots=0) == OK
    assert lib.qz_expert_product(None, None, None) == BAD


def test_rows_are_copied_where_that_pays(lib):
    """By slots, column blocks (256 columns, gated 128) and slots a row; the size is the workspace of such a call."""
    def size(slots, n=1024, x_rows=None, gated=False, fmt=0):
        p = qz.binding._Product(fmt=fmt, k=128, n=n, slots=slots, x_rows=slots if x_rows is None else x_rows, d_rows=A,
                                up_q=A if gated else None)
        return lib.qz_product_bytes(ctypes.byref(p))

    for gated in (False, True):
        assert size(2047, gated=gated) == 0 and size(2048, gated=gated) >= 2048 * (128 + 4)
        one = 128 if gated else 256
        assert size(8192, one, gated=gated) > 0 and size(8193, one, gated=gated) == 0
        assert size(8193, one + 8, gated=gated) > 0 and size(1 << 20, one + 8, gated=gated) > 0
        assert size(6400, x_rows=100, gated=gated) > 0 and size(6401, x_rows=100, gated=gated) == 0
    assert size(2048, fmt=1) >= 2048 * (64 + 8) and size(1 << 31) == 0 and size(4096, x_rows=0) == 0


def test_weight_grad_refusals(lib):
    def grad(**kw):
        base = dict(fmt=0, n_experts=4, out_type=1, accumulate=0, n=64, k=128, slots=256, dz_q=A, dz_sf=A, dz_amax=None,
                    x_q=A, x_sf=A, x_amax=None, d_offsets=A, d_counts=A, out=A)
        base.update(kw)
        return lib.qz_expert_weight_grad(ctypes.byref(qz.binding._WeightGrad(**base)), None, None)

    for kw in (dict(fmt=2), dict(out_type=2), dict(n_experts=0), dict(n_experts=1025), dict(n=4), dict(k=12), dict(slots=-32),
               dict(slots=250), dict(dz_q=None), dict(dz_sf=None), dict(x_q=None), dict(x_sf=None), dict(d_offsets=None),
               dict(d_counts=None), dict(out=None), dict(fmt=1), dict(fmt=1, dz_amax=A)):
        assert grad(**kw) == BAD, kw
    for kw in (dict(dz_q=A + 8), dict(x_q=A + 4), dict(dz_sf=A + 8), dict(x_sf=A + 1), dict(out=A + 4), dict(d_offsets=A + 2),
               dict(fmt=1, dz_amax=A + 1, x_amax=A)):
        assert grad(**kw) == ALIGN, kw
    assert lib.qz_expert_weight_grad(None, None, None) == BAD


def test_slot_refusals(lib):
    def act(ldd=64, ldp=64, slots=8, n=64, a=2, gated=0, off=A, cnt=A, E=3, dpre=A, ldq=64, dbias=None, dout=A, pre=A, opts=None):
        return lib.qz_expert_activation_grad(P(dout), ldd, P(pre), ldp, slots, n, a, gated, P(off), P(cnt), E, P(dpre), ldq,
                                             P(dbias), None, ctypes.byref(opts) if opts else None)

    for kw in (dict(n=4), dict(n=60), dict(a=4), dict(E=0), dict(E=1025), dict(slots=-1), dict(ldd=32), dict(ldp=60),
               dict(ldq=68), dict(gated=1), dict(off=None), dict(cnt=None), dict(dout=None), dict(pre=None), dict(dpre=None)):
        assert act(**kw) == BAD, kw
    for kw in (dict(dout=A + 8), dict(pre=A + 2), dict(dpre=A + 8), dict(dbias=A + 2), dict(off=A + 2)):
        assert act(**kw) == ALIGN, kw
    assert act(dbias=A) == BAD  # without its workspace
    need = lib.qz_activation_grad_bytes(8, 64, 0, 3)
    assert need >= 4 * 64 * 3 and lib.qz_activation_grad_bytes(8, 64, 1, 3) == 2 * need
    for bad in ((-1, 64, 0, 3), (8, 60, 0, 3), (8, 64, 0, 0), (8, 64, 0, 1025)):
        assert lib.qz_activation_grad_bytes(*bad) == 0
    assert act(dbias=A, opts=qz.binding._Opts(None, 0, P(A), need - 1)) == BAD
    assert act(dbias=A, opts=qz.binding._Opts(None, 0, P(A + 8), need)) == ALIGN

    def dispatch(x=A, ldx=64, slots=A, rows=A, T=4, k=2, S=8, H=64, w=None, y=A, ldy=64, o=None, ldo=0, dots=None):
        return lib.qz_dispatch_experts(P(x), ldx, P(slots), P(rows), T, k, S, H, P(w), P(y), ldy, P(o), ldo, P(dots), None)

    for kw in (dict(T=-1), dict(k=0), dict(k=33), dict(S=-1), dict(H=0), dict(H=60), dict(ldx=56), dict(ldy=65), dict(x=None),
               dict(slots=None), dict(rows=None), dict(y=None), dict(o=A, ldo=64), dict(dots=A), dict(o=A, ldo=8, dots=A)):
        assert dispatch(**kw) == BAD, kw
    for kw in (dict(x=A + 8), dict(y=A + 8), dict(o=A + 8, ldo=64, dots=A), dict(slots=A + 1), dict(rows=A + 2), dict(w=A + 1)):
        assert dispatch(**kw) == ALIGN, kw
    assert dispatch(T=0, S=0) == OK

    def combine(y=A, ldy=64, slots=A, T=4, k=2, S=8, H=64, w=None, r=None, ldr=0, out=A, ldo=64):
        return lib.qz_combine_experts(P(y), ldy, P(slots), T, k, S, H, P(w), P(r), ldr, P(out), ldo, None)

    for kw in (dict(T=-1), dict(k=33), dict(S=-1), dict(H=12), dict(ldy=8), dict(ldo=72 + 4), dict(r=A, ldr=32), dict(y=None),
               dict(out=None), dict(slots=None)):
        assert combine(**kw) == BAD, kw
    for kw in (dict(y=A + 8), dict(out=A + 4), dict(r=A + 8, ldr=64), dict(slots=A + 2), dict(w=A + 2)):
        assert combine(**kw) == ALIGN, kw
    assert combine(T=0) == OK


def test_binding_refuses_what_it_cannot_pass_on(lib):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="current CUDA device"):
        qz.route_experts(x, 2)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        qz.route_experts(x.double(), 2)
    with pytest.raises(ValueError, match="rows of logits"):
        qz.route_experts(torch.zeros(8, 4).T, 2)
    with pytest.raises(ValueError, match="ids"):
        qz.plan_experts(torch.zeros(4, 2), 8)
    with pytest.raises(ValueError, match="payload"):
        qz.expert_product(qz.FMT_MXFP8, torch.zeros(4, 8), None, None, None, None)
    with pytest.raises(ValueError, match="fmt"):
        q, w = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(2, 8, 32, dtype=torch.uint8)
        qz.expert_product(qz.FMT_FP8_BLOCK128, (q, q), (w, q), None, None, torch.zeros(4, 8))


def test_the_stride_of_a_single_row_does_not_matter():
    t = torch.zeros(64, dtype=torch.bfloat16).as_strided((1, 8), (13, 1))
    assert qz.binding._matrix(t, "t", torch.bfloat16, -1, (1, 8)) == (t.data_ptr(), 8)
    t = torch.zeros(64, dtype=torch.bfloat16).as_strided((2, 8), (16, 1))
    assert qz.binding._matrix(t, "t", torch.bfloat16, -1, (2, 8)) == (t.data_ptr(), 16)


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """Outputs and scratch of a call with a stream of its own come from that stream's pool: a block of the current
    stream's may still be in use there.  (The launches are stubs: this runs without a GPU.)"""
    b = qz.binding
    inside, made = [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    class Library:
        def __getattr__(self, name):
            return lambda *a: 64 if name.endswith("bytes") else 0

    new_empty = torch.Tensor.new_empty

    def recorded(t, *a, **kw):
        made.append(list(inside))
        return new_empty(t, *a, **kw)

    monkeypatch.setattr(b, "_on", on)
    monkeypatch.setattr(b, "load", Library)
    monkeypatch.setattr(b, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(b, "_plan_sizes", lambda *a: (64, 64))
    monkeypatch.setattr(b, "_region", lambda *a: 512)
    monkeypatch.setattr(torch.Tensor, "new_empty", recorded)
    i32, bf, u8 = torch.int32, torch.bfloat16, torch.uint8
    x, ids, lists = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32), torch.zeros(3, dtype=i32)
    rows = torch.zeros(4, 8, dtype=bf)
    calls = {
        "route": (2, lambda s: qz.route_experts(x, 2, stream=s)),
        "route_grad": (1, lambda s: qz.route_experts_grad(x, ids, torch.zeros(4, 2), stream=s)),
        "plan": (2, lambda s: qz.plan_experts(ids, 5, stream=s)),
        "product": (1, lambda s: qz.expert_product(
            qz.FMT_MXFP8, (torch.zeros(4, 32, dtype=u8), torch.zeros(4, 1, dtype=u8)),
            (torch.zeros(3, 8, 32, dtype=u8), torch.zeros(3, 512, dtype=u8)), lists, lists, rows, rows=lists.new_zeros(4),
            stream=s)),
        "activation_grad": (1, lambda s: qz.expert_activation_grad(
            rows, rows, lists, lists, rows.clone(), activation=qz.ACT_SILU, dbias=torch.zeros(3, 8), stream=s)),
    }
    for name, (n, call) in calls.items():
        for stream in (object(), None):
            made.clear()
            call(stream)
            assert made == [[] if stream is None else [stream]] * n, name
