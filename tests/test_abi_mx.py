"""Argument checks and sizes of the scored router and the MXFP4 entry points,
without a GPU: every refusal comes before any device work."""

import ctypes

import pytest
import torch

import __graft_entry__
from nvfp4_block_scaled_topk_gb300 import megamoe

P = None
F = ctypes.c_void_p(256)  # an aligned address that is never touched
ODD = ctypes.c_void_p(257)
INVALID, SHAPE, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return megamoe.load()


def _route(lib, logits=F, kind=1, T=4, E=8, ld=8, bias=P, score=0, n_group=1, topk_group=1, top=2,
           k=2, ids=F, w=F):
    return lib.megamoe_router_scored_topk(logits, kind, T, E, ld, bias, score, n_group, topk_group,
                                          top, k, 1, 1.0, ids, w, P)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(ld=7), INVALID), (dict(k=0), INVALID),
    (dict(k=9), INVALID), (dict(kind=2), INVALID), (dict(kind=7), INVALID), (dict(score=2), INVALID),
    (dict(n_group=0), INVALID), (dict(n_group=3), INVALID), (dict(n_group=4, topk_group=5), INVALID),
    (dict(topk_group=0), INVALID), (dict(top=3), INVALID), (dict(top=0), INVALID),
    (dict(logits=P), INVALID), (dict(ids=P), INVALID), (dict(w=P), INVALID),
    (dict(E=1025, ld=1025), SHAPE), (dict(E=64, ld=64, n_group=64), SHAPE),
    (dict(E=32, ld=32, k=17), SHAPE), (dict(T=1 << 31), SHAPE), (dict(logits=ODD), SHAPE),
    (dict(bias=ODD), SHAPE), (dict(ids=ODD), SHAPE), (dict(w=ODD), SHAPE)])
def test_router_refusals(lib, change, code):
    assert _route(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(ld_grad=7), INVALID), (dict(ids=P), INVALID), (dict(g=P), INVALID),
    (dict(out=P), INVALID), (dict(kind=2), INVALID), (dict(score=5), INVALID), (dict(out=ODD), SHAPE),
    (dict(g=ODD), SHAPE), (dict(E=2000, ld=2000, ld_grad=2000), SHAPE)])
def test_router_backward_refusals(lib, change, code):
    a = dict(logits=F, kind=1, T=4, E=8, ld=8, ids=F, g=F, score=0, k=2, out=F, ld_grad=8) | change
    assert lib.megamoe_router_scored_topk_backward(
        a["logits"], a["kind"], a["T"], a["E"], a["ld"], a["ids"], a["g"], a["score"], a["k"], 1, 1.0,
        a["out"], a["ld_grad"], P) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(ld=32), INVALID), (dict(kind=3), INVALID),
    (dict(layout=2), INVALID), (dict(x=P), INVALID), (dict(codes=P), INVALID),
    (dict(scales=P), INVALID), (dict(K=48), SHAPE), (dict(ld=68), SHAPE), (dict(x=ODD), SHAPE),
    (dict(codes=ODD), SHAPE), (dict(rows=1 << 31), SHAPE)])
def test_quantise_refusals(lib, change, code):
    a = dict(x=F, kind=0, rows=4, K=64, ld=64, t=0, codes=F, scales=F, layout=0) | change
    assert lib.megamoe_quantize_mxfp4(a["x"], a["kind"], a["rows"], a["K"], a["ld"], a["t"],
                                      a["codes"], a["scales"], a["layout"], P, P) == code


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(kind=2), INVALID), (dict(ld=32), INVALID), (dict(codes=P), INVALID),
    (dict(out=P), INVALID), (dict(K=40, ld=40), SHAPE), (dict(ld=66), SHAPE), (dict(out=ODD), SHAPE)])
def test_dequantise_refusals(lib, change, code):
    a = dict(codes=F, scales=F, rows=4, K=64, out=F, kind=0, ld=64) | change
    assert lib.megamoe_dequantize_mxfp4(a["codes"], a["scales"], a["rows"], a["K"], a["out"],
                                        a["kind"], a["ld"], P) == code
    assert lib.megamoe_swizzle_scales_mxfp4(F, 4, 40, F, P) == SHAPE
    assert lib.megamoe_swizzle_scales_mxfp4(P, 4, 64, F, P) == INVALID


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(ld_x=32), INVALID), (dict(ld_out=32), INVALID),
    (dict(kind=9), INVALID), (dict(epi=1), INVALID), (dict(epi=3), INVALID), (dict(x=P), INVALID),
    (dict(out=P), INVALID), (dict(w=P), INVALID), (dict(ws=P), INVALID), (dict(K=48), SHAPE),
    (dict(N=80, ld_out=80), SHAPE), (dict(ld_x=68), SHAPE), (dict(ld_out=68), SHAPE),
    (dict(x=ODD), SHAPE), (dict(w=ODD), SHAPE), (dict(ws=ODD), SHAPE), (dict(T=1 << 30), SHAPE),
    (dict(T=1 << 29, N=1 << 30, ld_out=1 << 30), SHAPE), (dict(bytes=10), SMALL)])
def test_linear_refusals(lib, change, code):
    a = dict(x=F, kind=0, T=100, K=64, ld_x=64, w=F, N=64, epi=2, out=F, ld_out=64, ws=F,
             bytes=1 << 30) | change
    assert lib.megamoe_linear_mxfp4(a["x"], a["kind"], a["T"], a["K"], a["ld_x"], a["w"], F, a["N"],
                                    a["epi"], a["out"], a["ld_out"], a["ws"], a["bytes"], P) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(g=P), INVALID), (dict(x=P), INVALID), (dict(w=P), INVALID),
    (dict(ws=P), INVALID), (dict(kind=9), INVALID), (dict(epi=1), INVALID), (dict(ld_g=32), INVALID),
    (dict(ld_x=32), INVALID), (dict(ld_w=32), INVALID), (dict(ld_gx=32), INVALID),
    (dict(ld_gw=32), INVALID), (dict(K=48), SHAPE), (dict(N=48), SHAPE), (dict(ld_w=65), SHAPE),
    (dict(g=ODD), SHAPE), (dict(gx=ODD), SHAPE), (dict(gw=ODD), SHAPE), (dict(bytes=10), SMALL)])
def test_linear_backward_refusals(lib, change, code):
    a = dict(g=F, kind=0, ld_g=64, x=F, ld_x=64, w=F, ld_w=64, T=100, K=64, N=64, gx=F, epi=2,
             ld_gx=64, gw=F, ld_gw=64, ws=F, bytes=1 << 30) | change
    assert lib.megamoe_linear_mxfp4_backward(
        a["g"], a["kind"], a["ld_g"], a["x"], a["kind"], a["ld_x"], a["w"], a["kind"], a["ld_w"],
        a["T"], a["K"], a["N"], a["gx"], a["epi"], a["ld_gx"], a["gw"], a["epi"], a["ld_gw"], a["ws"],
        a["bytes"], P) == code


@pytest.mark.parametrize("change,code", [
    (dict(w=P), INVALID), (dict(x=P), INVALID), (dict(ids=P), INVALID), (dict(out=P), INVALID),
    (dict(ws=P), INVALID), (dict(k=0), INVALID), (dict(pad=16), SHAPE), (dict(x=ODD), SHAPE),
    (dict(bytes=100), SMALL), (dict(k=17), SHAPE)])
def test_experts_refusals(lib, change, code):
    good = megamoe.CMxWeights(8, 256, 512, 256, 256, 256, 256)
    a = dict(w=ctypes.byref(good), x=F, ids=F, T=4, k=2, pad=32, out=F, ws=F, bytes=1 << 30) | change
    assert lib.megamoe_forward_mxfp4(a["w"], a["x"], a["ids"], F, a["T"], a["k"], a["pad"], a["out"],
                                     a["ws"], a["bytes"], P) == code
    for bad in (megamoe.CMxWeights(8, 200, 512, 256, 256, 256, 256),
                megamoe.CMxWeights(8, 256, 500, 256, 256, 256, 256),
                megamoe.CMxWeights(1024, 1 << 20, 1 << 20, 256, 256, 256, 256)):
        assert lib.megamoe_forward_mxfp4(ctypes.byref(bad), F, F, F, 4, 2, 32, F, F, 1 << 62,
                                         P) == SHAPE
    assert lib.megamoe_forward_mxfp4_from_logits(ctypes.byref(good), F, F, 1, 8, P, 0, 3, 1, 2, 1, 1.0,
                                                 4, 2, 32, F, F, 1 << 30, P) == INVALID
    assert lib.megamoe_forward_mxfp4_from_logits(ctypes.byref(good), F, P, 1, 8, P, 0, 1, 1, 2, 1, 1.0,
                                                 4, 2, 32, F, F, 1 << 30, P) == INVALID


def test_sizes(lib):
    assert megamoe.mx_atom_bytes(1, 32) == 128 * 8 and megamoe.mx_atom_bytes(129, 288) == 256 * 16
    small = lib.megamoe_workspace_size_mxfp4(8, 6, 384, 7168, 2048, 32)
    assert 0 < small < lib.megamoe_workspace_size_mxfp4(16, 6, 384, 7168, 2048, 32)
    assert small < lib.megamoe_workspace_size(8, 6, 384, 7168, 2048, 32)  # no bf16 h
    assert lib.megamoe_workspace_size_mxfp4(8, 0, 384, 7168, 2048, 32) == 0
    assert lib.megamoe_linear_mxfp4_workspace_size(-1, 64, 64) == 0
    assert lib.megamoe_linear_mxfp4_workspace_size(4096, 1536, 24576) >= 4096 * 1536 * 17 // 32
    assert lib.megamoe_linear_mxfp4_backward_workspace_size(333, 1536, 2048) >= (
        333 * 2048 + 352 * 2048 + 352 * 1536 + 1536 * 2048) * 17 // 32


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    x = torch.zeros(4, 64)
    for f in (lambda: megamoe.router_scored_topk(x, 2), lambda: megamoe.quantize_mxfp4(x),
              lambda: megamoe.linear_mxfp4_backward(x, x, x),
              lambda: megamoe.dequantize_mxfp4(x.to(torch.uint8), x.to(torch.uint8))):
        with pytest.raises(TypeError):
            f()


def test_mx_weights_struct_matches_the_header():
    import os
    import re

    from test_abi import ROOT, _c_to_ctypes

    src = open(os.path.join(ROOT, "include", "megamoe.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    body = re.search(r"typedef struct megamoe_mx_weights\s*\{(.*?)\}", src, re.S).group(1)
    fields = []
    for decl in body.split(";"):
        decl = " ".join(decl.split())
        if decl:
            name = re.search(r"([A-Za-z_]\w*)$", decl).group(1)
            fields.append((name, _c_to_ctypes(decl[: -len(name)])))
    assert list(megamoe.CMxWeights._fields_) == fields
