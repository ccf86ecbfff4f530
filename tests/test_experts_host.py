"""CPU-only checks of the experts' products (ep_expert_fp8, ep_expert_ffn, ep_expert_ffn_backward): the structures match
the header, bad arguments are refused on the host before any CUDA call (the addresses here are never dereferenced), and
the binding refuses what the C ABI cannot see."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID = 1
BF16, E4M3, E5M2, FP16, FP32 = range(5)


@pytest.fixture(scope="module")
def ep():
    from combine_get_dispatch_layout_gb300.build import build
    import combine_get_dispatch_layout_gb300 as ep

    build()
    ep.lib()
    return ep


def test_structures_match_the_header(ep, tmp_path):
    structs = {"ep_fp8_config_t": ep.layer.Fp8Config, "ep_ffn_config_t": ep.layer.FfnConfig}
    lines = []
    for c, py in structs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        for field, _ in py._fields_:
            lines.append(f'printf("{c}.{field} %zu\\n", offsetof({c}, {field}));')
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ep_layer.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", exe], check=True)
    got = dict(x.split() for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines())
    for c, py in structs.items():
        assert int(got.pop(c)) == ctypes.sizeof(py)
        for field, _ in py._fields_:
            assert int(got.pop(f"{c}.{field}")) == getattr(py, field).offset, (c, field)
    assert not got


def fp8(ep, **kw):
    a = dict(x=16, xs=16, rows=4, I=256, w=16, ws=16, off=16, cnt=None, E=2, O=256, y=16, ys=16, x_dtype=E4M3, y_dtype=BF16,
             act=0, x_mode=0, y_mode=0, x_ld=256, y_ld=256, xr=2, xb=1, yr=2, yb=1, cfg=True)
    a.update(kw)
    cfg = ep.layer.Fp8Config(a["x_dtype"], a["y_dtype"], a["act"], a["x_mode"], a["y_mode"], a["x_ld"], a["y_ld"], a["xr"],
                             a["xb"], a["yr"], a["yb"])
    return ep.lib().ep_expert_fp8(a["x"], a["xs"], a["rows"], a["I"], a["w"], a["ws"], a["off"], a["cnt"], a["E"], a["O"],
                                  cfg if a["cfg"] else None, a["y"], a["ys"], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=24), dict(xs=None), dict(xs=18), dict(rows=-1), dict(rows=1 << 31), dict(I=0), dict(I=192, x_ld=192),
    dict(w=None), dict(w=24), dict(ws=None), dict(ws=18), dict(off=None), dict(off=18), dict(cnt=18),
    dict(off=None, E=1, cnt=16), dict(E=0), dict(E=4097), dict(O=0), dict(O=1 << 31 - 1, I=1 << 20, x_ld=1 << 20, y_ld=1 << 31),
    dict(y=None), dict(y=17), dict(x_dtype=BF16), dict(x_dtype=FP16), dict(y_dtype=E5M2), dict(y_dtype=FP32), dict(act=2),
    dict(act=1, O=255), dict(x_mode=3), dict(x_mode=-1), dict(x_ld=240), dict(x_ld=264), dict(x_ld=1 << 40), dict(y_ld=255),
    dict(xr=-1), dict(xb=-1), dict(cfg=False),
    dict(y_dtype=E4M3, ys=None), dict(y_dtype=E4M3, ys=18), dict(y_dtype=E4M3, O=200), dict(y_dtype=E4M3, act=1, O=384),
    dict(y_dtype=E4M3, y_mode=3), dict(y_dtype=E4M3, yr=0), dict(y_dtype=E4M3, yb=0)])
def test_fp8_rejects(ep, kw):
    assert fp8(ep, **kw) == INVALID


def ffn(ep, backward, **kw):
    a = dict(x=16, rows=4, H=64, up=16, down=16, off=16, cnt=None, E=2, F=32, gate_up=16, act=16, y=16, dgu=16, dx=16, dup=16,
             ddown=16, dtype=BF16, wdtype=BF16, acc=0, x_ld=64, gu_ld=64, act_ld=32, y_ld=64, dx_ld=64, dgu_ld=64, cfg=True)
    a.update(kw)
    cfg = ep.layer.FfnConfig(a["dtype"], a["wdtype"], a["acc"], a["x_ld"], a["gu_ld"], a["act_ld"], a["y_ld"], a["dx_ld"],
                             a["dgu_ld"])
    cfg = cfg if a["cfg"] else None
    if backward:
        return ep.lib().ep_expert_ffn_backward(a["y"], a["x"], a["gate_up"], a["act"], a["rows"], a["H"], a["up"], a["down"],
                                               a["off"], a["cnt"], a["E"], a["F"], cfg, a["dgu"], a["dx"], a["dup"],
                                               a["ddown"], None)
    return ep.lib().ep_expert_ffn(a["x"], a["rows"], a["H"], a["up"], a["down"], a["off"], a["cnt"], a["E"], a["F"], cfg,
                                  a["gate_up"], a["act"], a["y"], None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=24), dict(rows=-1), dict(rows=1 << 31), dict(H=0), dict(H=60), dict(F=0), dict(F=36), dict(up=None),
    dict(up=24), dict(down=None), dict(down=24), dict(off=None), dict(off=18), dict(cnt=18), dict(off=None, E=1, cnt=16),
    dict(E=0), dict(E=4097), dict(gate_up=24), dict(act=None), dict(act=24), dict(y=24), dict(dtype=E4M3, wdtype=E4M3),
    dict(dtype=FP32, wdtype=FP32), dict(x_ld=56), dict(x_ld=68), dict(x_ld=1 << 40), dict(gu_ld=56), dict(gu_ld=66),
    dict(act_ld=24), dict(act_ld=33), dict(y_ld=56), dict(y_ld=65), dict(cfg=False),
    dict(H=1 << 30, F=1 << 20, x_ld=1 << 30, y_ld=1 << 30, dx_ld=1 << 30, gu_ld=1 << 21, dgu_ld=1 << 21, act_ld=1 << 20)])
def test_block_rejects(ep, backward, kw):
    assert ffn(ep, backward, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(y=None), dict(gate_up=None), dict(dgu=None), dict(dgu=24), dict(dx=24), dict(dup=24),
                                dict(ddown=24), dict(wdtype=FP16), dict(wdtype=E4M3), dict(dx_ld=56), dict(dx_ld=68),
                                dict(dgu_ld=56), dict(dgu_ld=70)])
def test_block_backward_rejects(ep, kw):
    assert ffn(ep, True, **kw) == INVALID


def test_empty_calls_need_nothing(ep):
    assert fp8(ep, rows=0, x=None, xs=None, w=None, ws=None, y=None, ys=None) == 0
    assert ffn(ep, False, rows=0, x=None, up=None, down=None, act=None, y=None, gate_up=None) == 0
    assert ffn(ep, True, rows=0, acc=1, x=None, up=None, down=None, act=None, y=None, gate_up=None, dgu=None, dx=None) == 0


# ------------------------------------------------------------------ the binding

def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype)


def bound_fp8(ep, **kw):
    f8 = torch.float8_e4m3fn
    a = dict(x=empty(0, 256, dtype=f8), x_scales=empty(0, 2, dtype=torch.float32), weights=empty(0, 256, 256, dtype=f8),
             weight_scales=empty(0, 2, 2, dtype=torch.float32), y=empty(0, 256), expert_offsets=None, stream=0)
    a.update(kw)
    ep.ep_expert_fp8(**a)


F8, F32 = torch.float8_e4m3fn, torch.float32


@pytest.mark.parametrize("kw,match", [
    (dict(x=empty(0, 256)), "x"), (dict(x=empty(0, 256, dtype=torch.uint8)), "x"), (dict(x=empty(256, dtype=F8)), "dimensions"),
    (dict(x_scales=empty(0, 3, dtype=F32)), "x_scales"), (dict(x_scales=empty(0, 2)), "x_scales"),
    (dict(x_scales=empty(0, 2, dtype=torch.float64)), "x_scales"),
    (dict(weights=empty(0, 256, 128, dtype=F8)), "weights"), (dict(weights=empty(0, 256, 256)), "weights"),
    (dict(weights=empty(0, 256, 256, dtype=torch.float8_e5m2)), "weights"),
    (dict(weight_scales=empty(0, 2, 1, dtype=F32)), "weight_scales"), (dict(weight_scales=None), "weight_scales"),
    (dict(y=empty(0, 128)), "y"), (dict(y=empty(0, 256, dtype=F32)), "y"), (dict(y=empty(0, 256, dtype=F8)), "y_scales"),
    (dict(y=empty(0, 256, dtype=F8), y_scales=empty(0, 1, dtype=F32)), "y_scales"),
    (dict(y=empty(0, 256, dtype=F8), y_scales=empty(0, 2, dtype=F32), scale_mode=2), "bytes"),
    (dict(expert_offsets=empty(2, dtype=torch.int32)), "expert_offsets"),
    (dict(expert_offsets=empty(1, dtype=torch.int64)), "expert_offsets"),
    (dict(x=empty(2, 256, dtype=F8), x_scales=empty(2, 2, dtype=F32), y=empty(2, 256)), "CUDA")])
def test_fp8_binding_refuses(ep, kw, match):
    with pytest.raises(ValueError, match=match):
        bound_fp8(ep, **kw)


def test_scales_that_overlap_are_refused_as_an_output(ep, monkeypatch):
    from torch._subclasses import fake_tensor

    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda *a: None)   # (the GPU need not exist)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with fake_tensor.FakeTensorMode():   # tensors that say where they are and have no memory
        scales = torch.empty(1, 2, device="cuda:0").expand(4, 2)
        y = torch.empty(4, 256, dtype=F8, device="cuda:0")
    with pytest.raises((ValueError, RuntimeError)):
        bound_fp8(ep, y=y, y_scales=scales)


def bound_ffn(ep, **kw):
    a = dict(x=empty(0, 64), w_gate_up=empty(2, 64, 64)[:0], w_down=empty(2, 64, 32)[:0], act=empty(0, 32), y=empty(0, 64), stream=0)
    a.update(kw)
    ep.ep_expert_ffn(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(x=empty(0, 64, dtype=F32)), "x"), (dict(x=empty(64)), "dimensions"), (dict(act=empty(0, 32, dtype=torch.float16)), "act"),
    (dict(w_gate_up=empty(0, 32, 64)), "w_gate_up"), (dict(w_down=empty(0, 32, 64)), "w_down"), (dict(w_down=None), "together"),
    (dict(y=None), "together"), (dict(y=empty(0, 32)), "y"), (dict(gate_up=empty(0, 32)), "gate_up"),
    (dict(x=empty(3, 64), act=empty(3, 32), y=empty(3, 64)), "CUDA"), (dict(expert_counts=empty(3, dtype=torch.int32)), "expert_counts")])
def test_block_binding_refuses(ep, kw, match):
    with pytest.raises(ValueError, match=match):
        bound_ffn(ep, **kw)


def bound_backward(ep, **kw):
    a = dict(grad_y=empty(0, 64), x=empty(0, 64), gate_up=empty(0, 64), act=empty(0, 32), w_gate_up=empty(0, 64, 64),
             w_down=empty(0, 64, 32), grad_gate_up=empty(0, 64), grad_x=empty(0, 64), stream=0)
    a.update(kw)
    ep.ep_expert_ffn_backward(**a)


@pytest.mark.parametrize("kw,match", [
    (dict(grad_y=None), "grad_y"), (dict(gate_up=None), "gate_up"), (dict(w_down=None), "w_down"), (dict(grad_gate_up=None), "grad_gate_up"),
    (dict(grad_x=empty(0, 32)), "grad_x"), (dict(grad_w_down=empty(0, 32, 64)), "grad_w_down"),
    (dict(grad_w_gate_up=empty(0, 64, 64, dtype=F32), grad_w_down=empty(0, 64, 32)), "grad_w_down"),
    (dict(grad_w_down=empty(0, 64, 32, dtype=torch.float16)), "grad_w_down"), (dict(w_gate_up=empty(0, 64, 32)), "w_gate_up")])
def test_block_backward_binding_refuses(ep, kw, match):
    with pytest.raises(ValueError, match=match):
        bound_backward(ep, **kw)


def test_accumulate_needs_a_truth_value(ep):
    with pytest.raises(RuntimeError, match="ambiguous"):
        bound_backward(ep, accumulate=torch.tensor([1, 1]))
